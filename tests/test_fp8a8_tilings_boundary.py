"""Argument checks of the FP8 x FP8 products by a given tiling, before any device work (no GPU)."""
import ctypes

import pytest

from block_quantized_weight_route_gb300 import build as qbuild

P, i32 = ctypes.c_void_p, ctypes.c_int
INVALID, SHAPE = 1, 2
A = P(256)


@pytest.fixture(scope="module")
def L():
    L = ctypes.CDLL(qbuild.build_library())
    L.qmm_dbg_fp8a8_plan.argtypes = [i32, i32, i32, i32, P]
    L.qmm_dbg_fp8a8_blk128.argtypes = [P, P, i32, i32, i32, P, P, P, i32, P, P]
    L.qmm_dbg_fp8a8_swiglu_blk128.argtypes = [P, P, i32, i32, i32, P, P, P, P, P, P]
    L.qmm_last_error.restype = ctypes.c_char_p
    return L


def plan(first, second=(0, 0, 0, 0), split=256):
    return ctypes.cast((i32 * 9)(*first, *second, split), P)


def test_the_products_own_checks_come_first(L):
    pl = plan((1, 256, 0, 0))
    assert L.qmm_dbg_fp8a8_blk128(A, A, 4, 200, 256, A, A, A, 1, pl, None) == SHAPE
    assert L.qmm_dbg_fp8a8_blk128(A, A, 4, 256, 256, A, A, None, 1, pl, None) == INVALID
    assert L.qmm_dbg_fp8a8_blk128(A, A, 4, 256, 256, A, A, A, 1, None, None) == INVALID
    assert b"qmm_dbg_fp8a8_blk128" in L.qmm_last_error()
    assert L.qmm_dbg_fp8a8_swiglu_blk128(A, A, 4, 256, 192, A, A, A, A, pl, None) == SHAPE
    assert L.qmm_dbg_fp8a8_swiglu_blk128(A, A, 4, 256, 256, A, A, A, A, None, None) == INVALID
    assert b"qmm_dbg_fp8a8_swiglu_blk128" in L.qmm_last_error()
    assert L.qmm_dbg_fp8a8_plan(4, 256, 256, 0, None) == INVALID
    assert L.qmm_dbg_fp8a8_plan(0, 256, 256, 0, pl) == SHAPE
    assert L.qmm_dbg_fp8a8_plan(4, 200, 256, 0, pl) == SHAPE
    assert L.qmm_dbg_fp8a8_plan(4, 256, 200, 1, pl) == SHAPE


@pytest.mark.parametrize("first,second,split", [
    ((1, 64, 0, 0), (0, 0, 0, 0), 256),         # no such pair tile
    ((0, 0, 8, 1), (0, 0, 0, 0), 256),          # no such narrow tile
    ((0, 0, 16, 3), (0, 0, 0, 0), 256),         # more CTAs than K blocks
    ((0, 0, 16, 0), (0, 0, 0, 0), 256),
    ((0, 0, 16, 9), (0, 0, 0, 0), 256),
    ((1, 192, 0, 0), (1, 128, 0, 0), 128),      # a tile of the first launch would reach into the second's columns
    ((0, 0, 16, 1), (1, 128, 0, 0), 64),        # not at a weight block
    ((1, 256, 0, 0), (0, 0, 0, 0), 512),
    ((1, 256, 0, 0), (0, 0, 0, 0), 0),
    ((0, 0, 16, 1), (0, 0, 0, 0), 128),         # no second tiling
])
def test_tilings_that_do_not_fit(L, first, second, split):
    assert L.qmm_dbg_fp8a8_blk128(A, A, 4, 256, 256, A, A, A, 1, plan(first, second, split), None) == INVALID
    assert b"no such tiling" in L.qmm_last_error()
    assert L.qmm_dbg_fp8a8_swiglu_blk128(A, A, 4, 256, 256, A, A, A, A, plan((1, 128, 0, 0)), None) == INVALID
    assert b"no such tiling" in L.qmm_last_error()
