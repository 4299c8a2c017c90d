"""Argument checks of the 8-bit norm and FP8 x FP8 entry points, before any device work (no GPU)."""
import ctypes

import pytest

from block_quantized_weight_route_gb300 import build as qbuild

P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
INVALID, SHAPE = 1, 2
A = P(256)


@pytest.fixture(scope="module")
def L():
    L = ctypes.CDLL(qbuild.build_library())
    norm = [P, i32, i64, P, i64, P, i64, i32, P, i32, f32, i32, i32]
    L.qmm_add_rmsnorm_fp8.argtypes = norm + [P] * 4
    L.qmm_add_rmsnorm_q8_1.argtypes = norm + [P] * 5
    L.qmm_fp8a8_blk128.argtypes = [P, P, i32, i32, i32, P, P, P, i32, P]
    L.qmm_fp8a8_swiglu_blk128.argtypes = [P, P, i32, i32, i32, P, P, P, P, P]
    L.qmm_last_error.restype = ctypes.c_char_p
    return L


def norm_args(**kw):
    a = dict(X=A, xdt=1, ldx=256, R=None, ldr=0, Rout=None, ldro=0, rdt=0, G=A, gdt=1, eps=1e-6, T=4, D=256)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("kw,st", [
    (dict(D=200, ldx=208), SHAPE), (dict(D=0), SHAPE), (dict(T=-1), SHAPE), (dict(D=16400, ldx=16400), SHAPE),
    (dict(X=None), INVALID), (dict(G=None), INVALID), (dict(xdt=2), INVALID), (dict(gdt=-1), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(eps=float("nan")), INVALID), (dict(ldx=128), INVALID), (dict(ldx=260), INVALID),
    (dict(X=P(264)), INVALID), (dict(R=A, ldr=256), INVALID), (dict(Rout=A, ldro=256), INVALID),
    (dict(R=A, ldr=256, Rout=A, ldro=128), INVALID), (dict(R=A, ldr=256, Rout=A, ldro=256, rdt=7), INVALID),
])
def test_norm(L, kw, st):
    assert L.qmm_add_rmsnorm_fp8(*norm_args(**kw), A, A, None, None) == st
    assert b"qmm_add_rmsnorm_fp8" in L.qmm_last_error()
    assert L.qmm_add_rmsnorm_q8_1(*norm_args(**kw), A, A, A, None, None) == st
    assert b"qmm_add_rmsnorm_q8_1" in L.qmm_last_error()


def test_norm_outputs(L):
    assert L.qmm_add_rmsnorm_fp8(*norm_args(), None, A, None, None) == INVALID
    assert L.qmm_add_rmsnorm_fp8(*norm_args(), A, None, None, None) == INVALID
    assert L.qmm_add_rmsnorm_fp8(*norm_args(), A, A, P(260), None) == INVALID
    assert L.qmm_add_rmsnorm_q8_1(*norm_args(), A, A, None, None, None) == INVALID
    assert L.qmm_add_rmsnorm_q8_1(*norm_args(D=240, ldx=240), A, A, A, None, None) == SHAPE   # not a multiple of 32


def test_products(L):
    f, g = L.qmm_fp8a8_blk128, L.qmm_fp8a8_swiglu_blk128
    assert f(A, A, 4, 200, 256, A, A, A, 1, None) == SHAPE
    assert f(A, A, 4, 0, 256, A, A, A, 1, None) == SHAPE
    assert f(A, A, 4, 256, 0, A, A, A, 1, None) == SHAPE
    assert f(A, A, -1, 256, 256, A, A, A, 1, None) == SHAPE
    assert f(A, A, 4, 256, 256, A, A, A, 2, None) == INVALID
    assert b"qmm_fp8a8_blk128" in L.qmm_last_error()
    for i in (0, 1, 5, 6, 7):
        args = [A, A, 4, 256, 256, A, A, A, 1, None]
        args[i] = None
        assert f(*args) == INVALID
        args[i] = P(264)
        assert f(*args) == INVALID
    assert g(A, A, 4, 256, 192, A, A, A, A, None) == SHAPE
    assert g(A, A, 4, 100, 256, A, A, A, A, None) == SHAPE
    for i in (0, 1, 5, 6, 7, 8):
        args = [A, A, 4, 256, 256, A, A, A, A, None]
        args[i] = None
        assert g(*args) == INVALID
        args[i] = P(264)
        assert g(*args) == INVALID
    assert b"qmm_fp8a8_swiglu_blk128" in L.qmm_last_error()


def test_sizes_whose_tiles_pass_32_bits(L):
    top = 2 ** 31 - 511
    assert L.qmm_add_rmsnorm_fp8(*norm_args(T=top), A, A, None, None) == SHAPE
    assert L.qmm_fp8a8_blk128(A, A, top, 256, 256, A, A, A, 1, None) == SHAPE
    assert L.qmm_fp8a8_blk128(A, A, 1, 2 ** 31 - 16, 1, A, A, A, 1, None) == SHAPE
    assert L.qmm_fp8a8_blk128(A, A, 1, 16, top, A, A, A, 1, None) == SHAPE
    assert L.qmm_fp8a8_swiglu_blk128(A, A, top, 256, 256, A, A, A, A, None) == SHAPE
    assert L.qmm_fp8a8_swiglu_blk128(A, A, 1, 16, 2 ** 30, A, A, A, A, None) == SHAPE
