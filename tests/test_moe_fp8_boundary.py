"""Argument checks of the router by scores, the FP8 expert stage and the product with an epilogue,
before any device work (no GPU)."""
import ctypes

import pytest

from block_quantized_weight_route_gb300 import build as qbuild

P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
INVALID, SHAPE, WORKSPACE = 1, 2, 4
A, ODD = P(256), P(264)


@pytest.fixture(scope="module")
def L():
    L = ctypes.CDLL(qbuild.build_library())
    L.moe_route_scored.argtypes = [P, i32, i64, P, P, i32, i32, i32, i32, i32, i32, i32, i32, f32, P, P, P]
    L.qmm_fp8a8_epilogue_blk128.argtypes = [P, P, i32, i32, i32, P, P, P, i32, i32, P, i64, i32, P, i32, P]
    L.moe_expert_stage_fp8.argtypes = [P, P, P, P, i32, i32, i32, i32, i32, P, P, P, P, P, i64, i32, P, i32, P, sz, P]
    L.moe_expert_stage_fp8_workspace_size.restype = sz
    L.moe_expert_stage_fp8_workspace_layout.argtypes = [i32] * 5 + [P]
    L.qmm_last_error.restype = ctypes.c_char_p
    return L


def route(L, **kw):
    a = dict(logits=A, ldt=0, ldl=64, bias=A, live=None, T=4, E=64, k=8, score=1, groups=8, kept=4, top=2, renorm=1,
             scale=1.0, ids=A, w=A, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.moe_route_scored(*a.values())


@pytest.mark.parametrize("kw,st", [
    (dict(T=-1), SHAPE), (dict(T=2 ** 31 - 511), SHAPE), (dict(E=0, groups=1), SHAPE), (dict(E=520, ldl=520), SHAPE), (dict(k=0), SHAPE),
    (dict(k=17), SHAPE), (dict(E=4, k=5, groups=1, kept=1), SHAPE), (dict(groups=0), SHAPE), (dict(groups=7), SHAPE),
    (dict(groups=64, kept=64, top=1), SHAPE), (dict(kept=0), SHAPE), (dict(kept=9), SHAPE), (dict(kept=1, k=9), SHAPE),
    (dict(groups=1, kept=2), SHAPE), (dict(top=0), SHAPE), (dict(top=3), SHAPE), (dict(E=8, ldl=8, k=4, top=2), SHAPE),
    (dict(ldt=2), INVALID), (dict(score=2), INVALID), (dict(score=-1), INVALID), (dict(ldl=63), INVALID), (dict(logits=None), INVALID),
    (dict(ids=None), INVALID), (dict(w=None), INVALID), (dict(logits=ODD), INVALID), (dict(bias=ODD), INVALID),
    (dict(ids=ODD), INVALID), (dict(w=ODD), INVALID), (dict(live=P(258)), INVALID),
])
def test_route(L, kw, st):
    assert route(L, **kw) == st
    assert b"moe_route_scored" in L.qmm_last_error()


def product(L, **kw):
    a = dict(Xq=A, Xs=A, M=4, K=256, N=256, W=A, S=A, bias=A, bdt=0, act=1, R=A, ldr=256, rdt=0, Y=P(512), ydt=1, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.qmm_fp8a8_epilogue_blk128(*a.values())


@pytest.mark.parametrize("kw,st", [
    (dict(K=200), SHAPE), (dict(N=0), SHAPE), (dict(M=-1), SHAPE), (dict(ydt=2), INVALID), (dict(bdt=2), INVALID), (dict(rdt=-1), INVALID),
    (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(ldr=255), INVALID), (dict(bias=ODD), INVALID), (dict(R=ODD), INVALID),
    (dict(Y=None), INVALID), (dict(W=None), INVALID), (dict(Xs=ODD), INVALID),
    (dict(R=P(512), ldr=264, rdt=1), INVALID), (dict(R=P(512)), INVALID), (dict(R=P(512), M=1), INVALID),   # in place: Y's type and pitch
])
def test_product(L, kw, st):
    assert product(L, **kw) == st
    assert b"qmm_fp8a8_epilogue_blk128" in L.qmm_last_error()


def stage(L, **kw):
    a = dict(Xq=A, Xs=A, ids=A, w=A, T=4, D=256, F=128, E=8, k=2, Wgu=A, Sgu=A, Wd=A, Sd=A, R=A, ldr=256, rdt=0, Y=P(512), ydt=1,
             ws=A, ws_bytes=1 << 30, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.moe_expert_stage_fp8(*a.values())


@pytest.mark.parametrize("kw,st", [
    (dict(T=-1), SHAPE), (dict(D=200), SHAPE), (dict(D=0), SHAPE), (dict(F=0), SHAPE), (dict(F=192), SHAPE), (dict(E=0), SHAPE),
    (dict(E=513), SHAPE), (dict(k=0), SHAPE), (dict(k=17), SHAPE), (dict(T=2 ** 22, k=2), SHAPE), (dict(E=512, F=2 ** 21), SHAPE),
    (dict(E=512, D=2 ** 22, ldr=2 ** 22), SHAPE), (dict(E=1, D=2 ** 20 + 16, ldr=2 ** 21), SHAPE),
    (dict(ydt=2), INVALID), (dict(rdt=2), INVALID), (dict(ldr=255), INVALID), (dict(ldr=258), INVALID), (dict(ws_bytes=4096), WORKSPACE),
    (dict(ws=P(128 + 16)), INVALID), (dict(R=P(512)), INVALID), (dict(R=P(512), rdt=1, ldr=260), INVALID),
] + [(dict([(n, v)]), INVALID) for n in ("Xq", "Xs", "ids", "w", "Wgu", "Sgu", "Wd", "Sd", "Y") for v in (None, ODD)] +
    [(dict(ws=None), INVALID), (dict(R=ODD), INVALID)])
def test_stage(L, kw, st):
    assert stage(L, **kw) == st
    assert b"moe_expert_stage_fp8" in L.qmm_last_error()


def test_workspace(L):
    f = L.moe_expert_stage_fp8_workspace_size
    assert f(4, 200, 128, 8, 2) == 0 and f(-1, 256, 128, 8, 2) == 0 and f(4, 256, 128, 8, 17) == 0
    off = (sz * 14)()
    for T, D, F, E, k in [(0, 256, 128, 8, 2), (1, 16, 128, 1, 1), (300, 2048, 768, 128, 8), (2 ** 18, 256, 128, 512, 16)]:
        assert L.moe_expert_stage_fp8_workspace_layout(T, D, F, E, k, ctypes.cast(off, P)) == 0
        offs, pairs = list(off), T * k
        sizes = [E * 4, E * 4 + 4, pairs * 4, pairs * 4, -(-pairs // 2048) * E * 4, None, 4, pairs * D, pairs * -(-D // 128) * 4, pairs * F,
                 pairs * (F // 128) * 4, pairs * D * 4, pairs * -(-D // 64) * 4]
        assert offs == sorted(offs) and all(o % 256 == 0 for o in offs) and offs[-1] == f(T, D, F, E, k)
        for i, n in enumerate(sizes):
            assert n is None or offs[i + 1] - offs[i] >= n
        # room for every tile: full ones and a short one per expert
        assert offs[6] - offs[5] >= 16 * min(pairs, pairs // 16 + E)
    assert L.moe_expert_stage_fp8_workspace_layout(4, 256, 128, 8, 2, None) == INVALID
