"""Python binding of the block-quantised prefill GEMM / routed-MoE expert-stage
library (C ABI in include/qmm.h, CUDA kernels for sm_103a in csrc/).

Argument marshalling only: every step runs in the library's kernels, on the
current torch CUDA stream.  There is no CPU path; if the shared library is
missing or the device is not a GB300 the calls raise.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB, build_library  # noqa: F401

QMM_WS_FIELDS = 19
WS_FIELD_NAMES = ("ids", "w", "counts", "offsets", "src", "row", "chunk_counts", "tiles", "tile_count",
                  "tiles256", "tile_count256", "X_perm", "Hq", "Hd", "Hs", "Hd32", "Yslot", "wrow", "total")
QMM_STAGE_SLOTS = 1

_STATUS = {0: "QMM_OK", 1: "QMM_ERR_INVALID_ARG", 2: "QMM_ERR_UNSUPPORTED_SHAPE",
           3: "QMM_ERR_UNSUPPORTED_DEVICE", 4: "QMM_ERR_WORKSPACE", 5: "QMM_ERR_CUDA", 6: "QMM_ERR_TIMEOUT"}


class QmmError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {_STATUS.get(status, status)}: {msg}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded shared library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(f"CUDA library not built ({LIB}); run block_quantized_weight_route_gb300.build")
        L = ctypes.CDLL(LIB)
        P, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.qmm_last_error.restype = ctypes.c_char_p
        L.qmm_last_error.argtypes = []
        L.qmm_check_status.restype = i32
        L.qmm_check_status.argtypes = [P]
        L.qmm_w4a16.restype = i32
        L.qmm_w4a16.argtypes = [P, i32, i32, i32, P, P, ctypes.c_float, P, i32, P]
        L.qmm_fp8_blk128.restype = i32
        L.qmm_fp8_blk128.argtypes = [P, i32, i32, i32, P, P, P, P]
        L.qmm_dense_workspace_size.restype = sz
        L.qmm_dense_workspace_size.argtypes = [i32, i32, i32]
        L.qmm_w4a16_ws.restype = i32
        L.qmm_w4a16_ws.argtypes = [P, i32, i32, i32, P, P, ctypes.c_float, P, i32, P, sz, P]
        L.qmm_fp8_blk128_ws.restype = i32
        L.qmm_fp8_blk128_ws.argtypes = [P, i32, i32, i32, P, P, P, P, sz, P]
        L.moe_route_workspace_size.restype = sz
        L.moe_route_workspace_size.argtypes = [i32, i32, i32]
        L.moe_route_permute.restype = i32
        L.moe_route_permute.argtypes = [P, i32, i32, i32, P, P, P, P, P, P, P, sz, P]
        L.moe_expert_stage_workspace_size.restype = sz
        L.moe_expert_stage_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.moe_expert_stage_workspace_layout.restype = i32
        L.moe_expert_stage_workspace_layout.argtypes = [i32, i32, i32, i32, i32, P]
        L.moe_route_permute_noalloc.restype = i32
        L.moe_route_permute_noalloc.argtypes = [P, i32, i32, i32, P, P, P, P, P, P, P]
        L.qmm_profile_enable.restype = i32
        L.qmm_profile_enable.argtypes = [i32]
        L.qmm_profile_read.restype = i32
        L.qmm_profile_read.argtypes = [P]
        L.qmm_profile_read_call.restype = i32
        L.qmm_profile_read_call.argtypes = [ctypes.c_long, P]
        L.moe_expert_stage_w4_iq4.restype = i32
        L.moe_expert_stage_w4_iq4.argtypes = [P, P, i32, i32, i32, i32, i32, P, P, P, P, P, P, P, sz, P]
        L.moe_expert_stage_w4_iq4_ex.restype = i32
        L.moe_expert_stage_w4_iq4_ex.argtypes = [P, P, i32, i32, i32, i32, i32, P, P, P, P, P, P, P, sz,
                                                 ctypes.c_uint, P]
        L.qmm_dbg_workspace_size.restype = sz
        L.qmm_dbg_workspace_size.argtypes = [i32, i32, i32, i32]
        L.qmm_dbg_gate_up_q8_1.restype = i32
        L.qmm_dbg_gate_up_q8_1.argtypes = [P, P, i32, i32, i32, i32, P, P, P, P, P, P, P, sz, P]
        L.qmm_dbg_down_iq4.restype = i32
        L.qmm_dbg_down_iq4.argtypes = [P, P, P, i32, i32, i32, i32, P, P, P, P, sz, P]
        L.qmm_dbg_combine.restype = i32
        L.qmm_dbg_combine.argtypes = [P, i32, P, P, i32, i32, i32, P, P]
        L.moe_expert_table_size.restype = sz
        L.moe_expert_table_size.argtypes = [i32]
        L.moe_expert_table_build.restype = i32
        L.moe_expert_table_build.argtypes = [i32, i32, i32, P, P, P, P, P, sz, P]
        L.moe_expert_stage_w4_iq4_table.restype = i32
        L.moe_expert_stage_w4_iq4_table.argtypes = [P, P, i32, i32, i32, i32, i32, P, P, P, P, sz, ctypes.c_uint, P]
        L.qmm_q8_0_q8_1_workspace_size.restype = sz
        L.qmm_q8_0_q8_1_workspace_size.argtypes = [i32, i32, i32]
        L.qmm_q8_0_q8_1.restype = i32
        L.qmm_q8_0_q8_1.argtypes = [P, P, i32, i32, i32, P, P, P, P, P, P, P, sz, P]
        f32, i64 = ctypes.c_float, ctypes.c_int64
        norm = [P, i32, i64, P, i64, P, i64, i32, P, i32, f32, i32, i32]
        L.qmm_add_rmsnorm_fp8.restype = i32
        L.qmm_add_rmsnorm_fp8.argtypes = norm + [P, P, P, P]
        L.qmm_add_rmsnorm_q8_1.restype = i32
        L.qmm_add_rmsnorm_q8_1.argtypes = norm + [P, P, P, P, P]
        L.qmm_fp8a8_blk128.restype = i32
        L.qmm_fp8a8_blk128.argtypes = [P, P, i32, i32, i32, P, P, P, i32, P]
        L.qmm_fp8a8_swiglu_blk128.restype = i32
        L.qmm_fp8a8_swiglu_blk128.argtypes = [P, P, i32, i32, i32, P, P, P, P, P]
        L.qmm_dbg_fp8a8_plan.restype = i32
        L.qmm_dbg_fp8a8_plan.argtypes = [i32, i32, i32, i32, P]
        L.qmm_dbg_fp8a8_blk128.restype = i32
        L.qmm_dbg_fp8a8_blk128.argtypes = [P, P, i32, i32, i32, P, P, P, i32, P, P]
        L.qmm_dbg_fp8a8_swiglu_blk128.restype = i32
        L.qmm_dbg_fp8a8_swiglu_blk128.argtypes = [P, P, i32, i32, i32, P, P, P, P, P, P]
        L.qmm_dbg_wait_timeout.restype = i32
        L.qmm_dbg_wait_timeout.argtypes = [ctypes.c_uint, P]
        _lib = L
    return _lib


def _check(fn: str, st: int) -> None:
    if st != 0:
        raise QmmError(fn, st, lib().qmm_last_error().decode())


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_current_device = getattr(torch._C, "_cuda_getDevice", None)   # (None: a torch without CUDA, which has no CUDA tensors)


def _device(t: torch.Tensor, name: str) -> int:
    """The index of t's device, which has to be the current one: the library launches
    there, and takes its error word and its tilings from there."""
    dev = t.get_device() if isinstance(t, torch.Tensor) else -1
    if dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dev != _current_device():
        raise ValueError(f"{name} is on cuda:{dev}, but the current device is cuda:{_current_device()}")
    return dev


def _need(t: torch.Tensor, name: str, dtypes, shape=None) -> torch.Tensor:
    _device(t, name)
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_F16 = (torch.float16, torch.int16, torch.uint16)
_U8 = (torch.uint8, torch.int8)


def _stream(device) -> ctypes.c_void_p:
    s = torch.cuda.current_stream(device)
    if s.device.index != _current_device():
        raise ValueError(f"the call's device is {s.device}, but the current device is cuda:{_current_device()}")
    return ctypes.c_void_p(s.cuda_stream)


def qmm_check_status(device=None) -> None:
    """Synchronise the current stream (of the current device, which `device` may name)
    and raise if a kernel wait timed out."""
    _check("qmm_check_status", lib().qmm_check_status(_stream(device)))


def qmm_dense_workspace_size(M: int, K: int, N: int) -> int:
    return int(lib().qmm_dense_workspace_size(M, K, N))


def _dense_ws(ws, M: int, K: int, N: int, device):
    """The K-split workspace of a dense call: the caller's uint8 tensor, else one
    of qmm_dense_workspace_size bytes from torch's allocator (None if 0)."""
    if ws is None:
        n = qmm_dense_workspace_size(M, K, N)
        if n == 0:
            return None, 0
        ws = torch.empty(n, dtype=torch.uint8, device=device)
    _need(ws, "ws", _U8, (ws.numel(),))
    return ws, ws.numel()


def qmm_w4a16(X, Wc, Ws, scale2: float, out_dtype=torch.float32, Y=None, ws=None):
    """Y[M,N] = scale2 * X . dequant(Wc, Ws)^T  (e2m1 codes, E4M3 per-16 scales).
    ws: device workspace for K splits of the last wave (default: allocated)."""
    M, K = X.shape
    N = Wc.shape[0]
    _need(X, "X", _BF16, (M, K))
    _need(Wc, "Wc", _U8, (N, K // 2))
    _need(Ws, "Ws", _U8, (N, K // 16))
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out_dtype must be float32 or bfloat16")
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=X.device)
    _need(Y, "Y", (out_dtype,), (M, N))
    ws, nws = _dense_ws(ws, M, K, N, X.device)
    st = lib().qmm_w4a16_ws(_ptr(X), M, K, N, _ptr(Wc), _ptr(Ws), float(scale2), _ptr(Y),
                            0 if out_dtype == torch.float32 else 1, _ptr(ws) if ws is not None else None, nws,
                            _stream(X.device))
    _check("qmm_w4a16", st)
    return Y


def qmm_fp8_blk128(X, W, S, Y=None, ws=None):
    """Y[M,N] (bf16) = sum over 128x128 blocks of S[n/128, kb] * X . e4m3(W)^T.
    ws: device workspace for K splits of the last wave (default: allocated)."""
    M, K = X.shape
    N = W.shape[0]
    _need(X, "X", _BF16, (M, K))
    _need(W, "W", _U8 + (torch.float8_e4m3fn,), (N, K))
    _need(S, "S", (torch.float32,), (N // 128, K // 128))
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _need(Y, "Y", _BF16, (M, N))
    ws, nws = _dense_ws(ws, M, K, N, X.device)
    st = lib().qmm_fp8_blk128_ws(_ptr(X), M, K, N, _ptr(W), _ptr(S), _ptr(Y),
                                 _ptr(ws) if ws is not None else None, nws, _stream(X.device))
    _check("qmm_fp8_blk128", st)
    return Y


def qmm_q8_0_q8_1_workspace_size(M: int, K: int, N: int) -> int:
    return int(lib().qmm_q8_0_q8_1_workspace_size(M, K, N))


def qmm_q8_0_q8_1(Xq, Xd, Wq, Wd, ws=None, fp32_out: bool = False) -> dict:
    """Dense Q8_0 x q8_1 projection with its output rounded to q8_1 blocks.
    Xq int8 [M, K], Xd fp16 bits [M, K/32]; Wq int8 [N, K], Wd fp16 bits [N, K/32].
    Returns Yq int8 [M, N], Yd / Ys fp16 bits [M, N/32] and, with fp32_out, the
    fp32 rows Y [M, N] before the rounding."""
    M, K = Xq.shape
    N = Wq.shape[0]
    _need(Xq, "Xq", _U8, (M, K))
    _need(Xd, "Xd", _F16, (M, K // 32))
    _need(Wq, "Wq", _U8, (N, K))
    _need(Wd, "Wd", _F16, (N, K // 32))
    dev = Xq.device
    if ws is None:
        ws = torch.empty(max(qmm_q8_0_q8_1_workspace_size(M, K, N), 256), dtype=torch.uint8, device=dev)
    _need(ws, "ws", _U8)
    Yq = torch.empty((M, N), dtype=torch.int8, device=dev)
    Yd = torch.empty((M, N // 32), dtype=torch.int16, device=dev)
    Ys = torch.empty((M, N // 32), dtype=torch.int16, device=dev)
    Y = torch.empty((M, N), dtype=torch.float32, device=dev) if fp32_out else None
    _check("qmm_q8_0_q8_1", lib().qmm_q8_0_q8_1(_ptr(Xq), _ptr(Xd), M, K, N, _ptr(Wq), _ptr(Wd), _ptr(Yq), _ptr(Yd),
                                                _ptr(Ys), _ptr(Y), _ptr(ws), ws.numel(), _stream(dev)))
    return dict(Yq=Yq, Yd=Yd, Ys=Ys, Y=Y)


_DTYPE = {torch.float32: 0, torch.bfloat16: 1}
_F8 = (torch.float8_e4m3fn, torch.uint8, torch.int8)
_F32 = (torch.float32,)
_Tensor = torch.Tensor


def _ok(t, dtypes, shape, dev: int) -> bool:
    """Whether _need would pass, given the current device.  The calls below take a few
    microseconds on the GPU, so what passes is checked in one expression; _need words the
    error of what does not."""
    return isinstance(t, _Tensor) and t.get_device() == dev and t.dtype in dtypes and t.shape == shape and t.is_contiguous()


# The current stream's handle of a device index, without making a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """t, or a copy of it that starts at a multiple of 16 bytes, as the library asks of
    every buffer.  Row slices of codes do by themselves; a row of scales can be as short as
    4 bytes.  (Callers look at the addresses first, which they need anyway.)"""
    return t if t.data_ptr() & 15 == 0 else t.clone()


def _pitch(t: torch.Tensor, name: str, shape, dev: int) -> int:
    """The row pitch of a matrix in fp32 or bf16 on device dev whose rows are contiguous."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev and t.dtype in _DTYPE and t.shape == shape and t.dim() == 2:
        if t.is_contiguous():
            return shape[1]
        if t.stride(1) == 1:
            return t.stride(0)
    _device(t, name)
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name} must have dtype in {tuple(_DTYPE)}, got {t.dtype}")
    if t.dim() != 2 or t.shape == shape:
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _norm_args(X, G, R, eps, Rout, Y, bf16_out):
    """Checked arguments that the two norms share: (X's device and shape, Rout, Y, the call's first 13 arguments)."""
    dev = _device(X, "X")
    shape = X.shape
    ldx = _pitch(X, "X", shape, dev)
    T, D = shape
    if not _ok(G, _DTYPE, (D,), dev):
        _need(G, "G", _DTYPE, (D,))
    if Y is None:
        if bf16_out:
            Y = torch.empty((T, D), dtype=torch.bfloat16, device=X.device)
    elif not _ok(Y, _BF16, shape, dev):
        _need(Y, "Y", _BF16, shape)
    if R is None:
        if Rout is not None:
            raise ValueError("Rout without R")
        return dev, shape, None, Y, (X.data_ptr(), _DTYPE[X.dtype], ldx, None, 0, None, 0, 0, G.data_ptr(),
                                _DTYPE[G.dtype], eps, T, D)
    ldr = _pitch(R, "R", shape, dev)
    if Rout is None:
        Rout = torch.empty((T, D), dtype=R.dtype, device=X.device)
    ldro = _pitch(Rout, "Rout", shape, dev)
    if Rout.dtype != R.dtype:
        raise TypeError("Rout must have R's dtype")
    return dev, shape, Rout, Y, (X.data_ptr(), _DTYPE[X.dtype], ldx, R.data_ptr(), ldr, Rout.data_ptr(), ldro,
                            _DTYPE[R.dtype], G.data_ptr(), _DTYPE[G.dtype], eps, T, D)


def qmm_add_rmsnorm_fp8(X, G, R=None, eps: float = 1e-6, Rout=None, Q=None, S=None, Y=None,
                        bf16_out: bool = False) -> dict:
    """RMS norm of X [T, D], or of the stored sum Rout = X + R, times G [D], as E4M3
    codes Q [T, D] with one fp32 scale per 128 columns S [T, ceil(D/128)].  X, R and
    G are fp32 or bf16; X, R, Rout, Q and S may be row slices.  Rout=R adds in place.
    bf16_out (or Y given): the normalised rows in bf16 too.  Returns Q, S, R
    (Rout, or None) and Y (or None)."""
    dev, shape, Rout, Y, args = _norm_args(X, G, R, eps, Rout, Y, bf16_out)
    groups = (shape[0], (shape[1] + 127) // 128)
    if Q is None:
        Q = torch.empty(shape, dtype=torch.float8_e4m3fn, device=X.device)
    elif not _ok(Q, _F8, shape, dev):
        _need(Q, "Q", _F8, shape)
    if S is None:
        S = torch.empty(groups, dtype=torch.float32, device=X.device)
    elif not _ok(S, _F32, groups, dev):
        _need(S, "S", _F32, groups)
    s = S.data_ptr()
    scales = _aligned(S) if s & 15 else None
    st = lib().qmm_add_rmsnorm_fp8(*args, Q.data_ptr(), s if scales is None else scales.data_ptr(),
                                   None if Y is None else Y.data_ptr(), _raw_stream(dev))
    if st:
        _check("qmm_add_rmsnorm_fp8", st)
    if scales is not None:
        S.copy_(scales)
    return {"Q": Q, "S": S, "R": Rout, "Y": Y}


def qmm_add_rmsnorm_q8_1(X, G, R=None, eps: float = 1e-6, Rout=None, Y=None, bf16_out: bool = False) -> dict:
    """qmm_add_rmsnorm_fp8 with the rows as q8_1 blocks of 32 (what qmm_q8_0_q8_1
    takes): Yq int8 [T, D], Yd / Ys fp16 bits [T, D/32], R and Y as there."""
    dev, (T, D), Rout, Y, args = _norm_args(X, G, R, eps, Rout, Y, bf16_out)
    Yq = torch.empty((T, D), dtype=torch.int8, device=X.device)
    Yd = torch.empty((T, D // 32), dtype=torch.int16, device=X.device)
    Ys = torch.empty((T, D // 32), dtype=torch.int16, device=X.device)
    st = lib().qmm_add_rmsnorm_q8_1(*args, Yq.data_ptr(), Yd.data_ptr(), Ys.data_ptr(),
                                    None if Y is None else Y.data_ptr(), _raw_stream(dev))
    if st:
        _check("qmm_add_rmsnorm_q8_1", st)
    return {"Yq": Yq, "Yd": Yd, "Ys": Ys, "R": Rout, "Y": Y}


def _need_operands(Xq, Xs, W, S, M: int, K: int, rows: int, blocks: int, name_w: str, name_s: str) -> None:
    """The operands of the two FP8 x FP8 products."""
    kb = (K + 127) // 128
    _need(Xq, "Xq", _F8, (M, K))
    _need(Xs, "Xs", _F32, (M, kb))
    _need(W, name_w, _F8, (rows, K))
    _need(S, name_s, _F32, (blocks, kb))


def qmm_fp8a8_blk128(Xq, Xs, W, S, out_dtype=torch.bfloat16, Y=None):
    """Y[M,N] = sum over 128-K blocks of Xs[m, kb] * S[n/128, kb] * e4m3(Xq) . e4m3(W)^T.
    Xq [M, K] and W [N, K] E4M3, Xs [M, ceil(K/128)] and S [ceil(N/128), ceil(K/128)] fp32.
    Slices of a batch's tokens do: scales that start off a multiple of 16 bytes are copied first."""
    dev = _device(Xq, "Xq")
    M, K = Xq.shape
    N = W.shape[0]
    if out_dtype not in _DTYPE:
        raise TypeError("out_dtype must be float32 or bfloat16")
    kb = (K + 127) // 128
    if not (_ok(Xq, _F8, Xq.shape, dev) and _ok(Xs, _F32, (M, kb), dev) and _ok(W, _F8, (N, K), dev) and
            _ok(S, _F32, ((N + 127) // 128, kb), dev)):
        _need_operands(Xq, Xs, W, S, M, K, N, (N + 127) // 128, "W", "S")
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=Xq.device)
    elif not _ok(Y, (out_dtype,), (M, N), dev):
        _need(Y, "Y", (out_dtype,), (M, N))
    xs, s = Xs.data_ptr(), S.data_ptr()
    if (xs | s) & 15:
        Xs, S = _aligned(Xs), _aligned(S)
        xs, s = Xs.data_ptr(), S.data_ptr()
    st = lib().qmm_fp8a8_blk128(Xq.data_ptr(), xs, M, K, N, W.data_ptr(), s, Y.data_ptr(),
                                _DTYPE[out_dtype], _raw_stream(dev))
    if st:
        _check("qmm_fp8a8_blk128", st)
    return Y


def qmm_fp8a8_swiglu_blk128(Xq, Xs, Wgu, Sgu, Hq=None, Hs=None):
    """H = silu(X . Wg^T) * (X . Wu^T) as E4M3 codes Hq [M, F] with one fp32 scale per
    128 columns Hs [M, F/128].  Xq, Xs as in qmm_fp8a8_blk128, slices too; Wgu [2F, K] E4M3
    (gate rows first), Sgu [2F/128, ceil(K/128)] fp32."""
    dev = _device(Xq, "Xq")
    M, K = Xq.shape
    F = Wgu.shape[0] // 2
    kb = (K + 127) // 128
    if not (_ok(Xq, _F8, Xq.shape, dev) and _ok(Xs, _F32, (M, kb), dev) and _ok(Wgu, _F8, (2 * F, K), dev) and
            _ok(Sgu, _F32, (2 * F // 128, kb), dev)):
        _need_operands(Xq, Xs, Wgu, Sgu, M, K, 2 * F, 2 * F // 128, "Wgu", "Sgu")
    if Hq is None:
        Hq = torch.empty((M, F), dtype=torch.float8_e4m3fn, device=Xq.device)
    elif not _ok(Hq, _F8, (M, F), dev):
        _need(Hq, "Hq", _F8, (M, F))
    if Hs is None:
        Hs = torch.empty((M, F // 128), dtype=torch.float32, device=Xq.device)
    elif not _ok(Hs, _F32, (M, F // 128), dev):
        _need(Hs, "Hs", _F32, (M, F // 128))
    xs, s, hs, scales = Xs.data_ptr(), Sgu.data_ptr(), Hs.data_ptr(), None
    if (xs | s | hs) & 15:
        Xs, Sgu, scales = _aligned(Xs), _aligned(Sgu), _aligned(Hs)
        xs, s, hs = Xs.data_ptr(), Sgu.data_ptr(), scales.data_ptr()
    st = lib().qmm_fp8a8_swiglu_blk128(Xq.data_ptr(), xs, M, K, F, Wgu.data_ptr(), s, Hq.data_ptr(), hs, _raw_stream(dev))
    if st:
        _check("qmm_fp8a8_swiglu_blk128", st)
    if scales is not None and scales is not Hs:
        Hs.copy_(scales)
    return Hq, Hs


def moe_route_workspace_size(T: int, E: int, k: int) -> int:
    return int(lib().moe_route_workspace_size(T, E, k))


def moe_route_permute(logits, k: int, ws=None) -> dict:
    """Top-k routing and stable per-expert grouping; returns ids, w, counts,
    offsets, src, row as CUDA tensors."""
    T, E = logits.shape
    _need(logits, "logits", (torch.float32,), (T, E))
    dev = logits.device
    out = dict(ids=torch.empty((T, k), dtype=torch.int32, device=dev),
               w=torch.empty((T, k), dtype=torch.float32, device=dev),
               counts=torch.empty(E, dtype=torch.int32, device=dev),
               offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
               src=torch.empty(T * k, dtype=torch.int32, device=dev),
               row=torch.empty((T, k), dtype=torch.int32, device=dev))
    if ws is None:
        ws = torch.empty(max(moe_route_workspace_size(T, E, k), 256), dtype=torch.uint8, device=dev)
    _need(ws, "ws", _U8)
    st = lib().moe_route_permute(_ptr(logits), T, E, k, _ptr(out["ids"]), _ptr(out["w"]), _ptr(out["counts"]),
                                 _ptr(out["offsets"]), _ptr(out["src"]), _ptr(out["row"]), _ptr(ws), ws.numel(),
                                 _stream(dev))
    _check("moe_route_permute", st)
    return out


def moe_expert_stage_workspace_size(T: int, D: int, F: int, E: int, k: int) -> int:
    return int(lib().moe_expert_stage_workspace_size(T, D, F, E, k))


def moe_expert_stage_workspace_layout(T: int, D: int, F: int, E: int, k: int) -> dict:
    arr = (ctypes.c_size_t * QMM_WS_FIELDS)()
    _check("moe_expert_stage_workspace_layout",
           lib().moe_expert_stage_workspace_layout(T, D, F, E, k, ctypes.cast(arr, ctypes.c_void_p)))
    return dict(zip(WS_FIELD_NAMES, [int(v) for v in arr]))


def moe_expert_stage_w4_iq4(X, logits, Wgu_c, Wgu_s, gu_scale2, Wd_idx, Wd_s, k: int, ws=None, Y=None,
                            slots: bool = False):
    """The routed expert stage: route, W4 gate/up + SwiGLU + q8_1, IQ4_NL down,
    weighted combine.  Returns Y [T, D] fp32 (and leaves intermediates in ws).
    slots=False: the combine is fused into the down product (fp32 atomic adds,
    summation order not fixed); slots=True: per-row down outputs in the
    workspace's Yslot, then the j-ordered combine (moe_expert_stage_w4_iq4_ex
    with QMM_STAGE_SLOTS)."""
    T, D = X.shape
    E = logits.shape[1]
    F = Wgu_c.shape[1] // 2
    _need(X, "X", _BF16, (T, D))
    _need(logits, "logits", (torch.float32,), (T, E))
    _need(Wgu_c, "Wgu_c", _U8, (E, 2 * F, D // 2))
    _need(Wgu_s, "Wgu_s", _U8, (E, 2 * F, D // 16))
    _need(gu_scale2, "gu_scale2", (torch.float32,), (E,))
    _need(Wd_idx, "Wd_idx", _U8, (E, D, F // 2))
    _need(Wd_s, "Wd_s", _F16, (E, D, F // 32))
    dev = X.device
    if ws is None:
        ws = torch.empty(max(moe_expert_stage_workspace_size(T, D, F, E, k), 256), dtype=torch.uint8, device=dev)
    _need(ws, "ws", _U8)
    if Y is None:
        Y = torch.empty((T, D), dtype=torch.float32, device=dev)
    _need(Y, "Y", (torch.float32,), (T, D))
    if slots:
        st = lib().moe_expert_stage_w4_iq4_ex(_ptr(X), _ptr(logits), T, D, F, E, k, _ptr(Wgu_c), _ptr(Wgu_s),
                                              _ptr(gu_scale2), _ptr(Wd_idx), _ptr(Wd_s), _ptr(Y), _ptr(ws),
                                              ws.numel(), QMM_STAGE_SLOTS, _stream(dev))
    else:
        st = lib().moe_expert_stage_w4_iq4(_ptr(X), _ptr(logits), T, D, F, E, k, _ptr(Wgu_c), _ptr(Wgu_s),
                                           _ptr(gu_scale2), _ptr(Wd_idx), _ptr(Wd_s), _ptr(Y), _ptr(ws), ws.numel(),
                                           _stream(dev))
    _check("moe_expert_stage_w4_iq4", st)
    return Y


def moe_expert_table_build(Wgu_c, Wgu_s, Wd_idx, Wd_s) -> torch.Tensor:
    """A pointer table over per-expert weight tensors (lists of E CUDA tensors:
    [2F, D/2] and [2F, D/16] uint8, [D, F/2] uint8, [D, F/32] fp16 bits).  Returns
    the table (a uint8 device tensor); the weight tensors must outlive its use."""
    E = len(Wgu_c)
    if not (len(Wgu_s) == len(Wd_idx) == len(Wd_s) == E) or E < 1:
        raise ValueError("four lists of E per-expert tensors")
    F2, D2 = Wgu_c[0].shape
    F, D = F2 // 2, D2 * 2
    for e in range(E):
        _need(Wgu_c[e], "Wgu_c[e]", _U8, (2 * F, D // 2))
        _need(Wgu_s[e], "Wgu_s[e]", _U8, (2 * F, D // 16))
        _need(Wd_idx[e], "Wd_idx[e]", _U8, (D, F // 2))
        _need(Wd_s[e], "Wd_s[e]", _F16, (D, F // 32))
    dev = Wgu_c[0].device
    n = int(lib().moe_expert_table_size(E))
    table = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
    arr = lambda ts: (ctypes.c_void_p * E)(*[t.data_ptr() for t in ts])  # noqa: E731
    _check("moe_expert_table_build",
           lib().moe_expert_table_build(D, F, E, arr(Wgu_c), arr(Wgu_s), arr(Wd_idx), arr(Wd_s), _ptr(table),
                                        table.numel(), _stream(dev)))
    return table


def moe_expert_stage_w4_iq4_table(X, logits, gu_scale2, table, F: int, k: int, ws=None, Y=None, slots: bool = False):
    """moe_expert_stage_w4_iq4 over a pointer table of per-expert weights
    (moe_expert_table_build)."""
    T, D = X.shape
    E = logits.shape[1]
    _need(X, "X", _BF16, (T, D))
    _need(logits, "logits", (torch.float32,), (T, E))
    _need(gu_scale2, "gu_scale2", (torch.float32,), (E,))
    _need(table, "table", _U8)
    dev = X.device
    if ws is None:
        ws = torch.empty(max(moe_expert_stage_workspace_size(T, D, F, E, k), 256), dtype=torch.uint8, device=dev)
    _need(ws, "ws", _U8)
    if Y is None:
        Y = torch.empty((T, D), dtype=torch.float32, device=dev)
    _need(Y, "Y", (torch.float32,), (T, D))
    _check("moe_expert_stage_w4_iq4_table",
           lib().moe_expert_stage_w4_iq4_table(_ptr(X), _ptr(logits), T, D, F, E, k, _ptr(gu_scale2), _ptr(table),
                                               _ptr(Y), _ptr(ws), ws.numel(), QMM_STAGE_SLOTS if slots else 0,
                                               _stream(dev)))
    return Y


def qmm_dbg_workspace_size(P: int, D: int, F: int, E: int) -> int:
    return int(lib().qmm_dbg_workspace_size(P, D, F, E))


def _dbg_ws(ws, P, D, F, E, dev):
    if ws is None:
        ws = torch.empty(max(qmm_dbg_workspace_size(P, D, F, E), 256), dtype=torch.uint8, device=dev)
    return _need(ws, "ws", _U8)


def qmm_dbg_gate_up_q8_1(X_perm, offsets, Wgu_c, Wgu_s, gu_scale2, ws=None):
    """Gate/up + SwiGLU + q8_1 of expert-grouped rows X_perm [P, D] (expert e owns
    rows offsets[e] .. offsets[e+1]-1).  Returns (Hq int8 [P, F], Hd, Hs fp16 bits
    as int16 [P, F/32])."""
    P, D = X_perm.shape
    E, F2 = Wgu_c.shape[0], Wgu_c.shape[1]
    F = F2 // 2
    _need(X_perm, "X_perm", _BF16, (P, D))
    _need(offsets, "offsets", (torch.int32,), (E + 1,))
    _need(Wgu_c, "Wgu_c", _U8, (E, F2, D // 2))
    _need(Wgu_s, "Wgu_s", _U8, (E, F2, D // 16))
    _need(gu_scale2, "gu_scale2", (torch.float32,), (E,))
    dev = X_perm.device
    ws = _dbg_ws(ws, P, D, F, E, dev)
    Hq = torch.empty((P, F), dtype=torch.int8, device=dev)
    Hd = torch.empty((P, F // 32), dtype=torch.int16, device=dev)
    Hs = torch.empty((P, F // 32), dtype=torch.int16, device=dev)
    st = lib().qmm_dbg_gate_up_q8_1(_ptr(X_perm), _ptr(offsets), P, D, F, E, _ptr(Wgu_c), _ptr(Wgu_s),
                                    _ptr(gu_scale2), _ptr(Hq), _ptr(Hd), _ptr(Hs), _ptr(ws), ws.numel(), _stream(dev))
    _check("qmm_dbg_gate_up_q8_1", st)
    return Hq, Hd, Hs


def qmm_dbg_down_iq4(Hq, Hd, offsets, Wd_idx, Wd_s, ws=None):
    """Down product of q8_1 rows (Hq int8 [P, F], Hd fp16 bits [P, F/32]) against
    IQ4_NL weights, grouped by offsets.  Returns Yslot fp32 [P, D]."""
    P, F = Hq.shape
    E, D = Wd_idx.shape[0], Wd_idx.shape[1]
    _need(Hq, "Hq", (torch.int8,), (P, F))
    _need(Hd, "Hd", _F16, (P, F // 32))
    _need(offsets, "offsets", (torch.int32,), (E + 1,))
    _need(Wd_idx, "Wd_idx", _U8, (E, D, F // 2))
    _need(Wd_s, "Wd_s", _F16, (E, D, F // 32))
    dev = Hq.device
    ws = _dbg_ws(ws, P, D, F, E, dev)
    Yslot = torch.empty((P, D), dtype=torch.float32, device=dev)
    st = lib().qmm_dbg_down_iq4(_ptr(Hq), _ptr(Hd), _ptr(offsets), P, D, F, E, _ptr(Wd_idx), _ptr(Wd_s),
                                _ptr(Yslot), _ptr(ws), ws.numel(), _stream(dev))
    _check("qmm_dbg_down_iq4", st)
    return Yslot


def qmm_dbg_combine(Yslot, row, w):
    """Y[t] = sum_j w[t, j] * Yslot[row[t, j]] (j ascending).  Returns Y fp32 [T, D]."""
    P, D = Yslot.shape
    T, k = row.shape
    _need(Yslot, "Yslot", (torch.float32,), (P, D))
    _need(row, "row", (torch.int32,), (T, k))
    _need(w, "w", (torch.float32,), (T, k))
    dev = Yslot.device
    Y = torch.empty((T, D), dtype=torch.float32, device=dev)
    st = lib().qmm_dbg_combine(_ptr(Yslot), P, _ptr(row), _ptr(w), T, k, D, _ptr(Y), _stream(dev))
    _check("qmm_dbg_combine", st)
    return Y


QMM_FP8A8_PLAN_FIELDS = 9


def qmm_dbg_fp8a8_plan(M: int, K: int, N: int, gated: bool = False) -> tuple:
    """The tiling that an FP8 x FP8 product of this shape takes: two (pair, bn, tn, cs)
    and the column where the second launch begins (N: there is none)."""
    arr = (ctypes.c_int * QMM_FP8A8_PLAN_FIELDS)()
    _check("qmm_dbg_fp8a8_plan", lib().qmm_dbg_fp8a8_plan(M, K, N, int(gated), ctypes.cast(arr, ctypes.c_void_p)))
    return tuple(arr[:4]), tuple(arr[4:8]), arr[8]


def _plan_array(plan):
    first, second, split = plan
    return (ctypes.c_int * QMM_FP8A8_PLAN_FIELDS)(*first, *second, split)


def qmm_dbg_fp8a8_blk128(Xq, Xs, W, S, plan, out_dtype=torch.bfloat16, Y=None):
    """qmm_fp8a8_blk128 by a given tiling (as qmm_dbg_fp8a8_plan returns it)."""
    M, K = Xq.shape
    N = W.shape[0]
    _need_operands(Xq, Xs, W, S, M, K, N, (N + 127) // 128, "W", "S")
    if out_dtype not in _DTYPE:
        raise TypeError("out_dtype must be float32 or bfloat16")
    if Y is None:
        Y = torch.empty((M, N), dtype=out_dtype, device=Xq.device)
    _need(Y, "Y", (out_dtype,), (M, N))
    _check("qmm_dbg_fp8a8_blk128",
           lib().qmm_dbg_fp8a8_blk128(_ptr(Xq), _ptr(Xs), M, K, N, _ptr(W), _ptr(S), _ptr(Y), _DTYPE[out_dtype],
                                      ctypes.cast(_plan_array(plan), ctypes.c_void_p), _stream(Xq.device)))
    return Y


def qmm_dbg_fp8a8_swiglu_blk128(Xq, Xs, Wgu, Sgu, plan):
    """qmm_fp8a8_swiglu_blk128 by a given tiling."""
    M, K = Xq.shape
    F = Wgu.shape[0] // 2
    _need_operands(Xq, Xs, Wgu, Sgu, M, K, 2 * F, 2 * F // 128, "Wgu", "Sgu")
    Hq = torch.empty((M, F), dtype=torch.float8_e4m3fn, device=Xq.device)
    Hs = torch.empty((M, F // 128), dtype=torch.float32, device=Xq.device)
    _check("qmm_dbg_fp8a8_swiglu_blk128",
           lib().qmm_dbg_fp8a8_swiglu_blk128(_ptr(Xq), _ptr(Xs), M, K, F, _ptr(Wgu), _ptr(Sgu), _ptr(Hq), _ptr(Hs),
                                             ctypes.cast(_plan_array(plan), ctypes.c_void_p), _stream(Xq.device)))
    return Hq, Hs


def qmm_dbg_wait_timeout(timeout_us: int, device=None) -> None:
    """Launch the wait-timeout probe (a bounded wait that nothing satisfies); the
    next qmm_check_status raises QmmError with status QMM_ERR_TIMEOUT."""
    _check("qmm_dbg_wait_timeout", lib().qmm_dbg_wait_timeout(int(timeout_us), _stream(device)))


PROFILE_PHASES = ("route", "gather", "gate_up", "down", "combine")


def qmm_profile_enable(on: bool) -> None:
    _check("qmm_profile_enable", lib().qmm_profile_enable(1 if on else 0))


def qmm_profile_read() -> dict:
    """Phase times (ms) of the last profiled expert-stage call (waits for it)."""
    arr = (ctypes.c_float * len(PROFILE_PHASES))()
    _check("qmm_profile_read", lib().qmm_profile_read(ctypes.cast(arr, ctypes.c_void_p)))
    return dict(zip(PROFILE_PHASES, [float(v) for v in arr]))


def qmm_profile_read_call(i: int) -> dict:
    """Phase times (ms) of the i-th profiled expert-stage call since profiling was
    switched on (one of the last 256; waits for that call only)."""
    arr = (ctypes.c_float * len(PROFILE_PHASES))()
    _check("qmm_profile_read_call", lib().qmm_profile_read_call(int(i), ctypes.cast(arr, ctypes.c_void_p)))
    return dict(zip(PROFILE_PHASES, [float(v) for v in arr]))


def workspace_view(ws: torch.Tensor, layout: dict, name: str, dtype, shape) -> torch.Tensor:
    """A typed view of one region of an expert-stage workspace."""
    n = 1
    for s in shape:
        n *= s
    nbytes = n * torch.empty((), dtype=dtype).element_size()
    off = layout[name]
    return ws[off:off + nbytes].view(dtype).view(*shape)
