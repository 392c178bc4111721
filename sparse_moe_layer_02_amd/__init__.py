"""Python binding of the MI355X MoE-layer library (``include/moe_mi355x.h``).

Argument marshalling only: each function below has the name of the C entry
point it calls, checks dtypes/devices/shapes of the torch tensors it is given,
and passes their device pointers plus the current HIP stream of their device,
with that device made current for the call.  Every step of
the layer runs in the library's HIP kernels; there is no CPU or PyTorch
fallback -- if the shared library is missing, importing a function raises.

PyTorch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# the in-tree build (python -m sparse_moe_layer_02_amd.build)
LIB_PATH = os.path.join(_HERE, "libmoe_mi355x.so")

MOE_F32, MOE_BF16 = 0, 1
_DT = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}
_lock = threading.Lock()
_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_SIGS = {
    "moe_router_logits": ([_P, _I, _P, _I, _I, _I, _P, _P], _I),
    "moe_router_split_weights": ([_P, _I, _I, _P, _P], _I),
    "moe_router_logits_planes": ([_P, _I, _P, _P, _I, _I, _I, _P, _P], _I),
    "moe_route": ([_P, _P, _I, _I, _I, _P, _P, _P, _P, _P], _I),
    "moe_permute": ([_P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P], _I),
    "moe_expert_ffn_workspace_bytes": ([_I, _I, _I, _I], ctypes.c_size_t),
    "moe_expert_ffn": ([_P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _P, ctypes.c_size_t, _P], _I),
    "moe_expert_ffn_gather": ([_P, _I, _I, _P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _P,
                               ctypes.c_size_t, _P], _I),
    "moe_expert_ffn_gather_noalloc": ([_P, _I, _I, _P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _P],
                                      _I),
    "moe_zero_experts": ([_P, _I, _P, _P, _I, _I, _I, _I, _P, _P], _I),
    "moe_combine": ([_P, _I, _P, _P, ctypes.c_float, _P, _I, _I, _I, _P, _P], _I),
    "moe_combine_identity": ([_P, _P, _I, _P, _P, ctypes.c_float, _I, _I, _I, _P, _P], _I),
    "moe_bias_update": ([_P, _I, _I, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                         ctypes.c_float, _P, _P, _P, _P], _I),
    "moe_router_similarity_workspace_bytes": ([_I, _I], ctypes.c_size_t),
    "moe_router_similarity": ([_P, _I, _I, _P, _P, _P, ctypes.c_size_t, _P], _I),
    "moe_forward_workspace_bytes": ([_I, _I, _I, _I, _I, _I, _I], ctypes.c_size_t),
    "moe_forward": ([_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_float, _P, _P,
                     _P, ctypes.c_size_t, _P], _I),
    "moe_status_string": ([_I], ctypes.c_char_p),
    "moe_profile_enable": ([_I], _I),
    "moe_profile_select": ([ctypes.c_char_p], _I),
    "moe_profile_summary": ([ctypes.c_char_p, ctypes.c_size_t], _I),
}


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {lib().moe_status_string(status).decode()} (status {status})")
        self.status = status


def lib():
    """The loaded shared library (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                                   "(python -c 'import __graft_entry__ as g; g.build()')")
            l = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in (*_SIGS.items(), *_block.SIGS.items(),
                                      *_train.SIGS.items()):
                f = getattr(l, name)
                f.argtypes = args
                f.restype = res
            _lib = l
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t: torch.Tensor):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _check(fn: str, status: int):
    if status != 0:
        raise MoEError(fn, status)


def _dev(*ts):
    # by device numbers: comparing torch.device objects costs more than all else here
    d = first = None
    for t in ts:
        if t is None:
            continue
        i = t.get_device()
        if i < 0:
            raise ValueError("tensors must live on the GPU")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        if d is None:
            d, first = i, t
        elif i != d:
            raise ValueError("tensors on different devices")
    return None if first is None else first.device


def _want(t, dtype, name):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")


def _require(ok, what):
    # shape checks the C calls cannot make themselves (they see pointers and
    # the sizes passed in); a failed one would let a kernel read or write
    # past a buffer, so it raises whatever the interpreter's flags
    if not ok:
        raise ValueError(f"argument check failed: {what}")


# --------------------------------------------------------------- the calls --

def moe_router_logits(x, w_router, logits, w_planes=None):
    """logits[T, E] (fp32) = x[T, H] @ w_router[E, H]^T.  w_planes: the
    router weights' bf16 planes from moe_router_split_weights (bitwise the
    same logits, without the split inside the large-batch kernel)."""
    d = _dev(x, w_router, logits, w_planes)
    _want(w_router, torch.float32, "w_router")
    _want(logits, torch.float32, "logits")
    T, H = x.shape
    E = w_router.shape[0]
    _require(w_router.shape == (E, H) and logits.shape == (T, E),
             "w_router.shape == (E, H) and logits.shape == (T, E)")
    if w_planes is None:
        with torch.cuda.device(d):
            _check("moe_router_logits", lib().moe_router_logits(
                _ptr(x), _DT[x.dtype], _ptr(w_router), T, H, E, _ptr(logits), _stream(x)))
        return
    _want(w_planes, torch.bfloat16, "w_planes")
    _require(w_planes.shape == (3, E, H), "w_planes.shape == (3, E, H)")
    with torch.cuda.device(d):
        _check("moe_router_logits_planes", lib().moe_router_logits_planes(
            _ptr(x), _DT[x.dtype], _ptr(w_router), _ptr(w_planes), T, H, E, _ptr(logits),
            _stream(x)))


def moe_router_split_weights(w_router, w_planes):
    """w_planes[3, E, H] (bf16) = the exact split w = hi + mid + lo of the fp32
    router weights (a weight-format preparation; redo it when w_router
    changes)."""
    d = _dev(w_router, w_planes)
    _want(w_router, torch.float32, "w_router")
    _want(w_planes, torch.bfloat16, "w_planes")
    E, H = w_router.shape
    _require(w_planes.shape == (3, E, H), "w_planes.shape == (3, E, H)")
    with torch.cuda.device(d):
        _check("moe_router_split_weights", lib().moe_router_split_weights(
            _ptr(w_router), E, H, _ptr(w_planes), _stream(w_router)))


def prepare_router(w_router, buf):
    """Split the router weights once into buf["w_planes"], which forward()
    then uses.  Redo it whenever w_router changes."""
    E, H = w_router.shape
    planes = buf.get("w_planes")
    if planes is None or planes.shape != (3, E, H) or planes.device != w_router.device:
        planes = torch.empty((3, E, H), dtype=torch.bfloat16, device=w_router.device)
    moe_router_split_weights(w_router, planes)
    buf["w_planes"] = planes
    return planes


def moe_route(logits, bias, K, topk_idx, topk_gate, counts, dev_status=None):
    """Top-K of logits + bias (lower id on ties), softmax gates, histogram."""
    d = _dev(logits, bias, topk_idx, topk_gate, counts, dev_status)
    T, E = logits.shape
    _want(logits, torch.float32, "logits")
    _want(bias, torch.float32, "bias")
    _want(topk_idx, torch.int32, "topk_idx")
    _want(topk_gate, torch.float32, "topk_gate")
    _want(counts, torch.int32, "counts")
    _require(bias.shape == (E,) and topk_idx.shape == (T, K) and topk_gate.shape == (T, K),
             "bias.shape == (E,) and topk_idx.shape == (T, K) and topk_gate.shape == (T, K)")
    _require(counts.shape == (E,), "counts.shape == (E,)")
    with torch.cuda.device(d):
        _check("moe_route", lib().moe_route(
            _ptr(logits), _ptr(bias), T, E, K, _ptr(topk_idx), _ptr(topk_gate), _ptr(counts),
            _ptr(dev_status), _stream(logits)))


def moe_permute(x, topk_idx, counts, n_ffn, offsets, x_perm, row_src, slot_row):
    """Expert-major, token-ascending grouping of the FFN selections; counts
    is moe_route's histogram of topk_idx.  With x_perm None only the indices
    are written (for moe_expert_ffn_gather); x still gives T, H and the
    dtype."""
    d = _dev(x, topk_idx, counts, offsets, x_perm, row_src, slot_row)
    for t, n in ((topk_idx, "topk_idx"), (counts, "counts"), (offsets, "offsets"),
                 (row_src, "row_src"), (slot_row, "slot_row")):
        _want(t, torch.int32, n)
    T, H = x.shape
    K = topk_idx.shape[1]
    _require(topk_idx.shape[0] == T and row_src.numel() >= T * K and slot_row.numel() >= T * K,
             "topk_idx.shape[0] == T and row_src.numel() >= T * K and slot_row.numel() >= T * K")
    _require(counts.numel() >= n_ffn and offsets.numel() >= n_ffn + 1,
             "counts.numel() >= n_ffn and offsets.numel() >= n_ffn + 1")
    if x_perm is not None:
        _require(x_perm.dtype == x.dtype and x_perm.shape[1] == H and x_perm.shape[0] >= T * K,
                 "x_perm.dtype == x.dtype and x_perm.shape[1] == H and x_perm.shape[0] >= T * K")
    with torch.cuda.device(d):
        _check("moe_permute", lib().moe_permute(
            _ptr(x) if x_perm is not None else None, _DT[x.dtype], _ptr(topk_idx), _ptr(counts),
            T, H, K, n_ffn, _ptr(offsets), _ptr(x_perm), _ptr(row_src), _ptr(slot_row),
            _stream(topk_idx)))


def moe_expert_ffn_workspace_bytes(rows_cap, n_ffn, I, dtype):
    return int(lib().moe_expert_ffn_workspace_bytes(rows_cap, n_ffn, I, _DT[dtype]))


def moe_expert_ffn(x_perm, offsets, w13, w2, y_perm, ws):
    """SwiGLU experts on the grouped rows; empty experts skipped."""
    d = _dev(x_perm, offsets, w13, w2, y_perm, ws)
    rows_cap, H = x_perm.shape
    N, I2, H2 = w13.shape
    I = I2 // 2
    _require(H2 == H and w2.shape == (N, H, I) and y_perm.shape == x_perm.shape,
             "H2 == H and w2.shape == (N, H, I) and y_perm.shape == x_perm.shape")
    _require(w13.dtype == w2.dtype == x_perm.dtype == y_perm.dtype,
             "w13.dtype == w2.dtype == x_perm.dtype == y_perm.dtype")
    with torch.cuda.device(d):
        _check("moe_expert_ffn", lib().moe_expert_ffn(
            _ptr(x_perm), _ptr(offsets), rows_cap, N, H, I, _ptr(w13), _ptr(w2), _DT[x_perm.dtype],
            _ptr(y_perm), _ptr(ws), ws.numel() * ws.element_size(), _stream(x_perm)))


def moe_expert_ffn_gather(x, K, row_src, offsets, w13, w2, y_perm, ws):
    """moe_expert_ffn reading row r's activations from x[row_src[r] // K]."""
    d = _dev(x, row_src, offsets, w13, w2, y_perm, ws)
    _want(row_src, torch.int32, "row_src")
    T, H = x.shape
    rows_cap = y_perm.shape[0]
    N, I2, H2 = w13.shape
    I = I2 // 2
    _require(H2 == H and w2.shape == (N, H, I) and y_perm.shape[1] == H,
             "H2 == H and w2.shape == (N, H, I) and y_perm.shape[1] == H")
    _require(row_src.numel() >= rows_cap, "row_src.numel() >= rows_cap")
    _require(w13.dtype == w2.dtype == x.dtype == y_perm.dtype,
             "w13.dtype == w2.dtype == x.dtype == y_perm.dtype")
    with torch.cuda.device(d):
        _check("moe_expert_ffn_gather", lib().moe_expert_ffn_gather(
            _ptr(x), T, K, _ptr(row_src), _ptr(offsets), rows_cap, N, H, I, _ptr(w13), _ptr(w2),
            _DT[x.dtype], _ptr(y_perm), _ptr(ws), ws.numel() * ws.element_size(), _stream(x)))


NOALLOC_SCRATCH_BYTES = 32 << 20   # MOE_EXPERT_FFN_NOALLOC_SCRATCH_BYTES


def moe_expert_ffn_gather_noalloc(x, K, row_src, offsets, w13, w2, y_perm):
    """moe_expert_ffn_gather with its workspace in the library's fixed
    per-GPU scratch (no allocation; for callers that cannot allocate).
    Calls that overlap on one GPU race; order them on one stream."""
    d = _dev(x, row_src, offsets, w13, w2, y_perm)
    _want(row_src, torch.int32, "row_src")
    T, H = x.shape
    rows_cap = y_perm.shape[0]
    N, I2, H2 = w13.shape
    I = I2 // 2
    _require(H2 == H and w2.shape == (N, H, I) and y_perm.shape[1] == H,
             "H2 == H and w2.shape == (N, H, I) and y_perm.shape[1] == H")
    _require(row_src.numel() >= rows_cap, "row_src.numel() >= rows_cap")
    _require(w13.dtype == w2.dtype == x.dtype == y_perm.dtype,
             "w13.dtype == w2.dtype == x.dtype == y_perm.dtype")
    with torch.cuda.device(d):
        _check("moe_expert_ffn_gather_noalloc", lib().moe_expert_ffn_gather_noalloc(
            _ptr(x), T, K, _ptr(row_src), _ptr(offsets), rows_cap, N, H, I, _ptr(w13), _ptr(w2),
            _DT[x.dtype], _ptr(y_perm), _stream(x)))


def moe_zero_experts(x, topk_idx, topk_gate, n_ffn, y_acc):
    """y_acc = (sum of identity-expert gates) * x, fp32."""
    d = _dev(x, topk_idx, topk_gate, y_acc)
    T, H = x.shape
    K = topk_idx.shape[1]
    _want(topk_idx, torch.int32, "topk_idx")
    _want(topk_gate, torch.float32, "topk_gate")
    _want(y_acc, torch.float32, "y_acc")
    _require(topk_idx.shape == (T, K) and topk_gate.shape == (T, K) and y_acc.shape == (T, H),
             "topk_idx.shape == (T, K) and topk_gate.shape == (T, K) and y_acc.shape == (T, H)")
    with torch.cuda.device(d):
        _check("moe_zero_experts", lib().moe_zero_experts(
            _ptr(x), _DT[x.dtype], _ptr(topk_idx), _ptr(topk_gate), T, H, K, n_ffn, _ptr(y_acc),
            _stream(x)))


def _combine_args(y_perm, slot_row, topk_gate, y):
    """Shapes and dtypes combine relies on: the C call reads y_perm rows at
    slot_row, T*K slots and gates, [T, H] rows of its inputs."""
    T, H = y.shape
    K = topk_gate.shape[1]
    _want(slot_row, torch.int32, "slot_row")
    _want(topk_gate, torch.float32, "topk_gate")
    _require(topk_gate.shape == (T, K) and slot_row.numel() >= T * K,
             "topk_gate.shape == (T, K) and slot_row.numel() >= T * K")
    _require(y_perm.dim() == 2 and y_perm.shape[1] == H and y_perm.dtype == y.dtype,
             "y_perm.dim() == 2 and y_perm.shape[1] == H and y_perm.dtype == y.dtype")
    return T, H, K


def moe_combine(y_perm, slot_row, topk_gate, ffn_scale, y_acc, y):
    """y = y_acc + sum of ffn_scale * gate * y_perm rows, in slot order."""
    d = _dev(y_perm, slot_row, topk_gate, y_acc, y)
    T, H, K = _combine_args(y_perm, slot_row, topk_gate, y)
    _want(y_acc, torch.float32, "y_acc")
    _require(y_acc.shape == (T, H), "y_acc.shape == (T, H)")
    with torch.cuda.device(d):
        _check("moe_combine", lib().moe_combine(
            _ptr(y_perm), _DT[y.dtype], _ptr(slot_row), _ptr(topk_gate), float(ffn_scale),
            _ptr(y_acc), T, H, K, _ptr(y), _stream(y)))


def moe_combine_identity(y_perm, x, slot_row, topk_gate, ffn_scale, y):
    """moe_zero_experts + moe_combine in one pass: y = (sum of the identity
    slots' gates) * x + sum of ffn_scale * gate * y_perm rows, in slot order."""
    d = _dev(y_perm, x, slot_row, topk_gate, y)
    T, H, K = _combine_args(y_perm, slot_row, topk_gate, y)
    _require(x.shape == (T, H) and x.dtype == y.dtype, "x.shape == (T, H) and x.dtype == y.dtype")
    with torch.cuda.device(d):
        _check("moe_combine_identity", lib().moe_combine_identity(
            _ptr(y_perm), _ptr(x), _DT[y.dtype], _ptr(slot_row), _ptr(topk_gate), float(ffn_scale),
            T, H, K, _ptr(y), _stream(y)))


def moe_forward_workspace_bytes(T, H, E, n_ffn, I, K, dtype):
    """Bytes of moe_forward's workspace (0 for sizes out of range)."""
    return int(lib().moe_forward_workspace_bytes(T, H, E, n_ffn, I, K, _DT[dtype]))


def moe_forward(x, w_router, bias, w13, w2, K, ffn_scale, y, ws, w_planes=None, dev_status=None):
    """The whole layer in one C call: the five calls of forward()'s default
    path with their intermediate tensors in ws (a uint8 tensor of at least
    moe_forward_workspace_bytes bytes)."""
    d = _dev(x, w_router, bias, w13, w2, y, ws, w_planes, dev_status)
    _want(w_router, torch.float32, "w_router")
    _want(bias, torch.float32, "bias")
    _want(ws, torch.uint8, "ws")
    for t, n in ((w13, "w13"), (w2, "w2"), (y, "y")):
        _want(t, x.dtype, n)
    T, H = x.shape
    E = w_router.shape[0]
    n_ffn, I = w13.shape[0], w2.shape[2]
    _require(w_router.shape == (E, H) and bias.shape == (E,) and y.shape == (T, H),
             "w_router.shape == (E, H) and bias.shape == (E,) and y.shape == (T, H)")
    _require(w13.shape == (n_ffn, 2 * I, H) and w2.shape == (n_ffn, H, I),
             "w13.shape == (n_ffn, 2I, H) and w2.shape == (n_ffn, H, I)")
    if w_planes is not None:
        _want(w_planes, torch.bfloat16, "w_planes")
        _require(w_planes.shape == (3, E, H), "w_planes.shape == (3, E, H)")
    if dev_status is not None:
        _want(dev_status, torch.int32, "dev_status")
        _require(dev_status.numel() >= 1, "dev_status.numel() >= 1")
    with torch.cuda.device(d):
        _check("moe_forward", lib().moe_forward(
            _ptr(x), _DT[x.dtype], _ptr(w_router), _ptr(w_planes), _ptr(bias), _ptr(w13),
            _ptr(w2), T, H, E, n_ffn, I, K, float(ffn_scale), _ptr(y), _ptr(dev_status),
            _ptr(ws), ws.numel(), _stream(x)))
    return y


def moe_bias_update(counts, T, n_ffn, target, kp, ki, kd, bias, integral, prev_err):
    """One PID update of the FFN experts' selection bias from a batch's counts."""
    d = _dev(counts, bias, integral, prev_err)
    _want(counts, torch.int32, "counts")
    for t, n in ((bias, "bias"), (integral, "integral"), (prev_err, "prev_err")):
        _want(t, torch.float32, n)
    _require(counts.numel() >= n_ffn and bias.numel() >= n_ffn,
             "counts.numel() >= n_ffn and bias.numel() >= n_ffn")
    _require(integral.numel() >= n_ffn and prev_err.numel() >= n_ffn,
             "integral.numel() >= n_ffn and prev_err.numel() >= n_ffn")
    with torch.cuda.device(d):
        _check("moe_bias_update", lib().moe_bias_update(
            _ptr(counts), int(T), int(n_ffn), float(target), float(kp), float(ki), float(kd),
            _ptr(bias), _ptr(integral), _ptr(prev_err), _stream(bias)))


def moe_router_similarity_workspace_bytes(E, H):
    return int(lib().moe_router_similarity_workspace_bytes(E, H))


def moe_router_similarity(w_router, sim, mean, ws):
    """Pairwise cosine similarity of the router's per-expert weight rows into
    sim [E, E] and its off-diagonal mean into mean [1] (fp32 tensors)."""
    d = _dev(w_router, sim, mean, ws)
    _want(w_router, torch.float32, "w_router")
    _want(sim, torch.float32, "sim")
    _want(mean, torch.float32, "mean")
    E, H = w_router.shape
    _require(sim.shape == (E, E) and mean.numel() >= 1, "sim.shape == (E, E) and mean.numel() >= 1")
    _require(w_router.is_contiguous() and sim.is_contiguous(),
             "w_router.is_contiguous() and sim.is_contiguous()")
    with torch.cuda.device(d):
        _check("moe_router_similarity", lib().moe_router_similarity(
            _ptr(w_router), E, H, _ptr(sim), _ptr(mean), _ptr(ws), ws.numel() * ws.element_size(),
            _stream(w_router)))


# ------------------------------------------------------------ diagnostics --

def moe_profile_enable(on: bool) -> bool:
    """Start (True) or stop (False) per-kernel event timing; returns the old state."""
    return bool(lib().moe_profile_enable(1 if on else 0))


def moe_profile_select(names=None) -> int:
    """Time only the named kernels (an iterable of names; None: every kernel)."""
    arg = None if names is None else ",".join(names).encode()
    return int(lib().moe_profile_select(arg))


def moe_profile_summary() -> dict:
    """{kernel name: (launches, total ms)} of the current timing session."""
    n = lib().moe_profile_summary(None, 0)
    if n < 0:
        raise RuntimeError("moe_profile_summary: an event could not be read")
    buf = ctypes.create_string_buffer(n + 1)
    lib().moe_profile_summary(buf, n + 1)
    out = {}
    for line in buf.value.decode().splitlines():
        name, cnt, ms = line.split()
        out[name] = (int(cnt), float(ms))
    return out


# ----------------------------------- 4-bit expert weights and block norms --

from . import block as _block  # noqa: E402
from .block import (MXFP4, block_forward, moe_expert_ffn_mxfp4,  # noqa: E402,F401
                    moe_expert_ffn_mxfp4_workspace_bytes, moe_grouped_gemm_mxfp4,
                    moe_grouped_gemm_mxfp4_workspace_bytes, moe_mxfp4_dequantize,
                    moe_mxfp4_quantize, moe_norm, moe_norm_residual, quantize_weights)

# ------------- routing losses, backward passes of the norms, 8-bit activations --

from . import train as _train  # noqa: E402
from .train import (MXFP8, alloc_checkpoint, moe_balance_loss,  # noqa: E402,F401
                    moe_balance_loss_workspace_bytes, moe_layer_norm, moe_layer_norm_backward,
                    moe_mxfp8_dequantize, moe_mxfp8_quantize, moe_norm_backward,
                    moe_norm_backward_workspace_bytes, moe_norm_checkpoint, moe_route_backward,
                    moe_swiglu, moe_swiglu_backward)


# ------------------------------------------------------- buffers + forward --

def alloc_buffers(T, H, E, n_ffn, I, K, dtype, device="cuda", grouped_copy=False,
                  separate_identity=False, mxfp4=False, residual=None):
    """Device buffers for one forward pass (torch allocations; no compute).
    grouped_copy: also allocate x_perm [T*K, H], and forward() then copies the
    grouped rows (moe_permute + moe_expert_ffn); by default the expert GEMM
    gathers them from x itself (moe_expert_ffn_gather) and x_perm is None.
    separate_identity: also allocate y_acc [T, H] fp32, and forward() runs the
    identity experts as their own call (moe_zero_experts, then moe_combine);
    by default combine computes their term itself (moe_combine_identity) and
    y_acc is None.  Both options give bitwise the same y.
    mxfp4: size the expert workspace for MXFP4 expert weights too.
    residual: the dtype of a residual stream around the layer, for
    block_forward(): also allocate x_norm and h_norm [T, H] in dtype and h_out
    [T, H] in residual."""
    rows = T * K
    ws_bytes = max(256, moe_expert_ffn_workspace_bytes(rows, n_ffn, I, dtype))
    if mxfp4:
        ws_bytes = max(ws_bytes, moe_expert_ffn_mxfp4_workspace_bytes(rows, n_ffn, I))
    block = {} if residual is None else dict(
        x_norm=torch.empty((T, H), dtype=dtype, device=device),
        h_norm=torch.empty((T, H), dtype=dtype, device=device),
        h_out=torch.empty((T, H), dtype=residual, device=device))
    f32, i32 = torch.float32, torch.int32
    return dict(
        logits=torch.empty((T, E), dtype=f32, device=device),
        topk_idx=torch.empty((T, K), dtype=i32, device=device),
        topk_gate=torch.empty((T, K), dtype=f32, device=device),
        counts=torch.empty((E,), dtype=i32, device=device),
        status=torch.zeros((1,), dtype=i32, device=device),
        offsets=torch.empty((n_ffn + 1,), dtype=i32, device=device),
        x_perm=torch.empty((rows, H), dtype=dtype, device=device) if grouped_copy else None,
        row_src=torch.empty((rows,), dtype=i32, device=device),
        slot_row=torch.empty((rows,), dtype=i32, device=device),
        y_perm=torch.empty((rows, H), dtype=dtype, device=device),
        ws_ffn=torch.empty((ws_bytes,), dtype=torch.uint8, device=device),
        y_acc=torch.empty((T, H), dtype=f32, device=device) if separate_identity else None,
        y=torch.empty((T, H), dtype=dtype, device=device),
        w_planes=None,   # the router weights' planes, set by prepare_router()
        # six-call path: a second stream (default priority) for the identity
        # experts, and the two events that order it against the current stream
        side_stream=torch.cuda.Stream(device=device) if separate_identity else None,
        ev_routed=torch.cuda.Event() if separate_identity else None,
        ev_identity=torch.cuda.Event() if separate_identity else None,
        **block,
    )


OVERLAP_MIN_TOKENS = 1024


def forward(x, w_router, bias, w13, w2, K, ffn_scale, buf):
    """One layer forward on the current stream, no host synchronisation.
    With the default buffers: router, routing, dispatch (indices only), the
    expert GEMMs gathering their rows from x, and combine with the identity
    experts' term folded in -- five calls.  With separate_identity buffers,
    the six calls of _forward_six.
    w13 and w2 may be MXFP4 (quantize_weights), with bf16 tokens and buffers of
    alloc_buffers(..., mxfp4=True): the experts then run on 4-bit weights
    (moe_expert_ffn_mxfp4)."""
    _same_form(w13, w2)
    if buf["y_acc"] is None:
        return _forward_fused(x, w_router, bias, w13, w2, K, ffn_scale, buf)
    return _forward_six(x, w_router, bias, w13, w2, K, ffn_scale, buf)


def _same_form(w13, w2):
    """Refuse expert weights of which one is MXFP4 and the other is not, before
    the first call of a pass."""
    if isinstance(w13, MXFP4) != isinstance(w2, MXFP4):
        raise TypeError("w13 and w2: both MXFP4 or neither")


def _forward_fused(x, w_router, bias, w13, w2, K, ffn_scale, buf):
    n_ffn = w13.shape[0]
    moe_router_logits(x, w_router, buf["logits"], buf.get("w_planes"))
    moe_route(buf["logits"], bias, K, buf["topk_idx"], buf["topk_gate"], buf["counts"],
              buf["status"])
    _dispatch_and_experts(x, K, n_ffn, w13, w2, buf)
    moe_combine_identity(buf["y_perm"], x, buf["slot_row"], buf["topk_gate"], ffn_scale,
                         buf["y"])
    return buf["y"]


def _forward_six(x, w_router, bias, w13, w2, K, ffn_scale, buf):
    """The six calls of one layer forward, enqueued on the current stream with
    no host synchronisation.  The identity experts depend only on the routing,
    so for batches of OVERLAP_MIN_TOKENS tokens or more they run on a second
    stream beside dispatch and the expert GEMMs (the GEMMs hold every CU's LDS
    but few of its wave slots), and combine waits for them: measured 0.3 %
    faster on the 8192-token layer and 0.6 % on the 16384-token one, while on
    64 tokens the cross-stream wait costs more than it hides.  Results are
    bitwise identical either way."""
    if x.shape[0] < OVERLAP_MIN_TOKENS:
        return forward_serial(x, w_router, bias, w13, w2, K, ffn_scale, buf)
    n_ffn = w13.shape[0]
    main = torch.cuda.current_stream(x.device)
    side = buf["side_stream"]
    moe_router_logits(x, w_router, buf["logits"], buf.get("w_planes"))
    moe_route(buf["logits"], bias, K, buf["topk_idx"], buf["topk_gate"], buf["counts"],
              buf["status"])
    buf["ev_routed"].record(main)
    side.wait_event(buf["ev_routed"])
    with torch.cuda.stream(side):
        moe_zero_experts(x, buf["topk_idx"], buf["topk_gate"], n_ffn, buf["y_acc"])
    buf["ev_identity"].record(side)
    _dispatch_and_experts(x, K, n_ffn, w13, w2, buf)
    main.wait_event(buf["ev_identity"])
    moe_combine(buf["y_perm"], buf["slot_row"], buf["topk_gate"], ffn_scale, buf["y_acc"],
                buf["y"])
    return buf["y"]


def _dispatch_and_experts(x, K, n_ffn, w13, w2, buf):
    """Dispatch and the FFN experts.  Without an x_perm buffer, dispatch
    writes only the indices and the first expert GEMM loads each grouped row
    straight from x (0.9 GB less HBM traffic on the 8192-token layer).  On
    MXFP4 weights the rows are always gathered."""
    if isinstance(w13, MXFP4):
        moe_permute(x, buf["topk_idx"], buf["counts"], n_ffn, buf["offsets"], None,
                    buf["row_src"], buf["slot_row"])
        moe_expert_ffn_mxfp4(x, None, K, buf["row_src"], buf["offsets"], *w13, *w2,
                             buf["y_perm"], buf["ws_ffn"])
    elif buf["x_perm"] is None:
        moe_permute(x, buf["topk_idx"], buf["counts"], n_ffn, buf["offsets"], None,
                    buf["row_src"], buf["slot_row"])
        moe_expert_ffn_gather(x, K, buf["row_src"], buf["offsets"], w13, w2, buf["y_perm"],
                              buf["ws_ffn"])
    else:
        moe_permute(x, buf["topk_idx"], buf["counts"], n_ffn, buf["offsets"], buf["x_perm"],
                    buf["row_src"], buf["slot_row"])
        moe_expert_ffn(buf["x_perm"], buf["offsets"], w13, w2, buf["y_perm"], buf["ws_ffn"])


def forward_serial(x, w_router, bias, w13, w2, K, ffn_scale, buf):
    """forward() with every call on the current stream in layer order (the
    six-call path does not use its second stream)."""
    _same_form(w13, w2)
    if buf["y_acc"] is None:
        return _forward_fused(x, w_router, bias, w13, w2, K, ffn_scale, buf)
    n_ffn = w13.shape[0]
    moe_router_logits(x, w_router, buf["logits"], buf.get("w_planes"))
    moe_route(buf["logits"], bias, K, buf["topk_idx"], buf["topk_gate"], buf["counts"],
              buf["status"])
    _dispatch_and_experts(x, K, n_ffn, w13, w2, buf)
    moe_zero_experts(x, buf["topk_idx"], buf["topk_gate"], n_ffn, buf["y_acc"])
    moe_combine(buf["y_perm"], buf["slot_row"], buf["topk_gate"], ffn_scale, buf["y_acc"],
                buf["y"])
    return buf["y"]
