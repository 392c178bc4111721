"""Binding of the 4-bit expert weights and the block norms
(``include/moe_mi355x_block.h``): the same conventions as the layer's calls,
which the package's namespace offers them beside."""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _DT, _I, _P, _check, _dev, _require, _want, lib

_F = ctypes.c_float
_Z = ctypes.c_size_t
_LL = ctypes.c_longlong
SIGS = {
    "moe_mxfp4_quantize": ([_P, _I, _LL, _I, _P, _P, _P, _P], _I),
    "moe_mxfp4_dequantize": ([_P, _P, _I, _LL, _I, _P, _P], _I),
    "moe_grouped_gemm_mxfp4_workspace_bytes": ([_I, _I], _Z),
    "moe_grouped_gemm_mxfp4": ([_P, _P, _P, _I, _I, _P, _I, _I, _I, _I, _P, _P, _I, _I, _P, _P,
                                _Z, _P], _I),
    "moe_expert_ffn_mxfp4_workspace_bytes": ([_I, _I, _I], _Z),
    "moe_expert_ffn_mxfp4": ([_P, _P, _I, _I, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _Z,
                              _P], _I),
    "moe_norm": ([_P, _I, _P, _F, _I, _I, _P, _I, _P], _I),
    "moe_norm_residual": ([_P, _I, _P, _F, _P, _I, _F, _P, _I, _P, _P, _P, _I, _I, _P], _I),
}


def _p(t):
    return None if t is None else t.data_ptr()


def _call(name, device, *args):
    """The C call `name` on the device's current stream, with the device current.
    One call of a decode step costs the host as long as its kernel runs, so the
    way there is short: plain integers for pointers, the stream's handle without
    a Stream object around it, no device switch where there is none to make."""
    f = getattr(lib(), name)
    i = device.index
    if i == torch._C._cuda_getDevice():
        status = f(*args, torch._C._cuda_getCurrentRawStream(i))
        if status:
            _check(name, status)
    else:
        with torch.cuda.device(i):
            _check(name, f(*args, torch._C._cuda_getCurrentRawStream(i)))


def _int(*sizes):
    """Sizes that the C calls take as int: ctypes would drop their upper bits."""
    _require(max(sizes) < 1 << 31, "sizes below 2^31")


BLOCK = 32                     # values that share a scale
GATES = {"none": 0, "channel": 1, "token": 2}


class MXFP4(NamedTuple):
    """Rows of C values in microscaled 4-bit floating point: codes
    [..., C / 2] and scales [..., C / 32], both uint8.  forward(),
    forward_serial() and block_forward() take a pair of them in the place of
    bf16 expert weights."""
    codes: torch.Tensor
    scales: torch.Tensor

    @property
    def shape(self):
        return (*self.codes.shape[:-1], 2 * self.codes.shape[-1])


def _mx(codes, scales, name):
    """Shape (rows..., cols) of a pair of codes and scales."""
    _want(codes, torch.uint8, name)
    _want(scales, torch.uint8, name)
    *rows, half = codes.shape
    _require(half % (BLOCK // 2) == 0 and scales.shape == (*rows, half // (BLOCK // 2)),
             "codes [..., C / 2] and scales [..., C / 32]")
    return (*rows, 2 * half)


def moe_mxfp4_quantize(x, codes, scales, n_rows=None):
    """codes, scales = x [..., C] (fp32 or bf16) in MXFP4.  n_rows: a one-element
    int32 tensor, only the first n_rows rows are converted."""
    d = _dev(x, codes, scales, n_rows)
    _require(_mx(codes, scales, "codes") == tuple(x.shape), "codes and scales of x's shape")
    cols = x.shape[-1]
    _int(cols)
    if n_rows is not None:
        _want(n_rows, torch.int32, "n_rows")
        _require(n_rows.numel() >= 1, "n_rows.numel() >= 1")
    _call("moe_mxfp4_quantize", d, _p(x), _DT[x.dtype], x.numel() // max(cols, 1), cols,
          _p(n_rows), _p(codes), _p(scales))


def moe_mxfp4_dequantize(codes, scales, y):
    """y [..., C] (fp32 or bf16) = the values that codes and scales stand for."""
    d = _dev(codes, scales, y)
    _require(_mx(codes, scales, "codes") == tuple(y.shape), "codes and scales of y's shape")
    cols = y.shape[-1]
    _int(cols)
    _call("moe_mxfp4_dequantize", d, _p(codes), _p(scales), _DT[y.dtype],
          y.numel() // max(cols, 1), cols, _p(y))


def quantize_weights(w):
    """The MXFP4 form of weights w [..., C] (fp32 or bf16, on the GPU), in new
    tensors: a preparation to be done once."""
    _require(w.shape[-1] % BLOCK == 0, "w.shape[-1] % 32 == 0")
    q = MXFP4(torch.empty((*w.shape[:-1], w.shape[-1] // 2), dtype=torch.uint8, device=w.device),
              torch.empty((*w.shape[:-1], w.shape[-1] // BLOCK), dtype=torch.uint8,
                          device=w.device))
    moe_mxfp4_quantize(w, q.codes, q.scales)
    return q


def moe_grouped_gemm_mxfp4_workspace_bytes(rows_cap, n_experts):
    return int(lib().moe_grouped_gemm_mxfp4_workspace_bytes(rows_cap, n_experts))


def moe_grouped_gemm_mxfp4(a, a_scales, offsets, w, w_scales, out, ws, row_src=None, K=1,
                           swiglu=False):
    """out[r] = a[r] @ w[e]^T for the rows r of every expert e (of offsets), on
    MXFP4 weights w [E, N, D / 2] and w_scales [E, N, D / 32].  a: bf16 [., D]
    with a_scales None, or MXFP4 codes and scales.  row_src: row r is row
    row_src[r] // K of a.  swiglu: out = silu(first half of the columns) *
    second half."""
    d = _dev(a, a_scales, offsets, w, w_scales, out, ws, row_src)
    _want(offsets, torch.int32, "offsets")
    E, N, D = _mx(w, w_scales, "w")
    rows_cap, width = out.shape
    _int(a.shape[0], K, rows_cap, E, D, N)
    if a_scales is None:
        _want(a, torch.bfloat16, "a")
        _require(a.dim() == 2 and a.shape[1] == D, "a.shape[1] == D")
    else:
        _require(_mx(a, a_scales, "a")[1:] == (D,), "a of D values a row")
    _require(offsets.numel() >= E + 1, "offsets.numel() >= E + 1")
    _require(width * (2 if swiglu else 1) == N, "out of N columns (swiglu: N / 2)")
    if row_src is None:
        _require(a.shape[0] >= rows_cap, "a.shape[0] >= out.shape[0]")
    else:
        _want(row_src, torch.int32, "row_src")
        _require(row_src.numel() >= rows_cap, "row_src.numel() >= out.shape[0]")
    _call("moe_grouped_gemm_mxfp4", d, _p(a), _p(a_scales), _p(row_src), a.shape[0], K,
          _p(offsets), rows_cap, E, D, N, _p(w), _p(w_scales), 1 if swiglu else 0,
          _DT[out.dtype], _p(out), _p(ws), ws.numel() * ws.element_size())


def moe_expert_ffn_mxfp4_workspace_bytes(rows_cap, n_ffn, I):
    return int(lib().moe_expert_ffn_mxfp4_workspace_bytes(rows_cap, n_ffn, I))


def moe_expert_ffn_mxfp4(x, x_scales, K, row_src, offsets, w13, w13_scales, w2, w2_scales, y_perm,
                         ws):
    """moe_expert_ffn_gather on MXFP4 weights.  x: bf16 [T, H] with x_scales
    None (the rows between the two products are bf16), or MXFP4 codes and
    scales (those rows are MXFP4 too)."""
    d = _dev(x, x_scales, row_src, offsets, w13, w13_scales, w2, w2_scales, y_perm, ws)
    _want(row_src, torch.int32, "row_src")
    _want(offsets, torch.int32, "offsets")
    _want(y_perm, torch.bfloat16, "y_perm")
    N, I2, H = _mx(w13, w13_scales, "w13")
    I = I2 // 2
    _require(I2 == 2 * I and _mx(w2, w2_scales, "w2") == (N, H, I), "w2 of shape (N, H, I)")
    if x_scales is None:
        _want(x, torch.bfloat16, "x")
        _require(x.dim() == 2 and x.shape[1] == H, "x.shape[1] == H")
    else:
        _require(_mx(x, x_scales, "x")[1:] == (H,), "x of H values a row")
    rows_cap = y_perm.shape[0]
    _int(x.shape[0], K, rows_cap, N, H, I2)
    _require(y_perm.shape == (rows_cap, H) and row_src.numel() >= rows_cap,
             "y_perm of H columns and row_src.numel() >= rows_cap")
    _require(offsets.numel() >= N + 1, "offsets.numel() >= n_ffn + 1")
    _call("moe_expert_ffn_mxfp4", d, _p(x), _p(x_scales), x.shape[0], K, _p(row_src),
          _p(offsets), rows_cap, N, H, I, _p(w13), _p(w13_scales), _p(w2), _p(w2_scales),
          _p(y_perm), _p(ws), ws.numel() * ws.element_size())


def _norm_weight(w, H, name):
    if w is not None:
        _want(w, torch.float32, name)
        _require(w.shape == (H,), name)


def moe_norm(x, weight, y, eps=1e-5):
    """y = x / sqrt(mean(x^2) + eps) * weight over the last dimension (weight
    None: ones)."""
    d = _dev(x, weight, y)
    T, H = x.shape
    _int(T, H)
    _norm_weight(weight, H, "weight")
    _require(y.shape == (T, H), "y.shape == x.shape")
    _call("moe_norm", d, _p(x), _DT[x.dtype], _p(weight), eps, T, H, _p(y), _DT[y.dtype])


def moe_norm_residual(y, residual, out, scale=1.0, w_post=None, gate=None, gate_kind="none",
                      w_next=None, next_out=None, eps=1e-5):
    """out = residual + scale * gate * norm(y; w_post) (w_post None: y itself),
    and, with next_out, next_out = norm(the fp32 sums; w_next).  gate_kind:
    "none", "channel" (gate [H]) or "token" (gate [T])."""
    d = _dev(y, residual, out, w_post, gate, w_next, next_out)
    T, H = y.shape
    _int(T, H)
    _norm_weight(w_post, H, "w_post")
    _norm_weight(w_next, H, "w_next")
    _require(gate_kind in GATES and (gate is None) == (gate_kind == "none"),
             'gate_kind "none" without a gate, "channel" or "token" with one')
    if gate is not None:
        _want(gate, torch.float32, "gate")
        _require(gate.shape == ((H,) if gate_kind == "channel" else (T,)),
                 "gate.shape == (H,) (channel) or (T,) (token)")
    _require(residual.shape == (T, H) and out.shape == (T, H) and out.dtype == residual.dtype,
             "residual and out of y's shape and one dtype")
    _require(w_next is None or next_out is not None, "w_next with next_out")
    if next_out is not None:
        _want(next_out, y.dtype, "next_out")
        _require(next_out.shape == (T, H), "next_out.shape == y.shape")
    _call("moe_norm_residual", d, _p(y), _DT[y.dtype], _p(w_post), eps, _p(gate),
          GATES[gate_kind], scale, _p(residual), _DT[residual.dtype], _p(out), _p(w_next),
          _p(next_out), T, H)


def block_forward(h, w_norm, w_router, bias, w13, w2, K, ffn_scale, buf, scale=1.0, w_post=None,
                  gate=None, gate_kind="none", w_next=None, eps=1e-5, x_norm=None):
    """The MoE layer as a block of a residual stream h [T, H] (fp32 or bf16),
    on the current stream: norm, layer (forward(), with bf16 or MXFP4 expert
    weights), norm of its output, gate, residual scale and sum, and the next
    block's norm.  buf: alloc_buffers(..., residual=h.dtype).  Returns
    buf["h_out"], and with w_next also buf["h_norm"]: the layer's input of a
    block that follows, which takes it as its x_norm.
    x_norm: the norm of h, where there is one already ([T, H] in the layer's
    dtype, its weight applied); the norm in front is then left out, and w_norm
    has to be None.  In a chain of blocks h and x_norm may be the last block's
    results in the same buf: they are read before this block's are written."""
    from . import _same_form, forward
    _same_form(w13, w2)
    if x_norm is None:
        x_norm = buf["x_norm"]
        moe_norm(h, w_norm, x_norm, eps)
    else:
        _require(w_norm is None, "w_norm None with x_norm")
        _require(x_norm.shape == h.shape and x_norm.dtype == buf["y"].dtype,
                 "x_norm of h's shape in the layer's dtype")
    y = forward(x_norm, w_router, bias, w13, w2, K, ffn_scale, buf)
    n = buf["h_norm"] if w_next is not None else None
    moe_norm_residual(y, h, buf["h_out"], scale, w_post, gate, gate_kind, w_next, n, eps)
    return buf["h_out"] if n is None else (buf["h_out"], n)
