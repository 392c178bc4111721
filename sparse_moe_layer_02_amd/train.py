"""Binding of the routing losses, the norms' backward passes and the 8-bit
activations (``include/moe_mi355x_train.h``): the same conventions as the
layer's calls, which the package's namespace offers them beside.  Gradients are
calls of their own with buffers of the caller's, like the forward calls."""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _DT, _I, _P, _dev, _require, _want, lib
from .block import _F, _LL, _Z, BLOCK, _call, _int, _norm_weight, _p

SIGS = {
    "moe_balance_loss_workspace_bytes": ([_I, _I, _I], _Z),
    "moe_balance_loss": ([_P, _P, _P, _I, _P, _I, _I, _I, _F, _F, _P, _P, _P, _P, _P, _Z, _P],
                         _I),
    "moe_route_backward": ([_P, _P, _P, _P, _I, _P, _P, _P, _F, _F, _I, _I, _I, _P, _P], _I),
    "moe_mxfp8_quantize": ([_P, _I, _LL, _I, _P, _P, _P, _P], _I),
    "moe_mxfp8_dequantize": ([_P, _P, _I, _LL, _I, _P, _P], _I),
    "moe_norm_checkpoint": ([_P, _I, _P, _F, _I, _I, _P, _I, _P, _P, _P], _I),
    "moe_layer_norm": ([_P, _I, _P, _P, _F, _I, _I, _P, _I, _P, _P, _P], _I),
    "moe_norm_backward_workspace_bytes": ([_I, _I], _Z),
    "moe_norm_backward": ([_P, _I, _P, _I, _P, _P, _F, _I, _I, _P, _P, _I, _P, _P, _Z, _P], _I),
    "moe_layer_norm_backward": ([_P, _I, _P, _I, _P, _P, _F, _I, _I, _P, _P, _I, _P, _P, _P, _Z,
                                 _P], _I),
    "moe_swiglu": ([_P, _I, _LL, _I, _P, _P, _P, _P, _P], _I),
    "moe_swiglu_backward": ([_P, _P, _P, _I, _LL, _I, _P, _P, _P, _P], _I),
}


class MXFP8(NamedTuple):
    """Rows of C values in 8 bits: e4m3 codes [..., C] and scales [..., C / 32],
    both uint8.  What a forward call keeps of its input as its `checkpoint`; the
    backward calls take one in the place of that input."""
    codes: torch.Tensor
    scales: torch.Tensor

    @property
    def shape(self):
        return tuple(self.codes.shape)


def alloc_checkpoint(shape, device="cuda"):
    """An MXFP8 of this shape (its contents undefined)."""
    _require(shape[-1] % BLOCK == 0, "shape[-1] % 32 == 0")
    return MXFP8(torch.empty(tuple(shape), dtype=torch.uint8, device=device),
                 torch.empty((*shape[:-1], shape[-1] // BLOCK), dtype=torch.uint8, device=device))


def _mx8(codes, scales, shape, name):
    """Check that codes and scales are MXFP8 rows of this shape."""
    if codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise TypeError(f"{name}: expected codes and scales of {torch.uint8}")
    cols = shape[-1]
    if cols % BLOCK or codes.shape != shape or scales.shape != (*shape[:-1], cols // BLOCK):
        raise ValueError(f"argument check failed: {name}: codes [..., C] and scales [..., C / 32] "
                         "of its tensor's shape")


def _kept(checkpoint, shape):
    """codes and scales of a checkpoint to be written, or two None."""
    if checkpoint is None:
        return None, None
    codes, scales = checkpoint
    _mx8(codes, scales, shape, "checkpoint")
    return codes, scales


def _rows(n_rows):
    if n_rows is not None:
        _want(n_rows, torch.int32, "n_rows")
        _require(n_rows.numel() >= 1, "n_rows.numel() >= 1")


def _tokens(logits, seq, n_seq):
    """T, E of the logits, with seq checked against them."""
    _want(logits, torch.float32, "logits")
    T, E = logits.shape
    _int(T, E, n_seq)
    if seq is None:
        _require(n_seq == 1, "one sequence without seq")
    else:
        _want(seq, torch.int32, "seq")
        _require(seq.shape == (T,), "seq.shape == (T,)")
    return T, E


# ------------------------------------------------------- the routing losses --

def moe_balance_loss_workspace_bytes(T, E, n_seq):
    return int(lib().moe_balance_loss_workspace_bytes(T, E, n_seq))


def moe_balance_loss(logits, topk_idx, counts, tokens, load, losses, ws, seq=None, group=None,
                     balance_coef=1.0, z_coef=0.0):
    """losses[0] = balance_coef * mean over tokens of sum_e load[seq, e] * p[e],
    losses[1] = z_coef * mean of logsumexp(logits)^2, of a batch's logits [T, E]
    and picks [T, K].  Also written: counts [n_seq, E] and tokens [n_seq + 1]
    (int32; the last of them all tokens) and load [n_seq, E], an expert's picks
    over an even share, averaged over its group.  seq [T]: each token's
    sequence, ids outside [0, n_seq) are padding; group [E]: each expert's
    group, ids outside [0, E) leave it out."""
    d = _dev(logits, topk_idx, counts, tokens, load, losses, ws, seq, group)
    n_seq = counts.shape[0]
    T, E = _tokens(logits, seq, n_seq)
    for t, n in ((topk_idx, "topk_idx"), (counts, "counts"), (tokens, "tokens")):
        _want(t, torch.int32, n)
    for t, n in ((load, "load"), (losses, "losses")):
        _want(t, torch.float32, n)
    _require(topk_idx.dim() == 2 and topk_idx.shape[0] == T, "topk_idx.shape == (T, K)")
    _require(counts.shape == (n_seq, E) and load.shape == (n_seq, E) and
             tokens.shape == (n_seq + 1,) and losses.shape == (2,),
             "counts, load of shape (n_seq, E), tokens (n_seq + 1,), losses (2,)")
    if group is not None:
        _want(group, torch.int32, "group")
        _require(group.shape == (E,), "group.shape == (E,)")
    _call("moe_balance_loss", d, _p(logits), _p(topk_idx), _p(seq), n_seq, _p(group), T, E,
          topk_idx.shape[1], balance_coef, z_coef, _p(counts), _p(tokens), _p(load), _p(losses),
          _p(ws), ws.numel() * ws.element_size())


def moe_route_backward(logits, d_logits, topk_idx=None, d_gate=None, tokens=None, load=None,
                       seq=None, d_losses=None, balance_coef=1.0, z_coef=0.0):
    """d_logits [T, E] = the gradient of moe_route's gates (d_gate [T, K], with
    topk_idx) and of moe_balance_loss's losses (tokens and load as it wrote
    them, d_losses [2]: the losses' own gradients, None: ones), either or both."""
    d = _dev(logits, d_logits, topk_idx, d_gate, tokens, load, seq, d_losses)
    n_seq = 1 if load is None else load.shape[0]
    if load is None:
        seq = None
    T, E = _tokens(logits, seq, n_seq)
    _want(d_logits, torch.float32, "d_logits")
    _require(d_logits.shape == (T, E), "d_logits.shape == logits.shape")
    _require(d_gate is not None or load is not None, "d_gate or load")
    K = 1
    if d_gate is not None:
        _want(d_gate, torch.float32, "d_gate")
        _require(topk_idx is not None, "topk_idx with d_gate")
        _want(topk_idx, torch.int32, "topk_idx")
        K = d_gate.shape[-1]
        _require(d_gate.shape == (T, K) and topk_idx.shape == (T, K),
                 "d_gate and topk_idx of shape (T, K)")
    _require((load is None) == (tokens is None), "load and tokens together")
    if load is not None:
        _want(load, torch.float32, "load")
        _want(tokens, torch.int32, "tokens")
        _require(load.shape == (n_seq, E) and tokens.shape == (n_seq + 1,),
                 "load of shape (n_seq, E), tokens (n_seq + 1,)")
    if d_losses is not None:
        _want(d_losses, torch.float32, "d_losses")
        _require(d_losses.shape == (2,), "d_losses.shape == (2,)")
    _call("moe_route_backward", d, _p(logits), _p(topk_idx), _p(d_gate), _p(seq), n_seq,
          _p(tokens), _p(load), _p(d_losses), balance_coef, z_coef, T, E, K, _p(d_logits))


# ------------------------------------------------- activations in 8 bits --

def moe_mxfp8_quantize(x, codes, scales, n_rows=None):
    """codes, scales = x [..., C] (fp32 or bf16) in MXFP8.  n_rows: a one-element
    int32 tensor, only the first n_rows rows are converted."""
    d = _dev(x, codes, scales, n_rows)
    _mx8(codes, scales, x.shape, "codes")
    cols = x.shape[-1]
    _int(cols)
    _rows(n_rows)
    _call("moe_mxfp8_quantize", d, _p(x), _DT[x.dtype], x.numel() // max(cols, 1), cols,
          _p(n_rows), _p(codes), _p(scales))


def moe_mxfp8_dequantize(codes, scales, y):
    """y [..., C] (fp32 or bf16) = the values that codes and scales stand for."""
    d = _dev(codes, scales, y)
    _mx8(codes, scales, y.shape, "codes")
    cols = y.shape[-1]
    _int(cols)
    _call("moe_mxfp8_dequantize", d, _p(codes), _p(scales), _DT[y.dtype],
          y.numel() // max(cols, 1), cols, _p(y))


def moe_swiglu(gu, hh, n_rows=None, checkpoint=None):
    """hh [rows, I] = silu(gu[:, :I]) * gu[:, I:], and gu [rows, 2I] in 8 bits
    to checkpoint.  n_rows: a one-element int32 tensor, only the first n_rows
    rows."""
    codes, scales = _kept(checkpoint, gu.shape)
    d = _dev(gu, hh, n_rows, codes, scales)
    _want(hh, gu.dtype, "hh")
    rows, I2 = gu.shape
    _require(hh.shape == (rows, I2 // 2) and I2 % 2 == 0, "hh.shape == (rows, I)")
    _int(I2)
    _rows(n_rows)
    _call("moe_swiglu", d, _p(gu), _DT[gu.dtype], rows, I2 // 2, _p(n_rows), _p(hh), _p(codes),
          _p(scales))


def moe_swiglu_backward(d_hh, gu, d_gu, hh=None, n_rows=None):
    """d_gu [rows, 2I] = moe_swiglu's gradient at gu (a tensor of d_hh's dtype,
    or an MXFP8 checkpoint of it); hh [rows, I]: the output, computed again."""
    saved = isinstance(gu, MXFP8)
    codes, scales = gu if saved else (gu, None)
    d = _dev(d_hh, codes, scales, d_gu, hh, n_rows)
    rows, I2 = d_gu.shape
    _int(I2)
    if saved:
        _mx8(codes, scales, d_gu.shape, "gu")
    else:
        _want(gu, d_hh.dtype, "gu")
        _require(gu.shape == d_gu.shape, "gu.shape == d_gu.shape")
    _want(d_gu, d_hh.dtype, "d_gu")
    _require(d_hh.shape == (rows, I2 // 2) and I2 % 2 == 0, "d_hh.shape == (rows, I)")
    if hh is not None:
        _want(hh, d_hh.dtype, "hh")
        _require(hh.shape == d_hh.shape, "hh.shape == d_hh.shape")
    _rows(n_rows)
    _call("moe_swiglu_backward", d, _p(d_hh), _p(codes), _p(scales), _DT[d_hh.dtype], rows,
          I2 // 2, _p(n_rows), _p(d_gu), _p(hh))


# -------------------------------------------------------------- the norms --

def moe_norm_checkpoint(x, weight, y, checkpoint, eps=1e-5):
    """moe_norm (the same bits), and x in 8 bits to checkpoint."""
    _require(checkpoint is not None, "a checkpoint")
    codes, scales = _kept(checkpoint, x.shape)
    d = _dev(x, weight, y, codes, scales)
    T, H = x.shape
    _int(T, H)
    _norm_weight(weight, H, "weight")
    _require(y.shape == (T, H), "y.shape == x.shape")
    _call("moe_norm_checkpoint", d, _p(x), _DT[x.dtype], _p(weight), eps, T, H, _p(y),
          _DT[y.dtype], _p(codes), _p(scales))


def moe_layer_norm(x, weight, bias, y, eps=1e-5, checkpoint=None):
    """y = (x - mean(x)) / sqrt(var(x) + eps) * weight + bias over the last
    dimension (weight None: ones, bias None: zeros), and x in 8 bits to
    checkpoint."""
    codes, scales = _kept(checkpoint, x.shape)
    d = _dev(x, weight, bias, y, codes, scales)
    T, H = x.shape
    _int(T, H)
    _norm_weight(weight, H, "weight")
    _norm_weight(bias, H, "bias")
    _require(y.shape == (T, H), "y.shape == x.shape")
    _call("moe_layer_norm", d, _p(x), _DT[x.dtype], _p(weight), _p(bias), eps, T, H, _p(y),
          _DT[y.dtype], _p(codes), _p(scales))


def moe_norm_backward_workspace_bytes(T, H):
    return int(lib().moe_norm_backward_workspace_bytes(T, H))


def _backward(name, dy, x, weight, dx, sums, ws, eps, d_residual):
    saved = isinstance(x, MXFP8)
    codes, scales = x if saved else (x, None)
    d = _dev(dy, codes, scales, weight, dx, d_residual, ws, *sums.values())
    T, H = dy.shape
    _int(T, H)
    if saved:
        _mx8(codes, scales, dy.shape, "x")
    _require(codes.shape == (T, H) and dx.shape == (T, H), "x and dx of dy's shape")
    _norm_weight(weight, H, "weight")
    for n, t in sums.items():
        _norm_weight(t, H, n)
    if d_residual is not None:
        _want(d_residual, dx.dtype, "d_residual")
        _require(d_residual.shape == (T, H), "d_residual.shape == dy.shape")
    _call(name, d, _p(dy), _DT[dy.dtype], _p(codes), 0 if saved else _DT[x.dtype], _p(scales),
          _p(weight), eps, T, H, _p(d_residual), _p(dx), _DT[dx.dtype],
          *(_p(t) for t in sums.values()), _p(ws),
          0 if ws is None else ws.numel() * ws.element_size())


def moe_norm_backward(dy, x, weight, dx, d_weight=None, ws=None, eps=1e-5, d_residual=None):
    """The backward pass of moe_norm at x (a tensor, or its MXFP8 checkpoint):
    dx [T, H], plus d_residual of dx's dtype, and d_weight [H] (fp32; with a
    workspace ws)."""
    _backward("moe_norm_backward", dy, x, weight, dx, dict(d_weight=d_weight), ws, eps, d_residual)


def moe_layer_norm_backward(dy, x, weight, dx, d_weight=None, d_bias=None, ws=None, eps=1e-5,
                            d_residual=None):
    """The backward pass of moe_layer_norm at x (a tensor, or its MXFP8
    checkpoint): dx [T, H], plus d_residual of dx's dtype, and d_weight, d_bias
    [H] (fp32; with a workspace ws)."""
    _backward("moe_layer_norm_backward", dy, x, weight, dx,
              dict(d_weight=d_weight, d_bias=d_bias), ws, eps, d_residual)
