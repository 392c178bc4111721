"""The norms before and after a block against their 64-bit form."""
import numpy as np
import pytest
import torch

import sparse_moe_layer_02_amd as moe
from _mxfp4 import EPS_BF16, EPS_F32
from _parity import device

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


def _t(a, dtype=F32):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=F32).to(device()).to(dtype)


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _norm(x, w, eps, ex=0.0):
    """(norm, bound): ex is how far x may be from the values in fp32."""
    H = x.shape[-1]
    ms = (x * x).mean(-1, keepdims=True) + eps
    r = 1.0 / np.sqrt(ms)
    # the sum of squares: at most H additions and H products; then the root and two products
    rel = (H / 2 + 8) * EPS_F32 + (np.abs(x) * ex).mean(-1, keepdims=True) / ms
    n = x * r * (1.0 if w is None else w)
    return n, np.abs(n) * rel + ex * r * (1.0 if w is None else np.abs(w))


def _round(v, e, dtype):
    return e + (EPS_BF16 if dtype is BF16 else EPS_F32) * (np.abs(v) + e) + 1e-37


def _close(got, want, bound):
    d = np.abs(_f64(got) - want) - bound
    assert np.isfinite(_f64(got)).all() and d.max() <= 0, d.max()


SHAPES = [(1, 8), (1, 6144), (3, 504), (5, 512), (7, 520), (9, 1000), (2, 8192), (3, 8200),
          (2, 16384), (2, 20008), (1, 32768), (1025, 64), (257, 2048)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("xt,yt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_norm(T, H, xt, yt):
    print(f"\n[case] norm {T}x{H} {xt}->{yt}", flush=True)
    rng = np.random.default_rng(H)
    x = _t(rng.standard_normal((T, H)) * np.exp2(rng.integers(-6, 6, (T, 1))), xt)
    for w in (None, _t(1 + 0.2 * rng.standard_normal(H))):
        y = torch.full((T, H), float("nan"), dtype=yt, device=x.device)
        moe.moe_norm(x, w, y, EPS)
        want, e = _norm(_f64(x), _f64(w), EPS)
        _close(y, want, _round(want, e, yt))


def _residual_case(T, H, yt, rt, gate, post, nxt, seed=0, scale=0.375):
    rng = np.random.default_rng(seed)
    y = _t(rng.standard_normal((T, H)) * np.exp2(rng.integers(-6, 6, (T, 1))), yt)
    res = _t(3 * rng.standard_normal((T, H)), rt)
    wp = _t(1 + 0.2 * rng.standard_normal(H)) if post else None
    wn = _t(1 + 0.2 * rng.standard_normal(H)) if nxt == "weight" else None
    g = {"none": None, "channel": _t(rng.standard_normal(H)),
         "token": _t(rng.standard_normal(T))}[gate]
    n = torch.full((T, H), float("nan"), dtype=yt, device=y.device) if nxt else None
    out = torch.full((T, H), float("nan"), dtype=rt, device=y.device)
    kw = dict(scale=scale, w_post=wp, gate=g, gate_kind=gate, w_next=wn, eps=EPS)
    return y, res, out, n, kw


def _residual_want(y, res, kw, nxt):
    z = _f64(y)
    ez = np.zeros_like(z)
    if kw["w_post"] is not None:
        z, ez = _norm(z, _f64(kw["w_post"]), EPS)
    g = _f64(kw["gate"])
    g = 1.0 if g is None else g[:, None] if kw["gate_kind"] == "token" else g
    z, ez = kw["scale"] * g * z, np.abs(kw["scale"] * g) * ez
    s = _f64(res) + z
    es = ez + 4 * EPS_F32 * np.abs(z) + EPS_F32 * np.abs(s)
    n = _norm(s, _f64(kw["w_next"]), EPS, es) if nxt else None
    return s, es, n


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("yt,rt", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("gate,post,nxt", [("token", True, "weight"), ("channel", True, "ones"),
                                           ("none", False, "weight"), ("channel", False, None)])
def test_norm_residual(T, H, yt, rt, gate, post, nxt):
    print(f"\n[case] norm_residual {T}x{H} y {yt} residual {rt} {gate} {post} {nxt}", flush=True)
    y, res, out, n, kw = _residual_case(T, H, yt, rt, gate, post, nxt, seed=H + T)
    moe.moe_norm_residual(y, res, out, next_out=n, **kw)
    s, es, want = _residual_want(y, res, kw, nxt)
    _close(out, s, _round(s, es, rt))
    if nxt:
        _close(n, want[0], _round(want[0], want[1], yt))


def test_norm_residual_in_place():
    """res_out may be the residual and next the block's output; the same bits as in new tensors."""
    y, res, out, n, kw = _residual_case(40, 768, BF16, F32, "token", True, "weight")
    moe.moe_norm_residual(y, res, out, next_out=n, **kw)
    y2, r2 = y.clone(), res.clone()
    moe.moe_norm_residual(y2, r2, r2, next_out=y2, **kw)
    assert torch.equal(r2, out) and torch.equal(y2, n)
    x = y.clone()
    moe.moe_norm(x, kw["w_post"], x, EPS)
    z = torch.empty_like(y)
    moe.moe_norm(y, kw["w_post"], z, EPS)
    assert torch.equal(x, z)


def test_rows_of_zeros_and_rows_that_are_not_finite():
    """A row of zeros gives zeros (eps > 0), and a NaN or infinity stays in its own row."""
    y, res, out, n, kw = _residual_case(6, 1032, BF16, BF16, "none", True, "weight", scale=1.0)
    clean = (out.clone(), n.clone())
    moe.moe_norm_residual(y, res, clean[0], next_out=clean[1], **kw)
    y[1], res[1] = 0, 0
    y[3, 5] = float("nan")
    y[4, 1031] = float("inf")
    moe.moe_norm_residual(y, res, out, next_out=n, **kw)
    assert (out[1] == 0).all() and (n[1] == 0).all()
    assert torch.isnan(n[3]).all() and torch.isnan(out[4, 1031])
    for t in (0, 2, 5):
        assert torch.equal(out[t], clean[0][t]) and torch.equal(n[t], clean[1][t])
