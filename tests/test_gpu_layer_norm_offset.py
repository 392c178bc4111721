"""The norm by mean and variance, forward and backward, of rows that are constant or far from zero
beside their spread."""
import numpy as np
import pytest
import torch

import _train as ref
import sparse_moe_layer_02_amd as moe
from _parity import device

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = float(np.float32(1e-5))
LENGTHS = [8, 128, 264, 1000, 2056, 6144, 8200, 8192, 12288, 20008, 32768]
MIXES = [(F32, F32, F32), (BF16, F32, F32), (BF16, F32, BF16), (F32, F32, BF16)]


def _t(a, dtype=F32):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=F32).to(device()).to(dtype)


def _nan(shape, dtype=F32):
    return torch.full(shape, float("nan"), dtype=dtype, device=device())


def _weights(H):
    rng = np.random.default_rng(H)
    return _t(1 + 0.2 * rng.standard_normal(H)), _t(rng.standard_normal(H))


def _backward(dy, x, w, eps, dxt=F32, res=None):
    T, H = dy.shape
    dx, dw, db = _nan((T, H), dxt), _nan((H,)), _nan((H,))
    ws = torch.empty(moe.moe_norm_backward_workspace_bytes(T, H), dtype=torch.uint8, device=device())
    moe.moe_layer_norm_backward(dy, x, w, dx, dw, db, ws, eps, d_residual=res)
    return dx, dw, db


def _centered(x, eps, mean):
    """ref.norm where the deviations' own mean is taken out of them.  The first mean is off by `off`, which
    grows with the row's offset, but alike for the whole row: of the deviations v1 (each within |v| + off, a
    half step off) the sum is off by SUMS steps of their own size, and so is what stays of the mean.  The
    squares' sum s0 less the mean's part of it, at most s0 / 16, is off by SUMS steps of 16/15 and one more;
    the products of g and v, less the mean's part, by SUMS steps of |g| off and as much for g's sum."""
    assert mean
    U, SUMS = ref.U, ref.SUMS
    off = (SUMS * U * np.abs(x)).mean(-1, keepdims=True)
    v = x - x.mean(-1, keepdims=True)
    v1 = np.abs(v) + off
    e = U * v1 + (SUMS + 1) * U * v1.mean(-1, keepdims=True) + U * np.abs(v)
    ms = (v * v).mean(-1, keepdims=True) + eps
    r = 1.0 / np.sqrt(ms)
    rel = 0.5 * ((2 * np.abs(v) * e + e * e).mean(-1, keepdims=True) / ms + (SUMS * 16 / 15 + 1) * U) + 4 * U
    return v * r, r * (e + 2 * SUMS * U * off) + np.abs(v * r) * (rel + U), r, rel


def _constants(n, seed):
    """Values of 24 significant bits between 2^-6 and 2^16."""
    rng = np.random.default_rng(seed)
    return (rng.uniform(1, 2, n) * np.exp2(rng.integers(-6, 16, n)) * rng.choice([-1, 1], n)).astype(np.float32)


@pytest.mark.parametrize("H", LENGTHS)
def test_constant_rows_give_the_bias(H):
    """Bit for bit with eps > 0, however large the constant; NaN with eps == 0."""
    T = 65
    x = _t(np.repeat(_constants(T, H)[:, None], H, 1))
    w, b = _weights(H)
    for yt in (F32, BF16):
        y = _nan((T, H), yt)
        moe.moe_layer_norm(x, w, b, y, EPS)
        assert torch.equal(y, b.to(yt).expand(T, H)), (y.float() - b).abs().max()
        moe.moe_layer_norm(x, w, b, y, 0.0)
        assert torch.isnan(y).all()
    if H % 32 == 0:
        y, kept = _nan((T, H)), moe.alloc_checkpoint((T, H))
        moe.moe_layer_norm(x, w, b, y, EPS, checkpoint=kept)
        assert torch.equal(y, b.expand(T, H))


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("dyt,xt,dxt", MIXES)
def test_backward_of_constant_rows(H, dyt, xt, dxt):
    """Their normed values are zeros, so nothing reaches the weight, and dx is (g - mean(g)) / sqrt(eps)."""
    T = 65
    rng = np.random.default_rng(H)
    x = _t(np.repeat(_constants(T, H)[:, None], H, 1), xt)
    dy, res, w = _t(rng.standard_normal((T, H)), dyt), _t(rng.standard_normal((T, H)), dxt), _weights(H)[0]
    dx, dw, db = _backward(dy, x, w, EPS, dxt, res)
    assert (dw == 0).all(), dw.abs().max()
    zero = np.zeros((T, H))                          # (any constant row has the gradient of this one)
    (want, _, b64), (e, _, e_b) = ref.norm_backward(ref.f64(dy), zero, ref.f64(w), EPS, True, ref.f64(res))
    ref.close(dx, want, ref.rounded(want, e, dxt), "dx")
    ref.close(db, b64, ref.rounded(b64, e_b, F32), "d_bias")
    assert torch.isnan(_backward(dy, x, w, 0.0)[0]).all()


def _offset_rows(T, H, offset, spread):
    rng = np.random.default_rng(H + int(offset))
    return _t(offset * rng.choice([-1, 1], (T, 1)) * rng.uniform(1, 1.9, (T, 1)) + spread * rng.standard_normal((T, H)))


OFFSETS = [(1000.0, 1.0), (1000.0, 0.01), (30000.0, 1.0), (3.0, 1e-3), (0.0, 1.0)]


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("offset,spread", OFFSETS)
@pytest.mark.parametrize("eps", [EPS, 0.0])
def test_rows_with_an_offset(H, offset, spread, eps, monkeypatch):
    """Within a bound that does not grow with the offset, but for its square's part of 2^-46."""
    T = 9
    x, (w, b) = _offset_rows(T, H, offset, spread), _weights(H)
    monkeypatch.setattr(ref, "norm", _centered)
    y = _nan((T, H))
    moe.moe_layer_norm(x, w, b, y, eps)
    want, e = ref.layer_norm(ref.f64(x), ref.f64(w), ref.f64(b), eps)
    ref.close(y, want, ref.rounded(want, e, F32), "y")
    dy = _t(np.random.default_rng(1).standard_normal((T, H)))
    dx, dw, db = _backward(dy, x, w, eps)
    (want, w64, b64), (e, e_w, e_b) = ref.norm_backward(ref.f64(dy), ref.f64(x), ref.f64(w), eps, True)
    ref.close(dx, want, ref.rounded(want, e, F32), "dx")
    ref.close(dw, w64, ref.rounded(w64, e_w, F32), "d_weight")
    ref.close(db, b64, ref.rounded(b64, e_b, F32), "d_bias")


@pytest.mark.parametrize("H", [128, 1000, 6144, 8200, 20008])
@pytest.mark.parametrize("exp", [-90, -45, 0, 50, 75, 100])
def test_rows_that_are_all_but_constant(H, exp, monkeypatch):
    """One value an fp32 step or a few from the others: the row is normed by that value's deviation,
    though the rows' spread is far below what their sum is rounded to."""
    print(f"\n[case] all but constant {H} 2^{exp}", flush=True)
    T = 129
    x = np.repeat((_constants(T, H + 1) * np.exp2(float(exp)).astype(np.float32))[:, None], H, 1)
    for t in range(T):
        for _ in range(1 + t % 4):
            x[t, (7 * t) % H] = np.nextafter(x[t, (7 * t) % H], np.float32(np.inf))
    x64 = x.astype(np.float64)
    rows = np.arange(T)
    v = x64 - x64[rows, (7 * rows + 1) % H][:, None]            # exact
    v = v - v.mean(1, keepdims=True)
    n = v / np.sqrt((v * v).mean(1, keepdims=True))
    y = _nan((T, H))
    moe.moe_layer_norm(_t(x), None, None, y, 0.0)
    # The values less the first mean are exact.  Taking out their mean leaves half a step of it, SUMS U
    # of x's steps, alike for the row: under 8 % of |v|'s mean, which is 1.9 / H of them or more.  The mean
    # of what is left is off by SUMS steps of |v|'s mean, so v in all by U |v| and 31 U mean |v| (1.08), its
    # squares' mean by 64 U (mean |v| is at most their root) and SUMS U, the root by half of it and 4 U:
    # |n| (51 + 2) U + mean |n| 34 U.
    ref.close(y, n, 2 * ref.SUMS * ref.U * (np.abs(n) + np.abs(n).mean(1, keepdims=True)))
    dy = _t(np.random.default_rng(1).standard_normal((T, H)) * np.exp2(min(exp, 50.0)))
    dx, dw, _ = _backward(dy, _t(x), None, 0.0)
    monkeypatch.setattr(ref, "norm", _centered)
    (want, w64, _), (e, e_w, _) = ref.norm_backward(ref.f64(dy), v, None, 0.0, True)    # (a shift changes nothing)
    ref.close(dx, want, ref.rounded(want, e, F32), "dx")
    ref.close(dw, w64, ref.rounded(w64, e_w, F32), "d_weight")


def test_offsets_that_need_a_scale():
    """Constant rows and rows with an offset past the size whose sums or squares fp32 holds."""
    T, H = 6, 1032
    rng = np.random.default_rng(0)
    c = _constants(T, 5)[:, None] * np.exp2(np.array([100.0, 108, 60, -100, -60, -20]))[:, None]
    w, b = _weights(H)
    y = _nan((T, H))
    x = _t(np.repeat(c.astype(np.float32), H, 1))
    moe.moe_layer_norm(x, w, b, y, EPS)
    assert torch.equal(y, b.expand(T, H))
    moe.moe_layer_norm(x, w, b, y, 0.0)
    assert torch.isnan(y).all()
    dy = _t(rng.standard_normal((T, H)))
    dx, dw, _ = _backward(dy, x, w, EPS)
    assert (dw == 0).all()
    want, e = (v[0] for v in ref.norm_backward(ref.f64(dy), np.zeros((T, H)), ref.f64(w), EPS, True))
    ref.close(dx, want, ref.rounded(want, e, F32), "dx")
