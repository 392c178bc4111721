"""Activations in 8 bits and the SwiGLU that keeps its input in them, against their 64-bit forms."""
import numpy as np
import pytest
import torch

import _train as ref
import sparse_moe_layer_02_amd as moe
from _parity import device

pytestmark = pytest.mark.gpu
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8


def _t(a, dtype=F32):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=F32).to(device()).to(dtype)


def _kept(shape, fill=0xA5):
    k = moe.alloc_checkpoint(shape)
    k.codes.fill_(fill), k.scales.fill_(fill)
    return k


def _check_quantize(x):
    kept = _kept(x.shape)
    moe.moe_mxfp8_quantize(x, *kept)
    codes, scales = ref.mx8_quantize(ref.f64(x))
    assert np.array_equal(kept.scales.cpu().numpy(), scales)
    got = kept.codes.cpu().numpy()
    assert np.array_equal(got, codes), np.argwhere(got != codes)[:5]
    return kept, codes, scales


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 96), (3, 64), (7, 2048), (1000, 160), (129, 6144)])
def test_there_and_back(rows, cols, dtype):
    print(f"\n[case] mxfp8 {rows}x{cols} {dtype}", flush=True)
    rng = np.random.default_rng(cols)
    x = _t(rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-30, 30, (rows, 1))) *
           np.exp2(rng.integers(-8, 1, (1, cols))), dtype)
    kept, codes, scales = _check_quantize(x)
    want = ref.mx8_values(codes, scales)
    for t in (F32, BF16):                            # exact in both
        y = torch.full(x.shape, float("nan"), dtype=t, device=x.device)
        moe.moe_mxfp8_dequantize(*kept, y)
        assert np.array_equal(ref.f64(y), want)


def test_every_bf16_value_beside_each_scale_of_a_block():
    """All finite bf16 values, in blocks with a largest value of every exponent (and both sides of 1.75
    times it): the code of each is that of the definition, ties and subnormals among them."""
    v = np.arange(65536, dtype=np.uint16).view(np.int16)
    v = torch.from_numpy(v).view(BF16).double().numpy()
    v = v[np.isfinite(v)]
    v = np.sort(np.abs(v))
    v = np.concatenate([v, -v])
    n = len(v) // 31 * 31
    for top in (1.75, 1.7578125, 1.0, 1.9921875):
        x = np.zeros((n // 31, 32))
        x[:, 1:] = v[:n].reshape(-1, 31)
        peak = np.exp2(np.floor(np.log2(np.maximum(np.abs(x).max(1), 2.0 ** -133)))) * top
        x[:, 0] = np.minimum(np.maximum(peak, np.abs(x).max(1)), 3.38e38)
        _check_quantize(_t(x, BF16))
        far = x.copy()                               # values far below the largest of their block
        far[:, 0] = np.minimum(far[:, 0] * 2.0 ** 12, 3.38e38)
        _check_quantize(_t(far, BF16))


def test_fp32_values_next_to_the_borders():
    """Ties between codes and between scales, one fp32 step to either side."""
    mid = (ref.E4M3[:-1] + ref.E4M3[1:]) / 2
    at = np.concatenate([mid, ref.E4M3[1:]])
    for e in (-100, -3, 0, 60):
        b = (at * 2.0 ** e).astype(np.float32)
        x = np.concatenate([b, np.nextafter(b, np.float32(0)), np.nextafter(b, np.float32(np.inf))])
        x = np.concatenate([x, -x])
        x = np.concatenate([x, np.zeros(-len(x) % 31, np.float32)]).reshape(-1, 31)
        x = np.concatenate([x, np.full((len(x), 1), 448.0 * 2.0 ** e, np.float32)], 1)
        x = np.clip(x, -448.0 * 2.0 ** e, 448.0 * 2.0 ** e)
        _check_quantize(_t(x))
        tops = np.array([447.99997, 448.0, 448.00003, 463.9, 464.0, 480.0, 512.0], np.float32) * np.float32(2.0 ** e)
        _check_quantize(_t(tops[:, None] * np.linspace(-1, 1, 32, dtype=np.float32)))


def test_blocks_that_are_not_finite_zero_or_tiny():
    x = np.ones((1, 32 * 6))
    x[0, 5], x[0, 40], x[0, 70] = np.nan, np.inf, -np.inf
    x[0, 96:128] = 0.0
    x[0, 128:160] = 2.0 ** -149
    x[0, 160:] = np.linspace(-1, 1, 32) * 2.0 ** -122
    kept, codes, scales = _check_quantize(_t(x))
    assert scales[0].tolist() == [255, 255, 255, 0, 0, scales[0, 5]]
    y = torch.empty((1, 192), device=device())
    moe.moe_mxfp8_dequantize(*kept, y)
    assert torch.isnan(y[0, :96]).all() and np.array_equal(ref.f64(y)[0, 96:], ref.mx8_values(codes, scales)[0, 96:])


def test_every_code_at_every_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, 1)
    want = ref.mx8_values(codes, scales)
    c, s = torch.from_numpy(codes).to(device()), torch.from_numpy(scales).to(device())
    y = torch.empty((256, 256), device=device())
    moe.moe_mxfp8_dequantize(c, s, y)
    with np.errstate(over="ignore"):
        f = want.astype(np.float32)                  # past 2^128: infinities
    assert np.array_equal(ref.f64(y), f.astype(np.float64), equal_nan=True)
    z = torch.empty((256, 256), dtype=BF16, device=device())
    moe.moe_mxfp8_dequantize(c, s, z)
    assert np.array_equal(ref.f64(z), ref.f64(torch.from_numpy(f).to(BF16)), equal_nan=True)


@pytest.mark.parametrize("n", [-3, 0, 1, 9, 16, 17, 1 << 30])
def test_rows_behind_the_last(n):
    """Only the first n rows are touched, in the conversion, the SwiGLU and its backward pass."""
    rows, I = 16, 64
    rng = np.random.default_rng(0)
    n_rows = torch.tensor([n], dtype=torch.int32, device=device())
    k = min(max(n, 0), rows)
    gu, d = _t(rng.standard_normal((rows, 2 * I)), BF16), _t(rng.standard_normal((rows, I)), BF16)
    whole, kept, kept2 = (_kept((rows, 2 * I)) for _ in range(3))
    moe.moe_mxfp8_quantize(gu, *whole)
    moe.moe_mxfp8_quantize(gu, *kept, n_rows=n_rows)
    hh, d_gu, h2 = (torch.full((rows, c), 7.0, dtype=BF16, device=device()) for c in (I, 2 * I, I))
    moe.moe_swiglu(gu, hh, n_rows, kept2)
    moe.moe_swiglu_backward(d, whole, d_gu, h2, n_rows)
    for a in (kept, kept2):
        assert torch.equal(a.codes[:k], whole.codes[:k]) and (a.codes[k:] == 0xA5).all()
        assert torch.equal(a.scales[:k], whole.scales[:k]) and (a.scales[k:] == 0xA5).all()
    for t in (hh, d_gu, h2):
        assert (t[k:] == 7).all() and (t[:k] != 7).any(1).all()


@pytest.mark.parametrize("rows,I", [(1, 8), (3, 40), (5, 24), (1, 2048), (700, 96), (33, 1000)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_swiglu(rows, I, dtype):
    print(f"\n[case] swiglu {rows}x{I} {dtype}", flush=True)
    rng = np.random.default_rng(I)
    gu = _t(rng.standard_normal((rows, 2 * I)) * 4, dtype)
    d = _t(rng.standard_normal((rows, I)), dtype)
    nan = lambda c: torch.full((rows, c), float("nan"), dtype=dtype, device=device())    # noqa: E731
    hh, d_gu, h2 = nan(I), nan(2 * I), nan(I)
    moe.moe_swiglu(gu, hh)
    want, e = ref.swiglu(ref.f64(gu))
    ref.close(hh, want, ref.rounded(want, e, dtype))
    moe.moe_swiglu_backward(d, gu, d_gu, h2)
    assert torch.equal(h2, hh)
    want, e = ref.swiglu_backward(ref.f64(d), ref.f64(gu))
    ref.close(d_gu, want, ref.rounded(want, e, dtype))
    a, b = gu.clone(), d.clone()                     # in place of both
    moe.moe_swiglu_backward(b, a, a, b)
    assert torch.equal(a, d_gu) and torch.equal(b, hh)


@pytest.mark.parametrize("rows,I", [(1, 32), (3, 96), (70, 1024), (700, 160)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_swiglu_of_kept_values(rows, I, dtype):
    rng = np.random.default_rng(I)
    gu = _t(rng.standard_normal((rows, 2 * I)) * 4, dtype)
    d = _t(rng.standard_normal((rows, I)), dtype)
    nan = lambda c: torch.full((rows, c), float("nan"), dtype=dtype, device=device())    # noqa: E731
    hh, h2, kept, want = nan(I), nan(I), _kept((rows, 2 * I)), _kept((rows, 2 * I))
    moe.moe_swiglu(gu, hh, checkpoint=kept)
    moe.moe_swiglu(gu, h2)
    moe.moe_mxfp8_quantize(gu, *want)
    assert torch.equal(hh, h2) and torch.equal(kept.codes, want.codes) and torch.equal(kept.scales, want.scales)
    v = ref.mx8_values(kept.codes.cpu().numpy(), kept.scales.cpu().numpy())
    d_gu, h3 = nan(2 * I), nan(I)
    moe.moe_swiglu_backward(d, kept, d_gu, h3)
    dw, e = ref.swiglu_backward(ref.f64(d), v)
    ref.close(d_gu, dw, ref.rounded(dw, e, dtype))
    hw, e = ref.swiglu(v)
    ref.close(h3, hw, ref.rounded(hw, e, dtype))


def test_swiglu_of_far_gates():
    """Gates of any finite size: the sigmoid's ends."""
    g = np.array([0.0, -0.0, 1e-30, -1e-30, 20, -20, 60, -60, 87, -87, 88.8, -88.8, 104, -104, 1e4, -1e4, 1e30, -1e30,
                  3e38, -3e38, -1.2784645, 2.0 ** -149, 88.0, -88.0])
    gu = _t(np.concatenate([g, np.resize([1.0, -0.5, 3.0], 24)])[None])
    d = _t(np.resize([1.0, 0.25, -2.0], 24)[None])
    hh, d_gu = torch.empty((1, 24), device=device()), torch.empty((1, 48), device=device())
    moe.moe_swiglu(gu, hh)
    x = ref.f64(gu)
    want, e = ref.swiglu(x)
    big = np.abs(want) > 3.4e38
    got = ref.f64(hh)
    assert (np.isinf(got) == big).all()
    ref.close(np.where(big, 0, got), np.where(big, 0, want), np.where(big, 0, e) + 1e-37)
    moe.moe_swiglu_backward(d, gu, d_gu)
    want, e = ref.swiglu_backward(ref.f64(d), x)
    big = np.abs(want) > 3.4e38
    got = ref.f64(d_gu)
    assert (np.isinf(got) == big).all()
    ref.close(np.where(big, 0, got), np.where(big, 0, want), np.where(big, 0, e) + 1e-37)


def test_more_than_4_gib():
    """Rows past 2^32 bytes, by their values at the ends."""
    rows, cols = (1 << 20) + 3, 4096
    kept = moe.alloc_checkpoint((rows, cols))
    x = torch.zeros((rows, cols), dtype=BF16, device=device())
    x[-2:] = _t(np.random.default_rng(0).standard_normal((2, cols)), BF16)
    moe.moe_mxfp8_quantize(x, *kept)
    codes, scales = ref.mx8_quantize(ref.f64(x[-2:]))
    assert np.array_equal(kept.codes[-2:].cpu().numpy(), codes)
    assert np.array_equal(kept.scales[-2:].cpu().numpy(), scales) and (kept.scales[:100] == 0).all()
    moe.moe_mxfp8_dequantize(*kept, x)
    assert np.array_equal(ref.f64(x[-2:]), ref.mx8_values(codes, scales)) and (x[:-2] == 0).all()
    hh = torch.full((rows, cols // 2), 3.0, dtype=BF16, device=device())
    d_gu = torch.full((rows, cols), 3.0, dtype=BF16, device=device())
    moe.moe_swiglu(x, hh)
    want, e = ref.swiglu(ref.f64(x[-2:]))
    ref.close(hh[-2:], want, ref.rounded(want, e, BF16))
    moe.moe_swiglu_backward(hh, kept, d_gu)
    want, e = ref.swiglu_backward(ref.f64(hh[-2:]), ref.f64(x[-2:]))
    ref.close(d_gu[-2:], want, ref.rounded(want, e, BF16))
    assert (d_gu[:-2] == 0).all()
