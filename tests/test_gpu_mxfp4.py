"""MXFP4 conversion and the grouped products on MXFP4 weights against plain
64-bit forms, through the binding."""
import numpy as np
import pytest
import torch

import sparse_moe_layer_02_amd as moe
from _mxfp4 import product, quantize, spans, values
from _parity import device, host

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _dev(a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a)).to(device())
    return t if dtype is None else t.to(dtype)


def _f64(t):
    return t.double().cpu().numpy()


def _inside(got, want, bound):
    """got within bound of want where want is finite, and of the same kind where it is not."""
    fine = np.isfinite(want)
    assert np.isfinite(got[fine]).all()
    d = np.abs(got[fine] - want[fine]) - bound[fine]
    assert d.size == 0 or d.max() <= 0, (d.max(), int((d > 0).sum()))
    assert np.isnan(got[np.isnan(want)]).all()


# ------------------------------------------------------------- conversion --

def _special_rows():
    rng = np.random.default_rng(3)
    r = [rng.standard_normal(32) * 2.0 ** e for e in (-126, -60, -9, 0, 9, 60, 120)]
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 7.99, 6.0]
    r.append(np.array(mids + [-m for m in mids] + [4.0] * 12))     # scale 1: ties and saturation
    r.append(np.zeros(32))
    r.append(np.concatenate([[-0.0, 0.0], np.full(30, 2.0 ** -140)]))   # subnormal, scale at its least
    r.append(np.full(32, 3.3e38) * rng.choice([-1, 1], 32))
    r.append(np.concatenate([[2.0 ** -125, 2.0 ** -124 * 1.5, 2.0 ** -126], np.zeros(29)]))
    return np.array(r).reshape(1, -1)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (129, 2048), (5, 7, 160), "special"])
def test_quantize_is_exact(dtype, shape):
    print(f"\n[case] quantize {dtype} {shape}", flush=True)
    rng = np.random.default_rng(5)
    if shape == "special":
        x = _special_rows()
    else:
        x = rng.standard_normal(shape) * np.exp2(rng.integers(-12, 12, (*shape[:-1], 1)))
    t = _dev(x, F32).to(dtype)
    q = moe.quantize_weights(t)
    codes, scales = quantize(_f64(t))
    assert np.array_equal(host(q.scales), scales)
    assert np.array_equal(host(q.codes), codes)
    want = values(codes, scales)
    for out in (F32, BF16):
        y = torch.full(t.shape, float("nan"), dtype=out, device=t.device)
        moe.moe_mxfp4_dequantize(q.codes, q.scales, y)
        assert np.array_equal(_f64(y), want)


def test_quantize_marks_blocks_that_are_not_finite():
    x = np.random.default_rng(7).standard_normal((4, 128)).astype(np.float32)
    x[0, 5], x[1, 40], x[2, 127], x[3, 64] = np.nan, np.inf, -np.inf, 1e30
    q = moe.quantize_weights(_dev(x))
    want = quantize(x.astype(np.float64))[1]
    assert np.array_equal(host(q.scales), want) and (want == 255).sum() == 3
    y = torch.empty(x.shape, dtype=F32, device=q.codes.device)
    moe.moe_mxfp4_dequantize(q.codes, q.scales, y)
    bad = np.repeat(want == 255, 32, axis=1)
    assert np.array_equal(np.isnan(host(y)), bad)


@pytest.mark.parametrize("n", [-3, 0, 1, 7, 20, 1000])
def test_quantize_takes_its_row_count_from_the_device(n):
    x = _dev(np.random.default_rng(1).standard_normal((20, 96)), F32)
    codes = torch.full((20, 48), 0xAB, dtype=torch.uint8, device=x.device)
    scales = torch.full((20, 3), 0xCD, dtype=torch.uint8, device=x.device)
    moe.moe_mxfp4_quantize(x, codes, scales, _dev(np.array([n], np.int32)))
    live = min(max(n, 0), 20)
    want = quantize(_f64(x))
    assert np.array_equal(host(codes)[:live], want[0][:live])
    assert np.array_equal(host(scales)[:live], want[1][:live])
    assert (host(codes)[live:] == 0xAB).all() and (host(scales)[live:] == 0xCD).all()


@pytest.mark.parametrize("out", [F32, BF16])
def test_every_code_and_scale(out):
    """All 16 codes at all 256 scales, the least and the NaN among them."""
    codes = np.tile(np.arange(16, dtype=np.uint8) * 16 + np.arange(16, dtype=np.uint8), (256, 1))
    scales = np.arange(256, dtype=np.uint8).reshape(256, 1)
    y = torch.empty((256, 32), dtype=out, device=device())
    moe.moe_mxfp4_dequantize(_dev(codes), _dev(scales), y)
    want = values(codes, scales)
    want[np.abs(want) > torch.finfo(F32).max] *= np.inf        # 4 and 6 times 2^127
    got = _f64(y)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(got[:255], want[:255])


# --------------------------------------------------------------- products --

def _rows(kind, m, D, rng):
    """(tensor, scales or None, float64 values) of m rows."""
    x = rng.standard_normal((m, D)) * np.exp2(rng.integers(-2, 3, (m, 1)))
    if kind == "bf16":
        t = _dev(x, BF16)
        return t, None, _f64(t)
    c, s = quantize(x)
    return _dev(c), _dev(s), values(c, s)


def _weights(E, N, D, rng):
    c, s = quantize(rng.standard_normal((E, N, D)) / np.sqrt(D))
    return _dev(c), _dev(s), values(c, s)


def _run_product(kind, counts, D, N, swiglu, out, gather=None, cap=None, seed=0, T=None, K=1):
    """One grouped product; gather: token picks per expert are drawn from T tokens with K slots."""
    rng = np.random.default_rng(seed)
    E, S = len(counts), int(np.sum(counts))
    cap = max(S, 1) if cap is None else cap
    offsets = spans(counts)
    w, ws_, wv = _weights(E, N, D, rng)
    if gather:
        a, as_, av = _rows(kind, T, D, rng)
        src = np.concatenate([np.sort(rng.permutation(T)[:c]) for c in counts] or [[]]).astype(np.int64)
        slot = rng.integers(0, K, S)
        row_src = np.full(cap, -7, np.int32)
        row_src[:S] = src * K + slot
        av = av[src]
    else:
        a, as_, av = _rows(kind, cap, D, rng)
        row_src = None
    width = N // 2 if swiglu else N
    y = torch.full((cap, width), float("nan"), dtype=out, device=device())
    work = torch.full((moe.moe_grouped_gemm_mxfp4_workspace_bytes(cap, E),), 0xAB,
                      dtype=torch.uint8, device=device())
    moe.moe_grouped_gemm_mxfp4(a, as_, _dev(offsets), w, ws_, y, work,
                               row_src=None if row_src is None else _dev(row_src), K=K,
                               swiglu=swiglu)
    torch.cuda.synchronize()
    got = _f64(y)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        want, bound = product(av[lo:hi], wv[e], swiglu, out is BF16)
        _inside(got[lo:hi], want, bound)
    assert np.isnan(got[S:]).all()                   # rows behind the last span untouched


RAGGED = (0, 1, 16, 0, 17, 33, 64, 65, 100, 129, 192, 193, 256, 257, 300, 0)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("swiglu,out", [(False, F32), (False, BF16), (True, BF16), (True, F32)])
def test_products_of_ragged_experts(kind, swiglu, out):
    print(f"\n[case] {kind} swiglu={swiglu} {out}", flush=True)
    _run_product(kind, RAGGED, 640, 544, swiglu, out, cap=sum(RAGGED) + 77)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("D", [128, 256, 384, 512, 640, 896, 1024, 1152, 2048])
@pytest.mark.parametrize("counts", [(3, 0, 30), (70, 5)])
def test_products_at_row_lengths(kind, D, counts):
    print(f"\n[case] {kind} D={D} {counts}", flush=True)
    _run_product(kind, counts, D, 80, False, F32, seed=D)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("N,swiglu", [(16, False), (16, True), (32, True), (48, False), (64, True),
                                      (240, True), (256, False), (272, False), (528, True)])
@pytest.mark.parametrize("counts", [(1, 2, 20), (200,)])
def test_products_at_widths(kind, N, swiglu, counts):
    print(f"\n[case] {kind} N={N} swiglu={swiglu} {counts}", flush=True)
    _run_product(kind, counts, 256, N, swiglu, BF16, seed=N)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T,K,counts", [(1, 1, (1,)), (1, 12, (1, 0, 1, 1)), (7, 3, (0, 7, 2, 0)),
                                        (32, 2, (32, 31, 0, 17, 16)), (33, 4, (33, 1, 32)),
                                        (700, 4, (700, 0, 40, 513))])
def test_products_through_the_dispatch_indices(kind, T, K, counts):
    print(f"\n[case] {kind} T={T} K={K} {counts}", flush=True)
    _run_product(kind, counts, 384, 96, True, BF16, gather=True, T=T, K=K,
                 cap=max(T * K, sum(counts)), seed=T)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("E,N,D", [(200, 512, 128), (512, 256, 128), (1500, 32, 128)])
def test_products_of_many_experts(kind, E, N, D):
    """Enough blocks that every column width of the small-batch kernel is chosen."""
    print(f"\n[case] {kind} E={E} N={N}", flush=True)
    counts = np.random.default_rng(E).integers(0, 3, E)
    _run_product(kind, tuple(counts), D, N, False, F32)
    _run_product(kind, tuple(np.minimum(counts, 1)), D, N, False, BF16, gather=True, T=24, K=100,
                 cap=2400)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("gather", [False, True])
def test_few_rows_on_average_and_many_in_one_expert(kind, gather):
    """The decode kernel takes a crowded expert 16 rows at a time, past 64 experts and empty ones."""
    counts = (100,) + (0,) * 70 + (5, 17, 0, 1, 32) + (0,) * 3
    _run_product(kind, counts, 640, 144, not gather, BF16, gather=gather, T=100, K=2, cap=200)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_malformed_offsets_stay_inside_the_buffers(kind):
    """Spans that run backwards or past the rows are clamped: rows of the spans that remain are
    right, and nothing is read or written outside."""
    rng = np.random.default_rng(8)
    cap, E, D, N = 60, 4, 128, 16
    a, as_, av = _rows(kind, cap, D, rng)
    w, ws_, wv = _weights(E, N, D, rng)
    off = np.array([-5, 20, 10, 40, 1000], np.int32)     # spans [0, 20), none, [10, 40), [40, 60)
    y = torch.full((cap, N), float("nan"), dtype=F32, device=device())
    work = torch.empty(moe.moe_grouped_gemm_mxfp4_workspace_bytes(cap, E), dtype=torch.uint8,
                       device=device())
    moe.moe_grouped_gemm_mxfp4(a, as_, _dev(off), w, ws_, y, work)
    got = _f64(y)
    for e, lo, hi in ((0, 0, 10), (2, 20, 40), (3, 40, 60)):
        want, bound = product(av[lo:hi], wv[e], False, False)
        _inside(got[lo:hi], want, bound)


@pytest.mark.parametrize("out", [F32, BF16])
def test_swiglu_of_far_gates(out):
    """Gates from far below to far above what exp reaches: 0 and the up column times the gate."""
    gates = np.array([-3e4, -200, -104, -88, -60, -10, -1, -0.0, 0.0, 1, 10, 60, 88, 104, 200, 3e4])
    D, N = 128, 32
    w = np.zeros((1, N, D))
    w[0, :16, 0], w[0, 16:, 1] = 1.0, 1.0
    c, s = quantize(w)
    a = np.zeros((16, D))
    a[:, 0], a[:, 1] = gates, 2.0
    t = _dev(a, BF16)
    y = torch.empty((16, 16), dtype=out, device=device())
    work = torch.empty(moe.moe_grouped_gemm_mxfp4_workspace_bytes(16, 1), dtype=torch.uint8,
                       device=device())
    moe.moe_grouped_gemm_mxfp4(t, None, _dev(spans([16])), _dev(c), _dev(s), y, work, swiglu=True)
    want, bound = product(_f64(t), values(c, s)[0], True, out is BF16)
    # below 2^-126 a result may be rounded to a coarser step or to zero
    _inside(_f64(y), want, bound + 2.0 ** -126)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_offsets_past_32_bits(kind):
    """Rows, weights and outputs that lie more than 4 GiB into their tensors."""
    D, N, E, T = 6144, 2048, 720, 400000          # bf16 rows 4.9 GB, codes 4.5 GB, out 1.6 GB
    dev, rng = device(), np.random.default_rng(9)
    w = torch.zeros((E, N, D // 2), dtype=torch.uint8, device=dev)
    ws_ = torch.zeros((E, N, D // 32), dtype=torch.uint8, device=dev)
    c, s = quantize(rng.standard_normal((2, N, D)) / np.sqrt(D))
    w[-2:], ws_[-2:] = _dev(c), _dev(s)
    rows = 4 * T if kind == "mxfp4" else T        # 4-bit rows: 1.6 M of them, 4.9 GB
    a = torch.zeros((rows, D // 2 if kind == "mxfp4" else D), device=dev,
                    dtype=torch.uint8 if kind == "mxfp4" else BF16)
    as_ = torch.zeros((rows, D // 32), dtype=torch.uint8, device=dev) if kind == "mxfp4" else None
    t, ts, tv = _rows(kind, 40, D, rng)
    a[-40:] = t
    if as_ is not None:
        as_[-40:] = ts
    off = np.zeros(E + 1, np.int32)
    off[-2], off[-1] = 25, 40
    src = torch.arange(rows - 40, rows, dtype=torch.int32, device=dev)
    y = torch.empty((40, N), dtype=F32, device=dev)
    work = torch.empty(moe.moe_grouped_gemm_mxfp4_workspace_bytes(40, E), dtype=torch.uint8,
                       device=dev)
    moe.moe_grouped_gemm_mxfp4(a, as_, _dev(off), w, ws_, y, work, row_src=src, K=1)
    for e, lo, hi in ((0, 0, 25), (1, 25, 40)):
        want, bound = product(tv[lo:hi], values(c[e], s[e]), False, False)
        _inside(_f64(y)[lo:hi], want, bound)


def test_conversion_past_32_bits():
    """More than 2^32 values: the last rows are converted where they belong."""
    rows, cols = (1 << 32) // 4096 + 8, 4096
    x = torch.zeros((rows, cols), dtype=BF16, device=device())
    x[-8:] = _dev(np.random.default_rng(1).standard_normal((8, cols)), BF16)
    q = moe.quantize_weights(x)
    codes, scales = quantize(_f64(x[-8:]))
    assert np.array_equal(host(q.codes[-8:]), codes) and np.array_equal(host(q.scales[-8:]), scales)
    assert not q.codes[:-8].any()
    y = torch.ones_like(x)
    moe.moe_mxfp4_dequantize(q.codes, q.scales, y)
    assert np.array_equal(_f64(y[-8:]), values(codes, scales)) and not y[:-8].any()


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_an_expert_that_holds_a_token_more_than_once(kind):
    """More rows than tokens in one expert (no dispatch makes them, the call takes them)."""
    rng = np.random.default_rng(2)
    T, K, S, D, N = 3, 40, 100, 128, 32
    a, as_, av = _rows(kind, T, D, rng)
    w, ws_, wv = _weights(1, N, D, rng)
    src = rng.integers(0, T * K, S).astype(np.int32)
    y = torch.full((S, N), float("nan"), dtype=F32, device=device())
    work = torch.empty(moe.moe_grouped_gemm_mxfp4_workspace_bytes(S, 1), dtype=torch.uint8,
                       device=device())
    moe.moe_grouped_gemm_mxfp4(a, as_, _dev(spans([S])), w, ws_, y, work, row_src=_dev(src), K=K)
    want, bound = product(av[src // K], wv[0], False, False)
    _inside(_f64(y), want, bound)


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
@pytest.mark.parametrize("D", [256, 640])
def test_nan_scales_stay_in_their_weight_row_and_activation_row(kind, D):
    """Scale byte 255: NaN, in that output column or row alone, also where the last chunk overlaps
    the one before; a row or column that has none is not touched by one that has."""
    rng = np.random.default_rng(4)
    counts, N = (5, 40), 48
    a, as_, av = _rows(kind, 45, D, rng)
    w, ws_, wv = _weights(2, N, D, rng)
    ws_[0, 7, D // 32 - 1] = 255
    ws_[1, 3, 0] = 255
    wv[0, 7, -32:] = np.nan
    wv[1, 3, :32] = np.nan
    if as_ is not None:
        as_[2, 1] = 255
        av[2, 32:64] = np.nan
    else:
        a[2, 40] = float("nan")
        av[2, 40] = np.nan
    y = torch.empty((45, N), dtype=F32, device=device())
    work = torch.empty(moe.moe_grouped_gemm_mxfp4_workspace_bytes(45, 2), dtype=torch.uint8,
                       device=device())
    moe.moe_grouped_gemm_mxfp4(a, as_, _dev(spans(counts)), w, ws_, y, work)
    got = _f64(y)
    for e, (lo, hi) in enumerate(((0, 5), (5, 45))):
        want, bound = product(av[lo:hi], wv[e], False, False)
        _inside(got[lo:hi], want, bound)
    assert np.isnan(got).sum() == 5 + 40 + N - 1


@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_extreme_scales(kind):
    """Weights at the least and near the largest scales, rows at the opposite ones."""
    rng = np.random.default_rng(6)
    D, N = 128, 16
    c, _ = quantize(rng.standard_normal((2, N, D)))
    s = np.empty((2, N, D // 32), np.uint8)
    s[0], s[1] = 0, 250
    x = rng.standard_normal((6, D))
    x[:3] *= 2.0 ** 100
    x[3:] *= 2.0 ** -100
    if kind == "bf16":
        a, as_ = _dev(x, F32).to(BF16), None
        av = _f64(a)
    else:
        cc, ss = quantize(x)
        a, as_, av = _dev(cc), _dev(ss), values(cc, ss)
    y = torch.empty((6, N), dtype=F32, device=device())
    work = torch.empty(moe.moe_grouped_gemm_mxfp4_workspace_bytes(6, 2), dtype=torch.uint8,
                       device=device())
    moe.moe_grouped_gemm_mxfp4(a, as_, _dev(spans((3, 3))), _dev(c), _dev(s), y, work)
    for e in range(2):
        want, bound = product(av[3 * e:3 * e + 3], values(c[e], s[e]), False, False)
        _inside(_f64(y)[3 * e:3 * e + 3], want, bound)


# ------------------------------------------------------------ expert FFN --

def _ffn_inputs(T, K, pool, E, H, I, seed):
    rng = np.random.default_rng(seed)
    picks = np.stack([rng.permutation(pool)[:K] for _ in range(T)]).reshape(-1)
    order = np.argsort(picks, kind="stable")
    order = order[picks[order] < E]
    counts = np.bincount(picks[order], minlength=E)
    row_src = np.zeros(T * K, np.int32)
    row_src[:len(order)] = order
    return rng, counts, row_src, order // K


@pytest.mark.parametrize("T,K,pool,E,H,I", [(1, 4, 6, 4, 128, 128), (5, 3, 9, 6, 256, 384),
                                            (64, 12, 48, 32, 640, 256), (300, 4, 12, 8, 512, 128),
                                            (600, 2, 3, 2, 1024, 640)])
def test_expert_ffn(T, K, pool, E, H, I):
    print(f"\n[case] ffn T={T} K={K} E={E}/{pool} H={H} I={I}", flush=True)
    rng, counts, row_src, tok = _ffn_inputs(T, K, pool, E, H, I, T)
    x = _dev(rng.standard_normal((T, H)), BF16)
    w13, w13s, v13 = _weights(E, 2 * I, H, rng)
    w2, w2s, v2 = _weights(E, H, I, rng)
    offsets = spans(counts)
    y = torch.full((T * K, H), float("nan"), dtype=BF16, device=device())
    work = torch.full((moe.moe_expert_ffn_mxfp4_workspace_bytes(T * K, E, I),), 0xAB,
                      dtype=torch.uint8, device=device())
    moe.moe_expert_ffn_mxfp4(x, None, K, _dev(row_src), _dev(offsets), w13, w13s, w2, w2s, y, work)
    got, xv = _f64(y), _f64(x)
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        h, eh = product(xv[tok[lo:hi]], v13[e], True, True)
        want, bound = product(h, v2[e], False, True, a_err=eh)
        _inside(got[lo:hi], want, bound)
    assert np.isnan(got[offsets[-1]:]).all()


@pytest.mark.parametrize("T", [3, 200])
def test_expert_ffn_on_4bit_rows_is_its_three_calls(T):
    """x in MXFP4: gate/up product, conversion of its rows, down product, bit for bit."""
    K, pool, E, H, I = 4, 12, 8, 384, 256
    rng, counts, row_src, _ = _ffn_inputs(T, K, pool, E, H, I, T)
    x, xs, _ = _rows("mxfp4", T, H, rng)
    w13, w13s, _ = _weights(E, 2 * I, H, rng)
    w2, w2s, _ = _weights(E, H, I, rng)
    offsets, row_src, cap = _dev(spans(counts)), _dev(row_src), T * K
    S = int(counts.sum())
    y = torch.full((cap, H), float("nan"), dtype=BF16, device=device())
    work = torch.full((moe.moe_expert_ffn_mxfp4_workspace_bytes(cap, E, I),), 0xAB,
                      dtype=torch.uint8, device=device())
    moe.moe_expert_ffn_mxfp4(x, xs, K, row_src, offsets, w13, w13s, w2, w2s, y, work)
    hh = torch.zeros((cap, I), dtype=BF16, device=device())
    work2 = torch.empty(moe.moe_grouped_gemm_mxfp4_workspace_bytes(cap, E), dtype=torch.uint8,
                        device=device())
    moe.moe_grouped_gemm_mxfp4(x, xs, offsets, w13, w13s, hh, work2, row_src=row_src, K=K,
                               swiglu=True)
    q = moe.quantize_weights(hh)
    z = torch.full((cap, H), float("nan"), dtype=BF16, device=device())
    moe.moe_grouped_gemm_mxfp4(q.codes, q.scales, offsets, w2, w2s, z, work2)
    assert S > 0 and torch.equal(y[:S], z[:S]) and torch.isfinite(y[:S].float()).all()
    assert torch.isnan(y[S:].float()).all()
