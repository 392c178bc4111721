"""The grouped 4-bit products and the experts on small batches, whose experts have few rows each and
take a kernel of their own; with it the choice between the kernels, malformed offsets in both, and
the layer at full width."""
import numpy as np
import pytest
import torch

import sparse_moe_layer_02_amd as moe
import workload
from _mxfp4 import product, quantize, spans, values
from _parity import device, host
from test_gpu_mxfp4 import _dev, _f64, _inside, _rows

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
KINDS = ("bf16", "mxfp4")


def _weights(E, N, D, seed):
    """4-bit weights of E experts, made on the GPU."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return moe.quantize_weights(torch.randn((E, N, D), generator=g, device=device()) / D ** 0.5)


def _value(q, e):
    return values(host(q.codes[e]), host(q.scales[e]))


def _kernels(f):
    """Names of the kernels that f() launches."""
    moe.moe_profile_enable(True)
    try:
        f()
        torch.cuda.synchronize()
        return set(moe.moe_profile_summary())
    finally:
        moe.moe_profile_enable(False)


def _work(cap, E):
    return torch.full((moe.moe_grouped_gemm_mxfp4_workspace_bytes(cap, E),), 0xAB, dtype=torch.uint8,
                      device=device())


# an expert of 40 rows takes three passes of 16; empty ones between
SMALL = (40, 0, 17, 1, 16, 0, 0, 33, 2) + (0,) * 6 + (3,)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [128, 384, 512, 640, 1024, 1152, 2048])
@pytest.mark.parametrize("N,swiglu,out", [(80, False, F32), (96, True, BF16), (544, True, F32),
                                          (4112, False, BF16)])
def test_small_batches(kind, D, N, swiglu, out):
    """Row lengths from one slice to several chunks, whose last one overlaps; 64 weight rows a block
    (N 80: 16 experts' blocks do not fill the CUs twice) and 128 (N 4112, and SwiGLU)."""
    print(f"\n[case] {kind} D={D} N={N} swiglu={swiglu} {out}", flush=True)
    rng = np.random.default_rng(D + N)
    E, S, cap = len(SMALL), sum(SMALL), 120
    off = spans(SMALL)
    w = _weights(E, N, D, D)
    a, s, v = _rows(kind, cap, D, rng)
    y = torch.full((cap, N // 2 if swiglu else N), float("nan"), dtype=out, device=device())
    ran = _kernels(lambda: moe.moe_grouped_gemm_mxfp4(a, s, _dev(off), w.codes, w.scales, y,
                                                      _work(cap, E), swiglu=swiglu))
    assert ran == {"mx_gemm_few_fp4" if kind == "mxfp4" else "mx_gemm_few_bf16"}
    got = _f64(y)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            _inside(got[lo:hi], *product(v[lo:hi], _value(w, e), swiglu, out is BF16))
    assert np.isnan(got[S:]).all()


def _picks(T, K, E, rng, crowd=True):
    """Dispatch of T tokens that pick K of E experts, the first of them always expert 0 (crowd)."""
    p = np.stack([1 + rng.permutation(E - 1)[:K] for _ in range(T)]) if crowd else \
        np.stack([rng.permutation(E)[:K] for _ in range(T)])
    if crowd:
        p[:, rng.integers(0, K)] = 0
    p = p.reshape(-1)
    src = np.argsort(p, kind="stable").astype(np.int32)
    return np.bincount(p, minlength=E), src


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,K,E,D", [(1, 4, 16, 640), (16, 12, 20, 1152), (64, 8, 64, 1152),
                                     (128, 2, 64, 2048)])
def test_small_batches_through_the_dispatch_indices(kind, T, K, E, D):
    print(f"\n[case] {kind} T={T} K={K} E={E} D={D}", flush=True)
    rng = np.random.default_rng(T)
    counts, src = _picks(T, K, E, rng)
    off, cap, N = spans(counts), T * K, 160
    w = _weights(E, N, D, T)
    a, s, v = _rows(kind, T, D, rng)
    y = torch.full((cap, N // 2), float("nan"), dtype=BF16, device=device())
    ran = _kernels(lambda: moe.moe_grouped_gemm_mxfp4(
        a, s, _dev(off), w.codes, w.scales, y, _work(cap, E), row_src=_dev(src), K=K, swiglu=True))
    assert ran == {"mx_gemm_few_fp4" if kind == "mxfp4" else "mx_gemm_few_bf16"}
    got = _f64(y)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            _inside(got[lo:hi], *product(v[src[lo:hi] // K], _value(w, e), True, True))


@pytest.mark.parametrize("T,K,E,H,I", [(1, 12, 24, 1152, 640), (16, 4, 8, 640, 1152),
                                       (64, 8, 64, 1152, 384)])
def test_experts_of_small_batches(T, K, E, H, I):
    """Both products in the small-batch kernel, row lengths past a chunk, one expert with every token."""
    print(f"\n[case] ffn T={T} K={K} E={E} H={H} I={I}", flush=True)
    rng = np.random.default_rng(T)
    counts, src = _picks(T, K, E, rng)
    off, cap = spans(counts), T * K
    w13, w2 = _weights(E, 2 * I, H, T), _weights(E, H, I, T + 1)
    x, _, v = _rows("bf16", T, H, rng)
    y = torch.full((cap, H), float("nan"), dtype=BF16, device=device())
    work = torch.full((moe.moe_expert_ffn_mxfp4_workspace_bytes(cap, E, I),), 0xAB, dtype=torch.uint8,
                      device=device())
    ran = _kernels(lambda: moe.moe_expert_ffn_mxfp4(x, None, K, _dev(src), _dev(off), *w13, *w2, y,
                                                    work))
    assert ran == {"mx_gemm_few_bf16"}
    got = _f64(y)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            h, eh = product(v[src[lo:hi] // K], _value(w13, e), True, True)
            _inside(got[lo:hi], *product(h, _value(w2, e), False, True, a_err=eh))


@pytest.mark.parametrize("spread", [0, 12, 30])
def test_4bit_rows_give_the_same_bits_in_either_kernel(spread):
    """Whether the rows come in a buffer of 120 rows (small-batch kernel) or of 600 (m-tile list, 32 x
    32 instructions): fp32 sums of products of 4-bit rows are the same bits, also where the blocks of
    a row differ by 2^30 in size."""
    rng = np.random.default_rng(spread)
    counts = (60, 17, 33) + (0,) * 61
    E, D, N, S = 64, 1152, 512, 110
    w, off = _weights(E, N, D, spread), _dev(spans(counts))
    a, s = quantize(rng.standard_normal((600, D)) *
                    np.exp2(rng.integers(-spread // 2, spread // 2 + 1, (600, D // 32)).repeat(32, 1)))
    got = []
    for cap, kernel in ((120, {"mx_gemm_few_fp4"}), (600, {"mx_gemm_any_fp4", "mx_tiles"})):
        y = torch.full((cap, N), float("nan"), dtype=F32, device=device())
        ran = _kernels(lambda: moe.moe_grouped_gemm_mxfp4(_dev(a[:cap]), _dev(s[:cap]), off, w.codes,
                                                          w.scales, y, _work(cap, E)))
        assert ran == kernel
        got.append(y[:S])
    assert torch.equal(*got) and torch.isfinite(got[0]).all()


def test_experts_on_4bit_rows_are_their_three_calls_in_either_kernel():
    """The experts know the number of tokens and take the small-batch kernel for both products, the
    down product called by itself takes the list: bit for bit the same."""
    T, K, E, H, I = 100, 4, 64, 1152, 512
    rng = np.random.default_rng(1)
    counts = np.array((60,) + (2,) * 63)
    off, cap, S = spans(counts), T * K, 186
    src = np.zeros(cap, np.int32)
    for e in range(E):
        src[off[e]:off[e + 1]] = np.sort(rng.permutation(T)[:counts[e]]) * K + e % K
    w13, w2 = _weights(E, 2 * I, H, 1), _weights(E, H, I, 2)
    x, xs, _ = _rows("mxfp4", T, H, rng)
    off, src = _dev(off), _dev(src)
    y = torch.empty((cap, H), dtype=BF16, device=device())
    z, hh = torch.empty_like(y), torch.zeros((cap, I), dtype=BF16, device=device())
    work = torch.empty(moe.moe_expert_ffn_mxfp4_workspace_bytes(cap, E, I), dtype=torch.uint8,
                       device=device())
    ran = _kernels(lambda: moe.moe_expert_ffn_mxfp4(x, xs, K, src, off, *w13, *w2, y, work))
    assert ran == {"mx_gemm_few_fp4", "mxfp4_quantize"}
    moe.moe_grouped_gemm_mxfp4(x, xs, off, *w13, hh, _work(cap, E), row_src=src, K=K, swiglu=True)
    q = moe.quantize_weights(hh)
    ran = _kernels(lambda: moe.moe_grouped_gemm_mxfp4(*q, off, *w2, z, _work(cap, E)))
    assert ran == {"mx_gemm_any_fp4", "mx_tiles"}
    assert torch.equal(y[:S], z[:S]) and torch.isfinite(y[:S].float()).all()


# ------------------------------------------------------- the largest scales --

@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("byte", [0, 1, 251, 252, 253, 254])
@pytest.mark.parametrize("cap", [4, 200])
def test_weights_at_the_least_and_largest_scales(kind, byte, cap):
    """Every code at the ends of the scales: 4-bit rows multiply the values themselves, bf16 rows the
    values in bf16, where 2^128 and more is an infinity.  Powers of two in the rows: nothing rounds."""
    D, N = 128, 16
    c = np.zeros((1, N, D // 2), np.uint8)
    c[0, :, 0] = np.arange(16)                       # value 0 of weight row n is code n, the rest 0
    s = np.full((1, N, D // 32), byte, np.uint8)
    a = np.zeros((4, D))
    a[:, 0] = [2.0 ** -100, 2.0 ** -3, 0.0, -(2.0 ** -120)]
    a[2, 1] = 1.0
    qa, qs = quantize(a)
    t, ts = (_dev(a, BF16), None) if kind == "bf16" else (_dev(qa), _dev(qs))
    pad = lambda x: None if x is None else torch.cat([x, x[:1].expand(cap - 4, -1)]).contiguous()  # noqa: E731
    y = torch.empty((cap, N), dtype=F32, device=device())
    moe.moe_grouped_gemm_mxfp4(pad(t), pad(ts), _dev(spans([cap])), _dev(c), _dev(s), y, _work(cap, 1))
    w = values(c[0], s[0])
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "bf16":
            w = np.where(np.abs(w) >= 2.0 ** 128, np.sign(w) * np.inf, w)
        want = (a[:, None, :2] * w[None, :, :2]).sum(-1).astype(np.float32)
    got, tiny = host(y)[:4], np.abs(want) < 2.0 ** -126
    same = (got == want) | (np.isnan(got) & np.isnan(want)) | (tiny & (np.abs(got) <= 2.0 ** -126))
    assert same.all(), (got[~same], want[~same])


# ------------------------------------------------------- malformed offsets --

LO, HI = -(1 << 31), (1 << 31) - 1
MALFORMED = [
    ("small batch, more spans than rows", 4, [0, 4] * 20, True),
    ("small batch, spans that overlap", 100, [0, 100, 50, 99, LO, HI] * 4 + [7], True),
    ("list past its capacity", 600, [0, 600] * 6 + [0], False),
    ("list, spans far outside", 600, [LO, -1, HI, 0, 601, 300, LO, HI, HI, 599, 600, 10], False),
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("what,cap,off,few", MALFORMED, ids=[m[0] for m in MALFORMED])
def test_malformed_offsets_write_nothing_outside(what, cap, off, few, kind, gather):
    """Spans that overlap, run backwards or lie outside, more of them than a launch has room for: the
    bytes around the output and the workspace stay, and so do rows that no span holds; a value that is
    written is that of a span that has its row."""
    print(f"\n[case] {what}, {kind}, gather={gather}", flush=True)
    rng = np.random.default_rng(len(off))
    D, N, G = 640, 80, 4096
    E = len(off) - 1
    w = _weights(E, N, D, E)
    a, s, v = _rows(kind, cap, D, rng)
    src = rng.integers(-5, cap + 5, cap).astype(np.int32) if gather else np.arange(cap, dtype=np.int32)
    need = moe.moe_grouped_gemm_mxfp4_workspace_bytes(cap, E)
    box = torch.full((2 * G + cap * N,), 777.0, dtype=F32, device=device())
    y = box[G:G + cap * N].view(cap, N)
    wbox = torch.full((2 * G + need,), 0xAB, dtype=torch.uint8, device=device())
    f = lambda: moe.moe_grouped_gemm_mxfp4(a, s, _dev(np.array(off, np.int32)), w.codes, w.scales, y,  # noqa: E731
                                           wbox[G:G + need], row_src=_dev(src) if gather else None)
    ran = _kernels(f)
    assert any("few" in k for k in ran) == few
    assert (box[:G] == 777).all() and (box[G + cap * N:] == 777).all()
    assert (wbox[:G] == 0xAB).all() and (wbox[G + need:] == 0xAB).all()
    got, rows = _f64(y), v[np.clip(src, 0, cap - 1)]
    fits = np.zeros((cap, N), bool)
    held = np.zeros(cap, bool)
    for e in range(E):
        lo = min(max(off[e], 0), cap)
        hi = min(max(off[e + 1], lo), cap)
        if lo < hi:
            want, bound = product(rows[lo:hi], _value(w, e), False, False)
            fits[lo:hi] |= np.abs(got[lo:hi] - want) <= bound
            held[lo:hi] = True
    untouched = got == 777
    assert (fits | untouched).all() and untouched[~held].all()


# ----------------------------------------------------- the layer, full width --

@pytest.mark.parametrize("T", [48, 400])
def test_layer_of_full_width_on_4bit_weights(T):
    """forward() at 6144 x 2048 with few experts: the experts' rows against 64 bits on the layer's own
    dispatch, and the layer's output from them."""
    print(f"\n[case] layer 6144 x 2048, T={T}", flush=True)
    cfg = workload.MoEConfig("wide", T=T, H=6144, N=4, Z=2, I=2048, K=3, dtype="bf16", sigma_w=0.02,
                             bias_lo=-0.1, bias_hi=0.1, scale=1.5)
    inp = workload.make_inputs(cfg, device())
    w13, w2 = moe.quantize_weights(inp["w13"]), moe.quantize_weights(inp["w2"])
    buf = moe.alloc_buffers(T, cfg.H, cfg.E, cfg.N, cfg.I, cfg.K, BF16, device(), mxfp4=True)
    y = _f64(moe.forward(inp["x"], inp["w_router"], inp["bias"], w13, w2, cfg.K, cfg.scale, buf))
    x, off, src = _f64(inp["x"]), host(buf["offsets"]), host(buf["row_src"])
    slot, gate, yp = host(buf["slot_row"]).reshape(T, cfg.K), _f64(buf["topk_gate"]), _f64(buf["y_perm"])
    assert off[-1] == (host(buf["topk_idx"]) < cfg.N).sum() > 0
    for e in range(cfg.N):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            h, eh = product(x[src[lo:hi] // cfg.K], _value(w13, e), True, True)
            _inside(yp[lo:hi], *product(h, _value(w2, e), False, True, a_err=eh))
    want = np.where(slot < 0, gate, 0).sum(1)[:, None] * x
    size = np.abs(want)
    for k in range(cfg.K):
        live = slot[:, k] >= 0
        term = cfg.scale * gate[live, k:k + 1] * yp[slot[live, k]]
        want[live] += term
        size[live] += np.abs(term)
    # fp32 sums of K + 1 terms, then one rounding to bf16
    assert (np.abs(y - want) <= 2.0 ** -8 * np.abs(want) + 16 * 2.0 ** -23 * size + 1e-30).all()
