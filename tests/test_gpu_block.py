"""The MoE layer as a block of a residual stream on 4-bit expert weights: the
operators together, as they are used, eagerly, on another stream and captured
into a HIP graph."""
import numpy as np
import pytest
import torch

import sparse_moe_layer_02_amd as moe
import workload
from _mxfp4 import EPS_BF16, product, quantize, values
from _parity import device, host

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-5
CFG = workload.MoEConfig("block", T=96, H=512, N=16, Z=8, I=256, K=4, dtype="bf16",
                         sigma_w=0.04, bias_lo=-0.1, bias_hi=0.1, scale=1.5)


def _setup(T, seed=0, res=F32):
    cfg = CFG.replace(T=T, seed=seed)
    dev = device()
    inp = workload.make_inputs(cfg, dev)
    rng = np.random.default_rng(seed)
    w = lambda: torch.as_tensor(1 + 0.1 * rng.standard_normal(cfg.H), dtype=F32).to(dev)  # noqa: E731
    st = dict(h=(inp["x"].float() * 2).to(res), w_norm=w(), w_post=w(), w_next=w(),
              gate=torch.as_tensor(1 + 0.3 * rng.standard_normal(T), dtype=F32).to(dev),
              w13=moe.quantize_weights(inp["w13"]), w2=moe.quantize_weights(inp["w2"]),
              w_router=inp["w_router"], bias=inp["bias"])
    buf = moe.alloc_buffers(cfg.T, cfg.H, cfg.E, cfg.N, cfg.I, cfg.K, BF16, dev, mxfp4=True,
                            residual=res)
    return cfg, st, buf


def _run(cfg, st, buf):
    return moe.block_forward(st["h"], st["w_norm"], st["w_router"], st["bias"], st["w13"],
                             st["w2"], cfg.K, cfg.scale, buf, scale=0.5, w_post=st["w_post"],
                             gate=st["gate"], gate_kind="token", w_next=st["w_next"], eps=EPS)


@pytest.mark.parametrize("T,res", [(1, F32), (40, BF16), (96, F32), (700, BF16)])
def test_block_matches_the_plain_form_stage_by_stage(T, res):
    """Each stage against 64 bits on the stage's own inputs (so that no routing near a tie and no
    rounding of an earlier stage counts), and the block's sum end to end."""
    print(f"\n[case] block T={T} {res}", flush=True)
    cfg, st, buf = _setup(T, res=res)
    h_out, h_norm = _run(cfg, st, buf)
    torch.cuda.synchronize()
    f64 = lambda t: t.double().cpu().numpy()                              # noqa: E731
    h, x = f64(st["h"]), f64(buf["x_norm"])
    n = h / np.sqrt((h * h).mean(-1, keepdims=True) + EPS) * f64(st["w_norm"])
    assert (np.abs(x - n) <= (EPS_BF16 + 1e-4) * np.abs(n) + 1e-30).all()
    off, src, slot = host(buf["offsets"]), host(buf["row_src"]), host(buf["slot_row"])
    S = off[-1]
    assert S == (host(buf["topk_idx"]) < cfg.N).sum()
    w13 = values(host(st["w13"].codes), host(st["w13"].scales))
    w2 = values(host(st["w2"].codes), host(st["w2"].scales))
    yp = f64(buf["y_perm"])
    for e in range(cfg.N):
        lo, hi = off[e], off[e + 1]
        a, ea = product(x[src[lo:hi] // cfg.K], w13[e], True, True)
        want, bound = product(a, w2[e], False, True, a_err=ea)
        assert (np.abs(yp[lo:hi] - want) <= bound).all(), e
    gate, slot = f64(buf["topk_gate"]), slot.reshape(T, cfg.K)
    y = f64(buf["y"])
    want = np.where(slot < 0, gate, 0).sum(1)[:, None] * x
    for k in range(cfg.K):
        live = slot[:, k] >= 0
        want[live] += cfg.scale * gate[live, k:k + 1] * yp[slot[live, k]]
    assert (np.abs(y - want) <= (EPS_BF16 + 1e-5) * np.abs(want) + 1e-5).all()
    z = y / np.sqrt((y * y).mean(-1, keepdims=True) + EPS) * f64(st["w_post"])
    s = h + 0.5 * f64(st["gate"])[:, None] * z
    tol = (EPS_BF16 if res is BF16 else 0) + 1e-4
    size = np.abs(h) + np.abs(s)
    assert (np.abs(f64(h_out) - s) <= tol * size).all()
    m = s / np.sqrt((s * s).mean(-1, keepdims=True) + EPS) * f64(st["w_next"])
    big = size / np.sqrt((s * s).mean(-1, keepdims=True) + EPS) * np.abs(f64(st["w_next"]))
    assert (np.abs(f64(h_norm) - m) <= EPS_BF16 * np.abs(m) + 2e-4 * big).all()


def test_forward_on_4bit_weights_is_forward_on_the_values_they_stand_for():
    """bf16 weights that 4 bits hold exactly: the same layer either way, to the rounding of the
    rows between the products."""
    cfg, st, buf = _setup(96)
    x = st["h"].to(BF16)
    w13, w2 = (torch.empty(q.shape, dtype=BF16, device=x.device) for q in (st["w13"], st["w2"]))
    moe.moe_mxfp4_dequantize(*st["w13"], w13)
    moe.moe_mxfp4_dequantize(*st["w2"], w2)
    y4 = moe.forward(x, st["w_router"], st["bias"], st["w13"], st["w2"], cfg.K, cfg.scale,
                     buf).float().clone()
    buf16 = moe.alloc_buffers(cfg.T, cfg.H, cfg.E, cfg.N, cfg.I, cfg.K, BF16, x.device)
    y16 = moe.forward(x, st["w_router"], st["bias"], w13, w2, cfg.K, cfg.scale, buf16).float()
    # fp32 sums in another order may round a value of hh or of an expert's output to the
    # neighbouring bf16 (2^-7 apart at most): far below the outputs' own size in the 2-norm
    rel = ((y4 - y16).norm() / y16.norm()).item()
    assert rel <= EPS_BF16, rel


@pytest.mark.parametrize("T", [7, 300])
def test_captured_block_replays_match_eager(T):
    cfg, st, buf = _setup(T)
    _run(cfg, st, buf)
    torch.cuda.synchronize()
    outs = ("x_norm", "y", "h_out", "h_norm")
    ref = {k: buf[k].clone() for k in outs}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for k in outs:
            buf[k].fill_(float("nan"))
        _run(cfg, st, buf)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for k in outs:
        assert torch.equal(buf[k], ref[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _run(cfg, st, buf)
    other = torch.randn(1 << 20, device=st["h"].device)
    for rep in range(4):
        for k in (*outs, "y_perm", "logits"):
            buf[k].fill_(float("nan"))
        buf["ws_ffn"].fill_(0xAB)
        buf["offsets"].fill_(-7)
        other.mul_(1.0001)
        torch.cuda.synchronize()
        graph.replay()
        other.add_(1.0)
        torch.cuda.synchronize()
        for k in outs:
            assert torch.equal(buf[k], ref[k]), (rep, k)


def test_two_blocks_on_two_streams():
    """Calls that share no buffer run beside each other; every result is that of the call alone."""
    runs = [_setup(T, seed) for T, seed in ((200, 1), (5, 2))]
    want = []
    for cfg, st, buf in runs:
        _run(cfg, st, buf)
        torch.cuda.synchronize()
        want.append((buf["h_out"].clone(), buf["h_norm"].clone()))
        buf["h_out"].fill_(0)
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, (cfg, st, buf) in zip(streams, runs):
            with torch.cuda.stream(s):
                _run(cfg, st, buf)
    torch.cuda.synchronize()
    for (cfg, st, buf), (a, b) in zip(runs, want):
        assert torch.equal(buf["h_out"], a) and torch.equal(buf["h_norm"], b)
