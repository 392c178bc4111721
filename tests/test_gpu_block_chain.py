"""Blocks one after another: the norm that a block leaves for the next one is that block's input."""
import pytest
import torch

import sparse_moe_layer_02_amd as moe
from test_gpu_block import EPS, _setup

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def _args(st):
    return st["w_router"], st["bias"], st["w13"], st["w2"]


def _tail(st):
    return dict(scale=0.5, w_post=st["w_post"], gate=st["gate"], gate_kind="token", eps=EPS)


def _chain(cfg, st, buf, blocks):
    """blocks blocks in one set of buffers, each but the first on the last one's norm."""
    h, x = st["h"], None
    for _ in range(blocks):
        h, x = moe.block_forward(h, st["w_norm"] if x is None else None, *_args(st), cfg.K, cfg.scale,
                                 buf, w_next=st["w_next"], x_norm=x, **_tail(st))
    return h, x


@pytest.mark.parametrize("T,res,separate", [(1, F32, False), (40, BF16, False), (300, F32, False),
                                            (1100, BF16, True), (1100, F32, True)])
def test_chain_of_blocks(T, res, separate):
    """A chain in one set of buffers against the same calls written out in buffers of their own; the
    norm in front of a block that is given one does not run."""
    print(f"\n[case] chain T={T} {res} separate={separate}", flush=True)
    cfg, st, _ = _setup(T, seed=3, res=res)
    new = lambda: moe.alloc_buffers(cfg.T, cfg.H, cfg.E, cfg.N, cfg.I, cfg.K, BF16, st["h"].device,  # noqa: E731
                                    mxfp4=True, residual=res, separate_identity=separate)
    h, x = st["h"], torch.empty_like(st["h"], dtype=BF16)
    moe.moe_norm(h, st["w_norm"], x, EPS)
    for _ in range(3):
        b = new()
        y = moe.forward(x, *_args(st), cfg.K, cfg.scale, b)
        moe.moe_norm_residual(y, h, b["h_out"], w_next=st["w_next"], next_out=b["h_norm"], **_tail(st))
        h, x = b["h_out"], b["h_norm"]
    buf = new()
    g, z = _chain(cfg, st, buf, 1)
    buf["x_norm"].fill_(float("nan"))
    for _ in range(2):
        g, z = moe.block_forward(g, None, *_args(st), cfg.K, cfg.scale, buf, w_next=st["w_next"],
                                 x_norm=z, **_tail(st))
    torch.cuda.synchronize()
    assert torch.equal(g, h) and torch.equal(z, x)
    assert torch.isnan(buf["x_norm"]).all()


def test_chain_on_an_fp32_stream_is_the_chain_that_norms_again():
    """With the sums kept in fp32 the norm left behind is bitwise the norm of the stream."""
    cfg, st, buf = _setup(96, seed=4)
    g, z = _chain(cfg, st, buf, 2)
    g, z = g.clone(), z.clone()
    h, _ = moe.block_forward(st["h"], st["w_norm"], *_args(st), cfg.K, cfg.scale, buf,
                             w_next=st["w_next"], **_tail(st))
    h, x = moe.block_forward(h, st["w_next"], *_args(st), cfg.K, cfg.scale, buf,
                             w_next=st["w_next"], **_tail(st))
    torch.cuda.synchronize()
    assert torch.equal(g, h) and torch.equal(z, x)


def test_captured_chain_replays_match_eager():
    cfg, st, buf = _setup(64, seed=5)
    h, x = _chain(cfg, st, buf, 3)
    torch.cuda.synchronize()
    ref = h.clone(), x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _chain(cfg, st, buf, 3)
    for rep in range(3):
        for k in ("h_out", "h_norm", "x_norm", "y", "y_perm"):
            buf[k].fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(h, ref[0]) and torch.equal(x, ref[1]), rep
