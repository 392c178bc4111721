"""A training step around the layer as its calls are used together: the norm that keeps its input in 8
bits, router, routing, losses, and the way back to the stream; and the experts' gate and up products with
the SwiGLU kept in 8 bits.  Eager, captured and replayed, and two at once."""
import numpy as np
import pytest
import torch

import _train as ref
import sparse_moe_layer_02_amd as moe
from _parity import device

pytestmark = pytest.mark.gpu
F32, BF16, I32, U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8
EPS, BC, ZC = 1e-5, 0.05, 0.01


class Step:
    """Buffers and calls of one step on T tokens."""

    def __init__(self, T=300, H=512, E=48, K=6, n_seq=3, seed=0):
        d, g = device(), torch.Generator("cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(s, generator=g, device=d)                          # noqa: E731
        e = lambda *s, dtype=F32: torch.empty(s, dtype=dtype, device=d)                 # noqa: E731
        self.K = K
        kept = moe.alloc_checkpoint((T, H))
        self.h = e(T, H)
        moe.moe_mxfp8_quantize(rnd(T, H) * 2, *kept)     # a stream that 8 bits hold exactly
        moe.moe_mxfp8_dequantize(*kept, self.h)
        self.w_norm, self.w_router, self.bias = 1 + 0.2 * rnd(H), rnd(E, H) * 0.05, 0.1 * rnd(E)
        self.d_gate, self.d_out, self.d_losses = rnd(T, K), 0.01 * rnd(T, H), torch.tensor([2.0, 3.0], device=d)
        self.seq = (torch.arange(T, device=d) * n_seq // T).to(I32)
        self.seq[T // 2: T // 2 + 20] = -1
        self.out = dict(kept_codes=kept.codes, kept_scales=kept.scales, x=e(T, H), logits=e(T, E),
                        idx=e(T, K, dtype=I32), gate=e(T, K), route_counts=e(E, dtype=I32),
                        counts=e(n_seq, E, dtype=I32), tokens=e(n_seq + 1, dtype=I32), load=e(n_seq, E),
                        losses=e(2), d_logits=e(T, E), d_x=e(T, H), d_h=e(T, H), d_w=e(H))
        self.ws = e(max(moe.moe_balance_loss_workspace_bytes(T, E, n_seq),
                        moe.moe_norm_backward_workspace_bytes(T, H)), dtype=U8)
        torch.cuda.synchronize()

    def run(self):
        o, kept = self.out, moe.MXFP8(self.out["kept_codes"], self.out["kept_scales"])
        moe.moe_norm_checkpoint(self.h, self.w_norm, o["x"], kept, EPS)
        moe.moe_router_logits(o["x"], self.w_router, o["logits"])
        moe.moe_route(o["logits"], self.bias, self.K, o["idx"], o["gate"], o["route_counts"])
        moe.moe_balance_loss(o["logits"], o["idx"], o["counts"], o["tokens"], o["load"], o["losses"], self.ws,
                             seq=self.seq, balance_coef=BC, z_coef=ZC)
        moe.moe_route_backward(o["logits"], o["d_logits"], o["idx"], self.d_gate, o["tokens"], o["load"], self.seq,
                               self.d_losses, BC, ZC)
        torch.matmul(o["d_logits"], self.w_router, out=o["d_x"])
        moe.moe_norm_backward(o["d_x"], kept, self.w_norm, o["d_h"], o["d_w"], self.ws, EPS, d_residual=self.d_out)

    def poison(self):
        for t in (*self.out.values(), self.ws):
            t.view(torch.uint8).fill_(255)

    def results(self):
        return {k: v.clone() for k, v in self.out.items()}


def _equal(a, b):
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_step_against_its_parts_and_the_whole():
    s = Step()
    s.poison()
    s.run()
    o = {k: ref.f64(v) for k, v in s.out.items()}
    h, w, wr = ref.f64(s.h), ref.f64(s.w_norm), ref.f64(s.w_router)
    codes, scales = ref.mx8_quantize(h)
    assert np.array_equal(s.out["kept_codes"].cpu().numpy(), codes)
    assert np.array_equal(ref.mx8_values(codes, scales), h)
    idx, seq = s.out["idx"].cpu().numpy(), s.seq.cpu().numpy()
    bc, zc = float(np.float32(BC)), float(np.float32(ZC))
    losses, e, counts, tokens, load = ref.balance_loss(o["logits"], idx, seq, 3, None, bc, zc)
    assert np.array_equal(o["counts"], counts) and np.array_equal(o["tokens"], tokens)
    ref.close(s.out["losses"], losses, e)
    dl = ref.f64(s.d_losses)
    want, e = ref.route_backward(o["logits"], idx, ref.f64(s.d_gate), seq, 3, tokens, o["load"], dl, bc, zc)
    ref.close(s.out["d_logits"], want, e + 1e-37)
    eps = float(np.float32(EPS))
    (dx, dw, _), (e, e_w, _) = ref.norm_backward(o["d_x"], h, w, eps, False, ref.f64(s.d_out))
    ref.close(s.out["d_h"], dx, ref.rounded(dx, e, F32))
    ref.close(s.out["d_w"], dw, ref.rounded(dw, e_w, F32))

    # the whole, by automatic differentiation in 64 bits on the CPU with the picks and loads as they are:
    # router logits within 1e-4 of their largest (about 4), so probabilities within 8e-4 of themselves and
    # gradients within a few times that of their largest
    x = torch.from_numpy(h).requires_grad_()
    wt, t = torch.from_numpy(w).requires_grad_(), torch.from_numpy
    n = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * wt
    logits = n @ t(wr).T
    p, inside = torch.softmax(logits, 1), t(seq >= 0)
    balance = (p * t(load)[t(np.maximum(seq, 0)).long()]).sum(1)
    z = torch.logsumexp(logits, 1) ** 2
    N = int(tokens[-1])
    loss = (torch.gather(p, 1, t(idx).long()) * t(ref.f64(s.d_gate))).sum() + \
        dl[0] * bc * balance[inside].sum() / N + dl[1] * zc * z[inside].sum() / N + (x * t(ref.f64(s.d_out))).sum()
    loss.backward()
    for got, want in ((o["d_h"], x.grad.numpy()), (o["d_w"], wt.grad.numpy())):
        assert np.abs(got - want).max() <= 5e-3 * np.abs(want).max()


def _capture(run):
    s = torch.cuda.Stream(device=device())
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    torch.cuda.synchronize()
    return graph


def test_captured_step_replays_match_eager():
    """Two graphs of two steps that share a workspace, replayed in turn between eager work."""
    a, b = Step(seed=1), Step(T=77, seed=2)
    b.ws = a.ws
    want = []
    for s in (a, b):
        s.run()
        want.append(s.results())
    graphs = [_capture(a.run), _capture(b.run)]
    for _ in range(3):
        for s, g, w in zip((a, b), graphs, want):
            s.poison()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            _equal(s.results(), w)
        graphs[0].replay(), graphs[1].replay()       # one after the other on one stream
        torch.cuda.synchronize()
        _equal(a.results(), want[0]), _equal(b.results(), want[1])
        b.run()
        _equal(b.results(), want[1])


def test_two_steps_on_two_streams():
    a, b = Step(T=1500, seed=1), Step(T=1400, seed=2)
    want = []
    for s in (a, b):
        s.run()
        want.append(s.results())
        s.poison()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(device=device()) for _ in range(2)]
    for _ in range(5):
        for s, stream in zip((a, b), streams):
            with torch.cuda.stream(stream):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip((a, b), want):
        _equal(s.results(), w)


def test_experts_on_kept_gate_and_up_values():
    """Dispatch, gate and up products, SwiGLU with its input kept, down product: the experts of
    moe_expert_ffn_mxfp4 with one more rounding, and the gradient at the kept values, on the grouped rows
    alone."""
    T, H, I, E, N, K = 90, 256, 128, 12, 8, 4
    d, rng = device(), np.random.default_rng(5)
    g = torch.Generator("cuda").manual_seed(7)
    x = torch.randn((T, H), generator=g, device=d).to(BF16)
    w13 = moe.quantize_weights(torch.randn((N, 2 * I, H), generator=g, device=d) * H ** -0.5)
    w2 = moe.quantize_weights(torch.randn((N, H, I), generator=g, device=d) * I ** -0.5)
    idx = torch.from_numpy(np.argsort(rng.random((T, E)), 1)[:, :K].astype(np.int32)).to(d)
    counts = torch.bincount(idx.flatten().long(), minlength=E).to(I32)
    e = lambda *s, dtype=I32: torch.empty(s, dtype=dtype, device=d)                     # noqa: E731
    offsets, row_src, slot_row = e(N + 1), e(T * K), e(T * K)
    moe.moe_permute(x, idx, counts, N, offsets, None, row_src, slot_row)
    rows = T * K
    S = int(offsets[-1])
    assert 0 < S < rows
    full = lambda c: torch.full((rows, c), 5.0, dtype=BF16, device=d)                   # noqa: E731
    ws = e(moe.moe_expert_ffn_mxfp4_workspace_bytes(rows, N, I), dtype=U8)
    gu, hh, y, want, d_hh = full(2 * I), full(I), full(H), full(H), full(I)
    kept, n_rows = moe.alloc_checkpoint((rows, 2 * I)), offsets[N:]
    d_gu, h2 = full(2 * I), full(I)
    d_hh.copy_(torch.randn((rows, I), generator=g, device=d))

    def run():
        moe.moe_grouped_gemm_mxfp4(x, None, offsets, *w13, gu, ws, row_src=row_src, K=K)
        moe.moe_swiglu(gu, hh, n_rows, kept)
        moe.moe_grouped_gemm_mxfp4(hh, None, offsets, *w2, y, ws)
        moe.moe_swiglu_backward(d_hh, kept, d_gu, h2, n_rows)

    run()
    h, e_h = ref.swiglu(ref.f64(gu[:S]))
    ref.close(hh[:S], h, ref.rounded(h, e_h, BF16))
    codes, scales = ref.mx8_quantize(ref.f64(gu[:S]))
    assert np.array_equal(kept.codes[:S].cpu().numpy(), codes)
    v = ref.mx8_values(codes, scales)
    dw, e_d = ref.swiglu_backward(ref.f64(d_hh[:S]), v)
    ref.close(d_gu[:S], dw, ref.rounded(dw, e_d, BF16))
    h, e_h = ref.swiglu(v)
    ref.close(h2[:S], h, ref.rounded(h, e_h, BF16))
    for t in (hh, d_gu, h2, y):
        assert (t[S:] == 5).all()
    moe.moe_expert_ffn_mxfp4(x, None, K, row_src, offsets, *w13, *w2, want, ws)
    # gate and up values rounded to bf16 in between: 2^-8 of each, twice in their product
    dev = (y[:S].float() - want[:S].float()).norm() / want[:S].float().norm()
    assert dev < 4 * ref.EPS_BF16
    first = [t.clone() for t in (hh, kept.codes, kept.scales, y, d_gu, h2)]
    graph = _capture(run)
    for _ in range(3):
        for t in (gu, hh, y, d_gu, h2):
            t.fill_(5.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((hh, kept.codes, kept.scales, y, d_gu, h2), first):
            assert torch.equal(a[:S], b[:S])
