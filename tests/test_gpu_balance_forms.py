"""Every form of the routing losses and of the logits' gradient: one block for one sequence of few rows
and the launches beside it, on both sides of the rule between them, and every shape that a row of the
pool is held in, aligned and not."""
import numpy as np
import pytest
import torch

import _train as ref
import sparse_moe_layer_02_amd as moe
from _parity import device
from test_gpu_balance import _case, _check_loss

pytestmark = pytest.mark.gpu
F32, I32 = torch.float32, torch.int32
BC, ZC = float(np.float32(0.02)), float(np.float32(0.003))


def _t(a, dtype=F32):
    return torch.as_tensor(np.ascontiguousarray(a)).to(device()).to(dtype)


def _padded(T, rng):
    """One sequence, with padding among its tokens."""
    return np.where(rng.random(T) < 0.3, rng.choice([-1, 1, 1 << 30, -(1 << 31)], T), 0).astype(np.int32)


# rows of 8, 16, 32 and 64 lanes with four values a load, then with one: a block takes 4096 / lanes rows
ONE = [(24, 511), (24, 512), (24, 513), (64, 255), (64, 256), (64, 257), (96, 127), (96, 128), (96, 129), (200, 64),
       (200, 65), (768, 63), (768, 64), (768, 65), (1024, 64), (5, 512), (5, 513), (13, 256), (13, 257), (30, 128),
       (30, 129), (50, 64), (50, 65), (1001, 64), (1001, 65)]


@pytest.mark.parametrize("E,T", ONE)
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("padded", [False, True])
def test_one_sequence_of_few_rows(E, T, grouped, padded):
    print(f"\n[case] one sequence T={T} E={E} grouped={grouped} padded={padded}", flush=True)
    rng = np.random.default_rng(E + T)
    for K in sorted({1, min(E, 4), min(E, 12)} | ({E} if E <= 64 else set())):
        logits, idx, _ = _case(T, E, K, 1, masked=0.2)
        logits[0] = -np.inf                          # a token with nothing left
        idx[T // 2, 0] = -1
        seq = _padded(T, rng) if padded else None
        group = rng.integers(-1, max(1, E // 3) + 1, E).astype(np.int32) if grouped else None
        _check_loss(logits, idx, seq, 1, group)


def test_all_experts_picked_by_one_block():
    """As many picks as a block ever counts alone: 64 tokens of 1024 picks, more than its turns."""
    logits, idx, _ = _case(64, 1024, 1024, 1)
    _check_loss(logits, idx, None, 1)


ARMS = [5, 8, 13, 16, 20, 30, 32, 33, 50, 64, 100, 101, 128, 200, 201, 256, 400, 401, 512, 700, 701, 768, 769, 1000, 1001, 1024]


@pytest.mark.parametrize("E", ARMS)
@pytest.mark.parametrize("what", ["gates", "losses", "both"])
@pytest.mark.parametrize("off", [0, 1])
def test_gradient_of_any_pool(E, what, off):
    """Gates' and losses' gradients, with masked experts, padding and two sequences; off: everything starts
    4 bytes past its alignment."""
    T, K, n = 37, min(E, 9), 2
    print(f"\n[case] gradient E={E} {what} off={off}", flush=True)
    logits, idx, seq = _case(T, E, K, n, masked=0.2, order="mixed")
    rng = np.random.default_rng(E)
    d_gate = rng.standard_normal((T, K)).astype(np.float32)
    dl = np.array([500.0, -3.0], np.float32)

    def at(a, dtype=F32):
        flat = torch.empty(a.size + 8, dtype=dtype, device=device())
        v = flat[off:off + a.size].view(a.shape)
        v.copy_(_t(a, dtype))
        return v

    kw, rkw = {}, {}
    if what != "gates":
        _, _, _, tokens, load = ref.balance_loss(logits.astype(np.float64), idx, seq, n)
        load = load.astype(np.float32)
        kw.update(tokens=at(tokens, I32), load=at(load), seq=at(seq, I32), d_losses=at(dl), balance_coef=BC, z_coef=ZC)
        rkw.update(tokens=tokens, load=load.astype(np.float64), seq=seq, n_seq=n, dl=dl.astype(np.float64), bc=BC, zc=ZC)
    if what != "losses":
        kw.update(topk_idx=at(idx, I32), d_gate=at(d_gate))
        rkw.update(idx=idx, d_gate=d_gate.astype(np.float64))
    x, d = at(logits), at(np.full((T, E), np.nan, np.float32))
    moe.moe_route_backward(x, d, **kw)
    want, e = ref.route_backward(logits.astype(np.float64), **rkw)
    ref.close(d, want, e + 1e-37)
    assert (d.cpu().numpy()[np.isneginf(logits)] == 0).all()


@pytest.mark.parametrize("E", ARMS)
@pytest.mark.parametrize("n", [1, 3])
def test_losses_of_any_pool(E, n):
    """Past the rows that one block takes: every shape of the sweep, with several rows a group of lanes."""
    T = 2100
    logits, idx, seq = _case(T, E, min(E, 6), n, masked=0.1, order="mixed")
    if n == 1:
        seq = _padded(T, np.random.default_rng(E))
    _check_loss(logits, idx, seq, n)


@pytest.mark.parametrize("T,K,n", [(2730, 12, 1), (2731, 12, 1), (1024, 32, 9), (1025, 32, 9), (16384, 2, 64), (16384, 2, 65),
                                   (16384, 2, 256), (16384, 2, 257), (4096, 8, 1024), (4096, 8, 1025)])
def test_both_sides_of_the_count_in_one_launch(T, K, n):
    """2^15 picks and 2^22 looks at a token's sequence, and the next more of either."""
    logits, idx, seq = _case(T, 48, K, n, order="mixed")
    _check_loss(logits, idx, seq, n)
