"""The norms of more rows than one dimension of a launch takes threads for."""
import pytest
import torch

import sparse_moe_layer_02_amd as moe
from _parity import device

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def _rows(T, H, value):
    return torch.full((T, H), value, dtype=BF16, device=device())


@pytest.mark.parametrize("T,H", [((1 << 28) + 5, 8), ((1 << 25) + 3, 520)])
def test_norms_of_very_many_rows(T, H):
    """Rows of 2s become rows of 1s (eps too small for bf16 to see), and the last rows, a value of
    their own each, are where they belong.  2^28 rows of one wave, and 2^25 of two, are 2^32 threads."""
    print(f"\n[case] norms of {T} x {H}", flush=True)
    x = _rows(T, H, 2.0)
    x[-4:] = 0
    for i in range(1, 5):
        x[-i, i] = 3.0                       # norm: 3 / sqrt(9 / H) at one place
    moe.moe_norm(x, None, x, 1e-9)
    assert (x[:-4] == 1).all()
    want = torch.zeros((4, H), dtype=torch.float64)
    for i in range(1, 5):
        want[4 - i, i] = H ** 0.5
    # one rounding to bf16, and a few of fp32
    assert ((x[-4:].double().cpu() - want).abs() <= 2.0 ** -8 * 1.001 * want).all()
    last = x[-4:].clone()
    # out = x + 1 * x = 2 x exactly, next = norm of it = norm(x) = x again for the rows of 1s
    out = torch.zeros_like(x)
    nxt = torch.zeros_like(x)
    moe.moe_norm_residual(x, x, out, next_out=nxt, eps=1e-9)
    assert (out[:-4] == 2).all() and torch.equal(out[-4:], 2 * last)
    assert (nxt[:-4] == 1).all()
    assert ((nxt[-4:].double().cpu() - want).abs() <= 2.0 ** -8 * 1.001 * want).all()
