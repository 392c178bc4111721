"""The grouped 4-bit products on tensors past 64 GiB."""
import numpy as np
import pytest
import torch

import sparse_moe_layer_02_amd as moe
from _mxfp4 import product, quantize, spans, values
from _parity import device

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
D, N = 4096, 16
FAR = 48                       # rows of interest at the end of a tensor


def _dev(a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a)).to(device())
    return t if dtype is None else t.to(dtype)


def _far_rows(kind, rng):
    """(rows, scales or None, the last FAR rows' values) of a tensor that passes 64 GiB by FAR + 64
    rows.  The rows at its beginning are zeros, the rest is not written."""
    pitch = 2 * D if kind == "bf16" else D // 2
    rows = (1 << 36) // pitch + FAR + 64
    dev = device()
    x = rng.standard_normal((FAR, D))
    if kind == "bf16":
        a, s = torch.empty((rows, D), dtype=BF16, device=dev), None
        a[:256] = 0
        a[-FAR:] = _dev(x, F32).to(BF16)
        v = a[-FAR:].double().cpu().numpy()
    else:
        c, e = quantize(x)
        a = torch.empty((rows, D // 2), dtype=torch.uint8, device=dev)
        s = torch.empty((rows, D // 32), dtype=torch.uint8, device=dev)
        a[:256], s[:256] = 0, 127
        a[-FAR:], s[-FAR:] = _dev(c), _dev(e)
        v = values(c, e)
    return a, s, v


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "mxfp4"])
def test_rows_past_64_gib(kind, gather):
    """A row's address is kept whole: rows that lie more than 2^36 bytes into their tensor are read
    where they are, through the dispatch indices and without."""
    print(f"\n[case] rows past 64 GiB, {kind}, gather={gather}", flush=True)
    rng = np.random.default_rng(11)
    a, s, v = _far_rows(kind, rng)
    rows, dev = a.shape[0], a.device
    c, e = quantize(rng.standard_normal((2, N, D)) / np.sqrt(D))
    counts = (30, FAR - 30)
    if gather:
        cap, first, off = FAR, 0, spans(counts)
        src = torch.arange(rows - FAR, rows, dtype=torch.int32, device=dev)
    else:
        cap, first, src = rows, rows - FAR, None
        off = (rows - FAR + spans(counts).astype(np.int64)).astype(np.int32)
    y = torch.empty((cap, N), dtype=F32, device=dev)
    work = torch.empty(moe.moe_grouped_gemm_mxfp4_workspace_bytes(cap, 2), dtype=torch.uint8,
                       device=dev)
    moe.moe_grouped_gemm_mxfp4(a, s, _dev(off), _dev(c), _dev(e), y, work, row_src=src, K=1)
    got = y[first:].double().cpu().numpy()
    for i, (lo, hi) in enumerate(((0, 30), (30, FAR))):
        want, bound = product(v[lo:hi], values(c[i], e[i]), False, False)
        d = np.abs(got[lo:hi] - want) - bound
        assert np.isfinite(got[lo:hi]).all() and d.max() <= 0, d.max()
