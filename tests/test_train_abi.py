"""The entry points of include/moe_mi355x_train.h on the host: exported as declared, bad arguments
refused with status codes before any HIP call, and what the Python calls refuse."""
import ctypes
import os
import re

import pytest
import torch

import sparse_moe_layer_02_amd as moe

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_mi355x_train.h")
OK, NULL, SHAPE, DTYPE, ALIGN, WS = 0, 1, 2, 3, 4, 5
P, F = ctypes.c_void_p, ctypes.c_float
FAKE = P(0x10000)        # never dereferenced: validation fails first
INF, NAN = F(float("inf")), F(float("nan"))


def _changed(f, args, at, value):
    a = list(args)
    a[at] = value
    return f(*a)


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_\w+)\s*\(", text))
    assert names == set(moe.train.SIGS) and not names & (set(moe._SIGS) | set(moe.block.SIGS))
    for n in names:
        assert hasattr(moe.lib(), n) and hasattr(moe, n), n


def test_balance_refusals():
    lib = moe.lib()
    f, need = lib.moe_balance_loss, lib.moe_balance_loss_workspace_bytes(64, 24, 4)
    assert need >= 16
    for bad in ((0, 24, 4), (64, 0, 4), (64, 1025, 4), (64, 24, 0), (64, 24, 65537)):
        assert lib.moe_balance_loss_workspace_bytes(*bad) == 0, bad
    # logits, idx, seq, n_seq, group, T, E, K, bc, zc, counts, tokens, load, losses, ws, bytes
    args = [FAKE, FAKE, FAKE, 4, FAKE, 64, 24, 4, F(1.0), F(0.0), FAKE, FAKE, FAKE, FAKE, FAKE,
            need, None]
    for at in (0, 1, 10, 11, 12, 13, 14):
        assert _changed(f, args, at, None) == NULL, at
    for at, v in ((2, None), (3, 0), (3, 65537), (5, 0), (5, -1), (5, 1 << 29), (6, 0), (6, 1025),
                  (7, 0), (7, 25), (8, INF), (8, NAN), (9, F(-float("inf")))):
        assert _changed(f, args, at, v) == SHAPE, (at, v)
    for at in (0, 1, 2, 4, 10, 11, 12, 13):
        assert _changed(f, args, at, P(0x10002)) == ALIGN, at
    assert _changed(f, args, 14, P(0x10080)) == ALIGN
    assert _changed(f, args, 15, need - 1) == WS


def test_route_backward_refusals():
    f = moe.lib().moe_route_backward
    # logits, idx, d_gate, seq, n_seq, tokens, load, d_losses, bc, zc, T, E, K, d_logits
    args = [FAKE, FAKE, FAKE, FAKE, 4, FAKE, FAKE, FAKE, F(1.0), F(0.0), 64, 24, 4, FAKE, None]
    for at in (0, 1, 5, 6, 13):
        assert _changed(f, args, at, None) == NULL, at
    a = list(args); a[2] = a[5] = a[6] = None                           # nothing to differentiate
    assert f(*a) == NULL
    for at, v in ((3, None), (4, 0), (10, 0), (10, 1 << 30), (11, 0), (11, 2000), (12, 0), (12, 25),
                  (8, NAN), (9, INF)):
        assert _changed(f, args, at, v) == SHAPE, (at, v)
    for at in (0, 1, 2, 3, 5, 6, 7, 13):
        assert _changed(f, args, at, P(0x10001)) == ALIGN, at
    a = list(args); a[2] = None; a[12] = 0; a[13] = P(0x10001)          # K unused without d_gate
    assert f(*a) == ALIGN


def test_conversion_refusals():
    q, d = moe.lib().moe_mxfp8_quantize, moe.lib().moe_mxfp8_dequantize
    args = [FAKE, 1, 4, 64, None, FAKE, FAKE, None]
    for at in (0, 5, 6):
        assert _changed(q, args, at, None) == NULL
    assert _changed(q, args, 1, 2) == DTYPE
    for at, v in ((2, 0), (2, -1), (3, 0), (3, 48), (3, -32), (2, 1 << 28)):
        assert _changed(q, args, at, v) == SHAPE, (at, v)
    for at, p in ((0, 0x10008), (5, 0x10008), (6, 0x10002), (4, 0x10002)):
        assert _changed(q, args, at, P(p)) == ALIGN, at
    args = [FAKE, FAKE, 0, 4, 64, FAKE, None]
    for at in (0, 1, 5):
        assert _changed(d, args, at, None) == NULL
    assert _changed(d, args, 2, -1) == DTYPE
    for at, v in ((3, 0), (4, 16)):
        assert _changed(d, args, at, v) == SHAPE
    for at, p in ((0, 0x10008), (1, 0x10001), (5, 0x10008)):
        assert _changed(d, args, at, P(p)) == ALIGN


def test_norm_refusals():
    lib = moe.lib()
    f = lib.moe_norm_checkpoint
    # x, dtype, weight, eps, T, H, y, dtype, codes, scales
    args = [FAKE, 1, FAKE, F(1e-5), 8, 256, FAKE, 0, FAKE, FAKE, None]
    for at in (0, 6, 8, 9):
        assert _changed(f, args, at, None) == NULL
    for at in (1, 7):
        assert _changed(f, args, at, 2) == DTYPE
    for at, v in ((4, 0), (5, 0), (5, 40), (5, 32800), (3, F(-1.0)), (3, NAN)):
        assert _changed(f, args, at, v) == SHAPE, (at, v)
    for at, p in ((0, 8), (2, 8), (6, 8), (8, 8), (9, 2)):
        assert _changed(f, args, at, P(0x10000 + p)) == ALIGN, at
    f = lib.moe_layer_norm
    # x, dtype, weight, bias, eps, T, H, y, dtype, codes, scales
    args = [FAKE, 1, FAKE, FAKE, F(1e-5), 8, 256, FAKE, 0, FAKE, FAKE, None]
    for at in (0, 7, 9, 10):
        assert _changed(f, args, at, None) == NULL, at
    for at in (1, 8):
        assert _changed(f, args, at, 5) == DTYPE
    for at, v in ((5, 0), (6, 0), (6, 40), (6, 32800), (4, INF)):
        assert _changed(f, args, at, v) == SHAPE, (at, v)
    for at, p in ((0, 8), (2, 4), (3, 4), (7, 8), (9, 8), (10, 1)):
        assert _changed(f, args, at, P(0x10000 + p)) == ALIGN, at
    a = list(args); a[9] = a[10] = None; a[6] = 12                      # no checkpoint: any multiple of 8
    assert f(*a) == SHAPE
    a[6] = 40; a[7] = P(0x10008)
    assert f(*a) == ALIGN


@pytest.mark.parametrize("mean", [False, True])
def test_norm_backward_refusals(mean):
    lib = moe.lib()
    f = lib.moe_layer_norm_backward if mean else lib.moe_norm_backward
    size = lib.moe_norm_backward_workspace_bytes
    need = size(64, 512)
    assert need >= 2 * 512 * 4
    for bad in ((0, 512), (64, 0), (64, 32776)):
        assert size(*bad) == 0
    # dy, dtype, x, dtype, scales, weight, eps, T, H, d_residual, dx, dtype, dw, (db,) ws, bytes
    args = [FAKE, 1, FAKE, 0, None, FAKE, F(1e-5), 64, 512, FAKE, FAKE, 0, FAKE,
            *([FAKE] if mean else []), FAKE, need, None]
    ws = 13 + mean
    for at in (0, 2, 10, ws):
        assert _changed(f, args, at, None) == NULL, at
    for at in (1, 3, 11):
        assert _changed(f, args, at, 2) == DTYPE, at
    for at, v in ((7, 0), (8, 0), (8, 12), (8, 32776), (6, F(-1e-9)), (6, NAN)):
        assert _changed(f, args, at, v) == SHAPE, (at, v)
    for at in (0, 2, 5, 9, 10, 12, *([13] if mean else [])):
        assert _changed(f, args, at, P(0x10008)) == ALIGN, at
    assert _changed(f, args, ws, P(0x10080)) == ALIGN
    assert _changed(f, args, ws + 1, need - 1) == WS
    a = list(args); a[4] = FAKE; a[3] = 9; a[8] = 40                    # MXFP8: whole blocks, x's dtype unused
    assert f(*a) == SHAPE
    a[8] = 512; a[4] = P(0x10002)
    assert f(*a) == ALIGN
    a = list(args); a[12] = None; a[ws] = None; a[ws + 1] = 0           # no sums: no workspace
    if mean:
        a[13] = None
    a[0] = P(0x10008)
    assert f(*a) == ALIGN


def test_swiglu_refusals():
    f = moe.lib().moe_swiglu
    # gu, dtype, rows, I, n_rows, hh, codes, scales
    args = [FAKE, 1, 64, 256, FAKE, FAKE, FAKE, FAKE, None]
    for at in (0, 5, 6, 7):
        assert _changed(f, args, at, None) == NULL, at
    assert _changed(f, args, 1, 2) == DTYPE
    for at, v in ((2, 0), (3, 0), (3, -32), (3, 24), (3, 1 << 30), (2, 1 << 26)):
        assert _changed(f, args, at, v) == SHAPE, (at, v)
    for at, p in ((0, 8), (4, 2), (5, 8), (6, 8), (7, 1)):
        assert _changed(f, args, at, P(0x10000 + p)) == ALIGN, at
    a = list(args); a[6] = a[7] = None; a[3] = 12
    assert f(*a) == SHAPE
    a[3] = 24; a[5] = P(0x10008)
    assert f(*a) == ALIGN
    f = moe.lib().moe_swiglu_backward
    # d_hh, gu, scales, dtype, rows, I, n_rows, d_gu, hh
    args = [FAKE, FAKE, FAKE, 1, 64, 256, FAKE, FAKE, FAKE, None]
    for at in (0, 1, 7):
        assert _changed(f, args, at, None) == NULL, at
    assert _changed(f, args, 3, -1) == DTYPE
    for at, v in ((4, 0), (5, 0), (5, 24), (5, 1 << 30), (4, 1 << 26)):
        assert _changed(f, args, at, v) == SHAPE, (at, v)
    for at, p in ((0, 8), (1, 8), (2, 1), (6, 2), (7, 8), (8, 8)):
        assert _changed(f, args, at, P(0x10000 + p)) == ALIGN, at


def test_binding_refuses_host_tensors():
    x, i = torch.zeros((4, 64)), torch.zeros((4, 2), dtype=torch.int32)
    kept = moe.alloc_checkpoint((4, 64), "cpu")
    assert kept.shape == (4, 64) and kept.scales.shape == (4, 2)
    for call in (lambda: moe.moe_layer_norm(x, None, None, x),
                 lambda: moe.moe_norm_checkpoint(x, None, x, kept),
                 lambda: moe.moe_norm_backward(x, x, None, x),
                 lambda: moe.moe_layer_norm_backward(x, kept, None, x),
                 lambda: moe.moe_mxfp8_quantize(x, *kept),
                 lambda: moe.moe_mxfp8_dequantize(*kept, x),
                 lambda: moe.moe_swiglu(x, x[:, :32].contiguous()),
                 lambda: moe.moe_swiglu_backward(x[:, :32].contiguous(), kept, x),
                 lambda: moe.moe_route_backward(x, x, i, x[:, :2].contiguous())):
        with pytest.raises(ValueError, match="GPU"):
            call()


@pytest.fixture
def calls(monkeypatch):
    """The binding on tensors without memory; the library's calls are recorded."""
    made = []
    monkeypatch.setattr(moe.train, "_dev", lambda *ts: torch.device("cuda", 0))
    monkeypatch.setattr(moe.train, "_call", lambda name, *a: made.append(name))
    return made


def _m(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="meta")


I32, U8, BF16 = torch.int32, torch.uint8, torch.bfloat16


def test_binding_checks_shapes_and_types(calls):
    T, E, K, n, H = 16, 8, 2, 3, 64
    logits, idx, ws = _m(T, E), _m(T, K, dtype=I32), _m(256, dtype=U8)
    good = dict(logits=logits, topk_idx=idx, counts=_m(n, E, dtype=I32), tokens=_m(n + 1, dtype=I32),
                load=_m(n, E), losses=_m(2), ws=ws, seq=_m(T, dtype=I32), group=_m(E, dtype=I32))
    moe.moe_balance_loss(**good)
    for name, t in dict(logits=_m(T, E, dtype=BF16), topk_idx=_m(T, K), tokens=_m(n, dtype=I32),
                        load=_m(n, E + 1), losses=_m(3), seq=_m(T - 1, dtype=I32),
                        group=_m(E), counts=_m(n, E)).items():
        with pytest.raises((ValueError, TypeError)):
            moe.moe_balance_loss(**{**good, name: t})
    with pytest.raises(ValueError, match="one sequence"):
        moe.moe_balance_loss(**{**good, "seq": None})
    back = dict(logits=logits, d_logits=_m(T, E), topk_idx=idx, d_gate=_m(T, K), load=good["load"],
                tokens=good["tokens"], seq=good["seq"], d_losses=_m(2))
    moe.moe_route_backward(**back)
    moe.moe_route_backward(logits, _m(T, E), idx, _m(T, K))
    for change in (dict(d_gate=_m(T, K + 1)), dict(d_logits=_m(T, E, dtype=BF16)), dict(topk_idx=None),
                   dict(tokens=None), dict(load=None), dict(d_losses=_m(1)), dict(seq=None),
                   dict(seq=_m(T)), dict(d_gate=None, load=None, tokens=None)):
        with pytest.raises((ValueError, TypeError)):
            moe.moe_route_backward(**{**back, **change})
    x, kept = _m(T, H, dtype=BF16), moe.MXFP8(_m(T, H, dtype=U8), _m(T, H // 32, dtype=U8))
    half = moe.MXFP8(_m(T, H // 2, dtype=U8), _m(T, H // 64, dtype=U8))
    moe.moe_layer_norm(x, _m(H), _m(H), _m(T, H), checkpoint=kept)
    moe.moe_norm_checkpoint(x, _m(H), _m(T, H), kept)
    for f in (lambda: moe.moe_layer_norm(x, _m(H + 8), None, x), lambda: moe.moe_layer_norm(x, None, _m(H, dtype=BF16), x),
              lambda: moe.moe_layer_norm(x, None, None, _m(T, H + 8)),
              lambda: moe.moe_layer_norm(x, None, None, x, checkpoint=half),
              lambda: moe.moe_norm_checkpoint(x, None, x, None),
              lambda: moe.moe_norm_checkpoint(x, None, x, moe.MXFP8(kept.codes, half.scales))):
        with pytest.raises((ValueError, TypeError)):
            f()
    for form in (x, kept):
        moe.moe_norm_backward(x, form, _m(H), x, _m(H), ws, d_residual=x)
        moe.moe_layer_norm_backward(x, form, None, _m(T, H), _m(H), _m(H), ws)
    for f in (lambda: moe.moe_norm_backward(x, half, None, x), lambda: moe.moe_norm_backward(x, x, None, _m(T, H + 8)),
              lambda: moe.moe_norm_backward(x, x, None, x, d_residual=_m(T, H)),
              lambda: moe.moe_norm_backward(x, x, None, x, _m(H + 1), ws),
              lambda: moe.moe_layer_norm_backward(x, x, None, x, _m(H), _m(T), ws)):
        with pytest.raises((ValueError, TypeError)):
            f()
    gu, hh = _m(T, H, dtype=BF16), _m(T, H // 2, dtype=BF16)
    moe.moe_swiglu(gu, hh, checkpoint=kept, n_rows=_m(1, dtype=I32))
    moe.moe_swiglu_backward(hh, kept, gu, hh)
    moe.moe_swiglu_backward(hh, gu, gu)
    for f in (lambda: moe.moe_swiglu(gu, gu), lambda: moe.moe_swiglu(gu, _m(T, H // 2)),
              lambda: moe.moe_swiglu(gu, hh, n_rows=_m(1)), lambda: moe.moe_swiglu(gu, hh, checkpoint=half),
              lambda: moe.moe_swiglu_backward(hh, half, gu), lambda: moe.moe_swiglu_backward(hh, gu, hh),
              lambda: moe.moe_swiglu_backward(hh, _m(T, H), gu),
              lambda: moe.moe_swiglu_backward(hh, gu, gu, hh=gu)):
        with pytest.raises((ValueError, TypeError)):
            f()
    with pytest.raises(ValueError):
        moe.alloc_checkpoint((4, 40), "cpu")
    with pytest.raises(ValueError):
        moe.moe_mxfp8_quantize(_m(T, 40), _m(T, 40, dtype=U8), _m(T, 1, dtype=U8))
    big = 1 << 31
    with pytest.raises(ValueError, match="2\\^31"):
        moe.moe_layer_norm(_m(big, 8), None, None, _m(big, 8))
    with pytest.raises(ValueError, match="2\\^31"):
        moe.moe_norm_backward(_m(big, 8), _m(big, 8), None, _m(big, 8))
    assert calls.count("moe_balance_loss") == 1 and calls.count("moe_route_backward") == 2
    assert len(calls) == 12
