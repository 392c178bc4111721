"""The entry points of include/moe_mi355x_block.h on the host: exported as
declared, and bad arguments refused with status codes before any HIP call."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import sparse_moe_layer_02_amd as moe
from _mxfp4 import E2M1, quantize, values

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_mi355x_block.h")
OK, NULL, SHAPE, DTYPE, ALIGN, WS = 0, 1, 2, 3, 4, 5
P, F = ctypes.c_void_p, ctypes.c_float
FAKE = P(0x10000)        # never dereferenced: validation fails first


def _changed(f, args, at, value):
    a = list(args)
    a[at] = value
    return f(*a)


def test_library_exports_every_declared_symbol():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(moe_\w+)\s*\(", text))
    assert names == set(moe.block.SIGS) and not names & set(moe._SIGS)
    for n in names:
        assert hasattr(moe.lib(), n), n


def test_conversion_refusals():
    q, d = moe.lib().moe_mxfp4_quantize, moe.lib().moe_mxfp4_dequantize
    args = [FAKE, 1, 4, 64, None, FAKE, FAKE, None]
    for at in (0, 5, 6):
        assert _changed(q, args, at, None) == NULL
    assert _changed(q, args, 1, 2) == DTYPE
    for at, v in ((2, 0), (2, -1), (3, 0), (3, 48), (3, 31), (2, 1 << 29)):
        assert _changed(q, args, at, v) == SHAPE, (at, v)
    for at, p in ((0, 0x10008), (5, 0x10008), (6, 0x10002), (4, 0x10002)):
        assert _changed(q, args, at, P(p)) == ALIGN, at
    args = [FAKE, FAKE, 0, 4, 64, FAKE, None]
    for at in (0, 1, 5):
        assert _changed(d, args, at, None) == NULL
    assert _changed(d, args, 2, -1) == DTYPE
    for at, v in ((3, 0), (4, 16), (4, -32)):
        assert _changed(d, args, at, v) == SHAPE
    for at, p in ((0, 0x10004), (1, 0x10001), (5, 0x10008)):
        assert _changed(d, args, at, P(p)) == ALIGN


def test_product_refusals():
    lib = moe.lib()
    f, need = lib.moe_grouped_gemm_mxfp4, lib.moe_grouped_gemm_mxfp4_workspace_bytes(300, 8)
    assert need >= 256 and lib.moe_grouped_gemm_mxfp4_workspace_bytes(0, 8) == 0
    assert lib.moe_grouped_gemm_mxfp4_workspace_bytes(300, 5000) == 0
    # a, a_scales, row_src, T, K, offsets, rows_cap, E, D, N, w, w_scales, swiglu, dtype, out, ws
    args = [FAKE, FAKE, FAKE, 16, 4, FAKE, 300, 8, 256, 64, FAKE, FAKE, 0, 1, FAKE, FAKE, need,
            None]
    for at in (0, 5, 10, 11, 14, 15):
        assert _changed(f, args, at, None) == NULL, at
    assert _changed(f, args, 13, 7) == DTYPE
    for at, v in ((3, 0), (4, 0), (3, 1 << 30), (6, 0), (7, -1), (7, 4097), (8, 0), (8, 192),
                  (9, 0), (9, 72), (9, 1 << 24)):
        assert _changed(f, args, at, v) == SHAPE, (at, v)
    a = list(args); a[6], a[9] = (1 << 31) - 1, 1 << 20; a[8] = 128     # more blocks than a launch takes
    assert f(*a) == SHAPE
    for at in (0, 10, 14):
        assert _changed(f, args, at, P(0x10008)) == ALIGN
    for at in (1, 2, 5, 11):
        assert _changed(f, args, at, P(0x10002)) == ALIGN
    assert _changed(f, args, 15, P(0x10080)) == ALIGN
    assert _changed(f, args, 16, need - 1) == WS
    a = list(args); a[2] = None; a[3] = a[4] = 0; a[16] = 0             # T and K unused without row_src
    assert f(*a) == WS
    a = list(args); a[7] = 0; a[10] = a[11] = None                      # no experts: nothing to do
    assert f(*a) == OK


def test_expert_ffn_refusals():
    lib = moe.lib()
    f, need = lib.moe_expert_ffn_mxfp4, lib.moe_expert_ffn_mxfp4_workspace_bytes(64, 8, 256)
    assert need > 64 * 256 * 2 and lib.moe_expert_ffn_mxfp4_workspace_bytes(64, 8, 0) == 0
    # x, x_scales, T, K, row_src, offsets, rows_cap, n_ffn, H, I, w13, s, w2, s, y, ws, bytes
    args = [FAKE, None, 16, 4, FAKE, FAKE, 64, 8, 512, 256, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
            need, None]
    for at in (0, 4, 5, 10, 11, 12, 13, 14, 15):
        assert _changed(f, args, at, None) == NULL, at
    for at, v in ((2, 0), (3, 0), (6, 0), (7, 5000), (8, 64), (8, 520), (9, 64), (9, 0),
                  (9, 1 << 30), (9, -128)):
        assert _changed(f, args, at, v) == SHAPE, (at, v)
    for at in (0, 10, 12, 14):
        assert _changed(f, args, at, P(0x10008)) == ALIGN
    for at in (1, 4, 5, 11, 13):
        assert _changed(f, args, at, P(0x10001)) == ALIGN
    assert _changed(f, args, 15, P(0x10010)) == ALIGN
    assert _changed(f, args, 16, need - 1) == WS
    a = list(args); a[7] = 0; a[10] = a[11] = a[12] = a[13] = None
    assert f(*a) == OK


def test_norm_refusals():
    lib = moe.lib()
    f = lib.moe_norm
    args = [FAKE, 1, None, F(1e-5), 8, 256, FAKE, 0, None]
    for at in (0, 6):
        assert _changed(f, args, at, None) == NULL
    for at in (1, 7):
        assert _changed(f, args, at, 2) == DTYPE
    for at, v in ((4, 0), (5, 0), (5, 12), (5, 32776), (3, F(-1.0)), (3, F(float("nan")))):
        assert _changed(f, args, at, v) == SHAPE, (at, v)
    for at in (0, 2, 6):
        assert _changed(f, args, at, P(0x10004)) == ALIGN
    g = lib.moe_norm_residual
    # y, dtype, w_post, eps, gate, kind, scale, residual, dtype, out, w_next, next, T, H
    args = [FAKE, 1, FAKE, F(1e-5), FAKE, 2, F(1.0), FAKE, 0, FAKE, FAKE, FAKE, 8, 256, None]
    for at in (0, 4, 7, 9):
        assert _changed(g, args, at, None) == NULL, at
    for at in (1, 8):
        assert _changed(g, args, at, 9) == DTYPE
    for at, v in ((5, 3), (5, -1), (6, F(float("inf"))), (3, F(-1e-3)), (12, 0), (13, 100)):
        assert _changed(g, args, at, v) == SHAPE, (at, v)
    for at in (0, 2, 4, 7, 9, 10, 11):
        assert _changed(g, args, at, P(0x10008)) == ALIGN, at


def test_binding_refuses_host_tensors():
    x = torch.zeros((4, 64))
    u8 = torch.zeros((4, 32), dtype=torch.uint8)
    with pytest.raises(ValueError):
        moe.moe_mxfp4_quantize(x, u8, torch.zeros((4, 2), dtype=torch.uint8))
    with pytest.raises(ValueError):
        moe.moe_norm(x, None, torch.zeros((4, 64)))
    with pytest.raises(ValueError):
        moe.quantize_weights(torch.zeros((4, 48)))


def test_plain_conversion_on_known_blocks():
    """The tests' own plain form: every code comes back from its value, at any scale."""
    x = np.concatenate([E2M1, -E2M1, E2M1 * 0.999, np.full(8, 5.0)])
    codes, scales = quantize(x[None])
    assert scales.tolist() == [[127]]
    v = values(codes, scales)[0]
    assert np.array_equal(v[:8], E2M1) and np.array_equal(v[8:16], -E2M1)
    assert (v[24:] == 4.0).all()                     # 5 is a tie: to the even code
    for e in (-100, 3, 90):
        c2, s2 = quantize(x[None] * 2.0 ** e)
        assert np.array_equal(c2, codes) and s2[0, 0] == 127 + e
