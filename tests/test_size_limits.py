"""The largest sizes that the headers allow are not refused, and the next ones are (on the host: the
pointers are off their alignment, so that a call whose sizes pass ends at that check)."""
import ctypes

import pytest

import sparse_moe_layer_02_amd as moe

SHAPE, ALIGN = 2, 4
P = ctypes.c_void_p
FAKE, OFF = P(0x10000), P(0x10002)      # never dereferenced


@pytest.mark.parametrize("cols", [32, 96, 160, 2048, 6144, 12320, 1 << 20, (1 << 31) - 32])
def test_mxfp8_rows(cols):
    lib = moe.lib()
    most = ((1 << 34) - 1) // cols
    for rows, want in ((most, ALIGN), (most + 1, SHAPE)):
        assert lib.moe_mxfp8_quantize(OFF, 1, rows, cols, None, FAKE, FAKE, None) == want, rows
        assert lib.moe_mxfp8_dequantize(FAKE, FAKE, 0, rows, cols, OFF, None) == want, rows


@pytest.mark.parametrize("I,kept", [(8, False), (24, False), (32, True), (96, True), (2080, True), (1 << 20, True),
                                    ((1 << 30) - 32, True)])
def test_swiglu_rows(I, kept):
    lib = moe.lib()
    most = ((1 << 34) - 1) // (2 * I)
    s = FAKE if kept else None
    for rows, want in ((most, ALIGN), (most + 1, SHAPE)):
        assert lib.moe_swiglu(OFF, 1, rows, I, None, FAKE, s, s, None) == want, rows
        assert lib.moe_swiglu_backward(OFF, FAKE, s, 1, rows, I, None, FAKE, None, None) == want, rows


@pytest.mark.parametrize("cols", [32, 96, 160, 2048, 6144, 12320, 1 << 20, (1 << 31) - 32])
def test_mxfp4_rows(cols):
    lib = moe.lib()
    most = ((1 << 34) - 1) // cols
    for rows, want in ((most, ALIGN), (most + 1, SHAPE)):
        assert lib.moe_mxfp4_quantize(OFF, 1, rows, cols, None, FAKE, FAKE, None) == want, rows
        assert lib.moe_mxfp4_dequantize(FAKE, FAKE, 0, rows, cols, OFF, None) == want, rows


def test_most_sequences_and_experts():
    f, F = moe.lib().moe_balance_loss, ctypes.c_float
    need = moe.lib().moe_balance_loss_workspace_bytes(64, 1024, 65536)
    # logits, idx, seq, n_seq, group, T, E, K, bc, zc, counts, tokens, load, losses, ws, bytes
    for n_seq, E, want in ((65536, 1024, ALIGN), (65537, 1024, SHAPE), (65536, 1025, SHAPE)):
        assert f(OFF, FAKE, FAKE, n_seq, FAKE, 64, E, 4, F(1.0), F(0.0), FAKE, FAKE, FAKE, FAKE, FAKE, need, None) == want
