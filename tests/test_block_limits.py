"""Sizes at which the calls of include/moe_mi355x_block.h end, on the host."""
import ctypes

import sparse_moe_layer_02_amd as moe

OK, SHAPE, WS = 0, 2, 5
FAKE = ctypes.c_void_p(0x10000)        # never dereferenced: the checks fail first


def test_products_end_where_row_addresses_do():
    """Rows of a: up to 2^39 values, counted by T with the dispatch indices and by rows_cap
    without; a workspace of no bytes shows that the sizes were taken."""
    f = moe.lib().moe_grouped_gemm_mxfp4
    D, rows = 4096, (1 << 39) // 4096

    def call(scales, src, T, cap):
        return f(FAKE, scales, src, T, 1, FAKE, cap, 2, D, 16, FAKE, FAKE, 0, 0, FAKE, FAKE, 0,
                 None)

    for scales in (None, FAKE):
        assert call(scales, FAKE, rows, 64) == WS
        assert call(scales, FAKE, rows + 1, 64) == SHAPE
        assert call(scales, None, 0, rows) == WS
        assert call(scales, None, 0, rows + 1) == SHAPE
    g = moe.lib().moe_expert_ffn_mxfp4

    def ffn(T):
        return g(FAKE, None, T, 1, FAKE, FAKE, 64, 2, D, 128, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 0,
                 None)

    assert ffn(rows) == WS and ffn(rows + 1) == SHAPE
