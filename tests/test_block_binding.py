"""What the Python calls of the 4-bit experts and the block refuse before anything runs, on the host."""
import pytest
import torch

import sparse_moe_layer_02_amd as moe

BF16, U8 = torch.bfloat16, torch.uint8


@pytest.fixture
def recorded(monkeypatch):
    """Every library call that would be made, as its name; tensors may be of any device."""
    calls = []
    record = lambda name: lambda *a, **k: calls.append(name)                        # noqa: E731
    for name in ("moe_router_logits", "moe_route", "moe_permute", "moe_expert_ffn_gather",
                 "moe_expert_ffn", "moe_expert_ffn_mxfp4", "moe_zero_experts", "moe_combine",
                 "moe_combine_identity"):
        monkeypatch.setattr(moe, name, record(name))
    for name in ("moe_norm", "moe_norm_residual"):
        monkeypatch.setattr(moe.block, name, record(name))
    return calls


def _layer(T=8, H=128, E=6, N=4, I=128, K=2, separate=False):
    t = lambda *s, dtype=BF16: torch.zeros(s, dtype=dtype)                          # noqa: E731
    q = lambda *s: moe.MXFP4(t(*s[:-1], s[-1] // 2, dtype=U8), t(*s[:-1], s[-1] // 32, dtype=U8))  # noqa: E731
    names = ("logits", "topk_idx", "topk_gate", "counts", "status", "offsets", "row_src", "slot_row",
             "y_perm", "ws_ffn", "y")
    buf = dict({n: None for n in names}, x_perm=None, y_acc=t(T, H) if separate else None)
    return (t(T, H), t(E, H), t(E), (t(N, 2 * I, H), t(N, H, I)), (q(N, 2 * I, H), q(N, H, I)), K,
            buf)


@pytest.mark.parametrize("separate", [False, True])
@pytest.mark.parametrize("forward", ["forward", "forward_serial"])
def test_one_expert_weight_in_mxfp4_and_the_other_not(recorded, forward, separate):
    x, w_router, bias, plain, packed, K, buf = _layer(separate=separate)
    f = getattr(moe, forward)
    for w13, w2 in ((packed[0], plain[1]), (plain[0], packed[1])):
        with pytest.raises(TypeError, match="w13 and w2.*MXFP4"):
            f(x, w_router, bias, w13, w2, K, 1.0, buf)
        with pytest.raises(TypeError, match="w13 and w2.*MXFP4"):
            moe.block_forward(x, None, w_router, bias, w13, w2, K, 1.0, buf)
    assert recorded == []                            # refused before anything runs
    for w13, w2 in (plain, packed):
        f(x, w_router, bias, w13, w2, K, 1.0, buf)
    assert recorded.count("moe_expert_ffn_gather") == recorded.count("moe_expert_ffn_mxfp4") == 1
