"""A layer's FFN workspace serves every batch up to its max_tokens."""
import pytest
import torch

import __graft_entry__ as entry
from expert_routing_moe_gb300 import MoELayer, _abi as abi


@pytest.mark.parametrize("max_tokens", [1, 64, 65, 100, 500, 2000])
def test_workspace_covers_smaller_batches(max_tokens):
    entry.build()
    N, H, I, k = 128, 128, 128, 8
    w = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    layer = MoELayer(torch.zeros(N, H), w(N, I, H), w(N, I, H), w(N, H, I), k=k, max_tokens=max_tokens)
    for T in {t for t in (1, 16, 17, 32, 33, 64, 65, 90, 500, 2000) if t <= max_tokens}:
        need = abi.workspace_size(abi.MOE_OP_FFN, T, H, I, N, k, k, False, abi.MOE_DTYPE_BF16)
        assert layer.ws_ffn.numel() >= need, T
