"""Calls that make their own workspace, on a stream that is not the current one."""
import numpy as np
import pytest
import torch

import _kv4
import expert_routing_moe_gb300 as moe
from _gpu import DEV

pytestmark = pytest.mark.gpu


def test_the_workspace_belongs_to_the_call_s_stream():
    """It is cleared on the stream that uses it, whatever the current stream is busy with."""
    c = _kv4.Cache(np.random.default_rng(1), [4000], 1, 128)
    t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    cache = moe.Kv4Cache(t(c.bytes), t(c.table), torch.tensor([4000], dtype=torch.int32, device=DEV), 128, t(c.k_scale), t(c.v_scale))
    q = torch.randn(1, 8, 128, device=DEV).bfloat16()
    starts = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    want, got = torch.empty_like(q), torch.full_like(q, float("nan"))
    n = moe.attention_kv4_workspace(1, 8, 1, 128)
    moe.moe_attention_kv4(q, cache, starts, want, 0.1, max_new=1, workspace=torch.zeros(n, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    junk = torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV)   # what the allocator will hand out again
    del junk
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    moe.moe_attention_kv4(q, cache, starts, got, 0.1, max_new=1, stream=other)
    other.synchronize()
    assert torch.equal(got, want)
    torch.cuda.synchronize()
