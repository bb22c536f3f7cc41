"""Starts of rows that are no starts: reported, and the other sequences have their results."""
import numpy as np
import pytest
import torch

import _kv4
import expert_routing_moe_gb300 as moe
from _gpu import DEV, status_tensor

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("new", [1, 100])
@pytest.mark.parametrize("bad", [[5, LOW], [5, LOW + 3], [HIGH, LOW], [HIGH, 0], [-1, HIGH], [LOW, 1]])
def test_far_starts(new, bad):
    D, n_q, n_kv = 64, 8, 1
    c = _kv4.Cache(np.random.default_rng(new), [200, 10, 150], n_kv, D)
    t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    cache = moe.Kv4Cache(t(c.bytes), t(c.table), torch.tensor(c.lengths, dtype=torch.int32, device=DEV), D, t(c.k_scale), t(c.v_scale))
    q = torch.randn(new, n_q, D, device=DEV).bfloat16()
    i32 = dict(dtype=torch.int32, device=DEV)
    want, got = torch.empty_like(q), torch.empty_like(q)
    ws = torch.zeros(moe.attention_kv4_workspace(new, n_q, n_kv, D), dtype=torch.uint8, device=DEV)
    st = status_tensor()
    moe.moe_attention_kv4(q, cache, torch.tensor([0, new, new, new], **i32), want, 0.1, max_new=new, workspace=ws, st=st)
    assert st.tolist() == [0, 0]
    # the first sequence keeps its rows; what follows has no rows that are there
    moe.moe_attention_kv4(q, cache, torch.tensor([0, new, *bad], **i32), got, 0.1, max_new=new, workspace=ws, st=st)
    torch.cuda.synchronize()
    assert st.tolist()[0] == 3 and st.tolist()[1] in (1, 2) and torch.equal(got, want)
