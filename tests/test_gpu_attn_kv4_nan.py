"""A query that is not a number gives a row that is not one, in `out` and in `lse`, wherever its pieces are joined."""
import numpy as np
import pytest
import torch

import _kv4
import expert_routing_moe_gb300 as moe
from _gpu import DEV, assert_status_ok, status_tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_q,n_kv,new", [(16, 16, 512), (16, 16, 1), (8, 1, 512)])
@pytest.mark.parametrize("window", [0, 700, 900])
def test_out_and_lse_agree(n_q, n_kv, new, window):
    """Items of prompts are cut where their rows' windows lie on one side of the cut."""
    rng = np.random.default_rng(window + new)
    D, lengths = 64, [1500, 1460, 1400, 1303]
    t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    c = _kv4.Cache(rng, lengths, n_kv, D)
    cache = moe.Kv4Cache(t(c.bytes), t(c.table), torch.tensor(lengths, dtype=torch.int32, device=DEV), D, t(c.k_scale), t(c.v_scale))
    T = 4 * new
    q = torch.randn(T, n_q, D, device=DEV).bfloat16()
    rows = torch.arange(T, device=DEV) % 5 == 0
    q[rows, :, 3] = float("nan")
    out, lse, st = torch.zeros_like(q), torch.zeros(T, n_q, device=DEV), status_tensor()
    moe.moe_attention_kv4(q, cache, torch.arange(5, dtype=torch.int32, device=DEV) * new, out, 0.1, max_new=new, window=window, lse=lse, st=st)
    torch.cuda.synchronize()
    assert_status_ok(st)
    assert torch.isnan(out[rows]).all() and torch.isnan(lse[rows]).all()
    assert torch.isfinite(out[~rows]).all() and torch.isfinite(lse[~rows]).all()
