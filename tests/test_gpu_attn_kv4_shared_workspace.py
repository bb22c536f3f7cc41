"""One zero-filled workspace serves attention calls of any sizes in turn."""
import numpy as np
import pytest
import torch

import _kv4
import expert_routing_moe_gb300 as moe
from _gpu import DEV, assert_status_ok, status_tensor

pytestmark = pytest.mark.gpu


class Call:
    """An attention call with its inputs, and what it gives with a workspace of its own."""

    def __init__(self, seed, D, lengths, new, n_q, n_kv):
        rng = np.random.default_rng(seed)
        t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
        c = _kv4.Cache(rng, lengths, n_kv, D)
        self.cache = moe.Kv4Cache(t(c.bytes), t(c.table), torch.tensor(lengths, dtype=torch.int32, device=DEV), D, t(c.k_scale), t(c.v_scale))
        self.starts = t(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
        self.q = t(rng.normal(size=(sum(new), n_q, D))).bfloat16()
        self.max_new, self.bytes = max(new), moe.attention_kv4_workspace(sum(new), n_q, n_kv, D)
        self.want = self.run(torch.zeros(self.bytes, dtype=torch.uint8, device=DEV))

    def run(self, ws):
        out = torch.full_like(self.q, float("nan"))
        lse = torch.full(self.q.shape[:2], float("nan"), device=DEV)
        st = status_tensor()
        moe.moe_attention_kv4(self.q, self.cache, self.starts, out, 0.1, max_new=self.max_new, lse=lse, workspace=ws, st=st)
        torch.cuda.synchronize()
        assert_status_ok(st)
        return out, lse


def test_head_sizes_and_kernels_in_turn():
    """Prompts whose rows are cut across CTAs, of both head sizes, and 16-row streaming tiles whose pieces lie all over the buffer."""
    prompt = {D: Call(D, D, [4000], [40], 8, 1) for D in (64, 128)}
    stream = {D: Call(D + 1, D, [3300, 3200, 3299, 3100, 3000, 3298], [2] * 6, 32, 4) for D in (64, 128)}
    ws = torch.zeros(max(c.bytes for c in [*prompt.values(), *stream.values()]), dtype=torch.uint8, device=DEV)
    order = [prompt[64], stream[128], prompt[64], prompt[128], prompt[64], prompt[128], stream[64], prompt[128], stream[128], stream[64]]
    for i, c in enumerate(order):
        assert not torch.isnan(c.want[0]).any()
        got = c.run(ws)
        assert torch.equal(got[0], c.want[0]) and torch.equal(got[1], c.want[1]), "call %d" % i
