"""One workspace serves pools of different sizes in turn."""
import numpy as np
import pytest
import torch

import expert_routing_moe_gb300 as moe
from _gpu import DEV
from test_gpu_kv4_pages import PAGE, Book, Gpu, _filled, _vec

pytestmark = pytest.mark.gpu


def test_pools_of_two_sizes_in_turn():
    rng = np.random.default_rng(1)
    big = Book(1, 1, 300, 1, PAGE * 72, rng)
    big.ref[150:] = 1                                   # held by their caller
    small = _filled([100, 0, 0], 4, 40, rng)
    small.assign(np.array([0, 0, 0]))
    g, h = Gpu(big, 64, 1), Gpu(small, 64, 1)
    ws = torch.zeros(moe.kv4_pool_workspace(g.pool), dtype=torch.uint8, device=DEV)
    for _ in range(3):
        moe.moe_kv4_compact(g.pool, None, ws, g.st)     # a list of 150 pages
        big.compact()
        g.same(big)
        add = np.array([1, 1, 1])
        moe.moe_kv4_reserve(h.pool, _vec(add), ws, h.st)   # two copy the page they share, the last keeps it
        assert small.reserve(add) == 0
        h.same(small)
        parent = np.array([1, 1, 1])
        moe.moe_kv4_assign(h.pool, _vec(parent), h.st)
        small.assign(parent)
        for b, d in ((big, g),):                        # the packed pages move back up
            b.ref[:] = np.roll(b.ref, 150)
            d.ref.copy_(torch.from_numpy(b.ref))
    assert g.st.tolist() == [0, 0] and h.st.tolist() == [0, 0]
