"""Packing a pool whose tables name pages that are not in use."""
import numpy as np
import pytest
import torch

import expert_routing_moe_gb300 as moe
from test_gpu_kv4_pages import PAGE, Book, Gpu

pytestmark = pytest.mark.gpu


def test_an_entry_that_names_a_free_page_is_reported_and_stays():
    rng = np.random.default_rng(1)
    b = Book(2, 3, 300, 1, PAGE * 72, rng)
    b.table[0, 0], b.ref[299], b.len[0] = 299, 1, 10
    g = Gpu(b, 64, 1)
    moe.moe_kv4_compact(g.pool, None, g.ws, g.st)      # 299 goes to 0
    b.compact()
    g.same(b)
    assert g.st.tolist() == [0, 0]
    g.table[1, 0] = b.table[1, 0] = 299                # free now
    g.table[1, 1] = b.table[1, 1] = 300                # and no page at all
    moe.moe_kv4_compact(g.pool, None, g.ws, g.st)
    b.compact()
    g.same(b)
    assert g.st.tolist()[0] == 3 and g.st.tolist()[1] in (299, 300)
