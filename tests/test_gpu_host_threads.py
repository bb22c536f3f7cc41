"""Calls of several host threads whose kernel takes different amounts of shared memory: no thread's setting makes another's
launch fail."""
import threading

import pytest
import torch

import expert_routing_moe_gb300 as moe
from _gpu import DEV

pytestmark = pytest.mark.gpu


def _at_once(calls, turns):
    """Each call `turns` times in a thread of its own; what went wrong."""
    wrong, start = [], threading.Barrier(len(calls))

    def work(call):
        start.wait()
        try:
            for i in range(turns):
                call()
                if i % 100 == 99:          # (a thread whose stream is full waits within its launch)
                    torch.cuda.synchronize()
        except Exception as e:
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return wrong


@pytest.mark.parametrize("T,widths", [(1, (2048, 4096, 8000)), (8, (2048, 3000, 4096, 8000))])
def test_heads_of_other_widths(T, widths):
    """Many rows: x lies in shared memory, whose size goes by the number of columns."""
    calls, outs = [], []
    for K in widths:
        w = moe.Weight4.pack(torch.randn(14720, K, device=DEV))
        x, want, y = torch.randn(T, K, device=DEV).bfloat16(), torch.empty(T, 14720, device=DEV), torch.empty(T, 14720, device=DEV)
        moe.moe_linear_w4(x, w, want)
        s = torch.cuda.Stream()
        outs.append((want, y))
        calls.append(lambda x=x, w=w, y=y, s=s: moe.moe_linear_w4(x, w, y, stream=s))
    torch.cuda.synchronize()
    assert _at_once(calls, 20000) == []
    assert all(torch.equal(want, y) for want, y in outs)


def test_forks_of_few_and_of_many_sequences():
    """A fork's tables pass through shared memory, whose size goes by the number of sequences."""
    calls, pools = [], []
    for S in (3, 2500):
        pages = moe.KvPages(1, S, 1, 64, S, 64, DEV)
        pages.reserve(torch.full((S,), 5, dtype=torch.int32, device=DEV))
        parent, s = torch.arange(S, dtype=torch.int32, device=DEV).flip(0).contiguous(), torch.cuda.Stream()
        pools.append((pages, pages.page_table.clone()))
        calls.append(lambda pages=pages, parent=parent, s=s: moe.moe_kv4_assign(pages.pool, parent, pages.status, stream=s))
    torch.cuda.synchronize()
    assert _at_once(calls, 20000) == []
    # (an even number of turns)
    assert all(torch.equal(pages.page_table, table) and pages.device_status()[0] == 0 for pages, table in pools)
