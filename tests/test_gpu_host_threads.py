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
