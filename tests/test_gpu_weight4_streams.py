"""Weight4.pack on another stream: its memory is not that of a tensor which the current stream still reads."""
import pytest
import torch

import expert_routing_moe_gb300 as moe
from _gpu import DEV

pytestmark = pytest.mark.gpu


def test_packing_leaves_what_the_current_stream_reads():
    N, K = 1024, 1024
    w, side = torch.randn(N, K, device=DEV), torch.cuda.Stream()
    want = moe.Weight4.pack(w)
    a = torch.full((moe.w4_bytes(N, K),), 7, dtype=torch.uint8, device=DEV)
    b = torch.zeros_like(a)
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)             # 0.1 s, after which `a` is read
    b.copy_(a)
    del a
    got = moe.Weight4.pack(w, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert (b == 7).all()
    assert torch.equal(got.tensors[0], want.tensors[0]) and torch.equal(got.tensors[1], want.tensors[1])
