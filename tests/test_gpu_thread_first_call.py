"""The first call that a host thread makes, where the entry point describes its operands to TMA before it launches anything."""
import threading

import numpy as np
import pytest
import torch

import expert_routing_moe_gb300 as moe
from _gpu import DEV, dev
from test_gpu_kv4_weigh import Case
from test_gpu_linear_w4 import Weights

pytestmark = pytest.mark.gpu


def _product():
    w, x = Weights(np.random.default_rng(0), 300, 256), torch.randn(70, 256, device=DEV).bfloat16()
    return lambda y, stream: moe.moe_linear_w4(x, w.w, y, stream=stream), torch.zeros(70, 300, device=DEV)


def _weigh():
    c = Case(1, [500, 90], [200, 3], 8, 2, 64)
    q_start, lse = dev(c.q_start), dev(c.lse)
    return lambda score, stream: moe.moe_kv4_weigh(c.q_dev, c.cache, q_start, lse, score, c.scale, c.max_new, workspace=c.ws, stream=stream), torch.zeros_like(dev(c.score))


def _route():
    T, H, N, k = 4096, 256, 64, 4
    x, w = torch.randn(T, H, device=DEV).bfloat16(), torch.randn(N, H, device=DEV)
    ids, gates = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
    return lambda logits, stream: moe.moe_route(x, w, logits, ids, gates, k, stream=stream), torch.zeros(T, N, device=DEV)


@pytest.mark.parametrize("make", [_product, _weigh, _route])
@pytest.mark.parametrize("side", [False, True])
def test_first_call_of_a_thread(make, side):
    call, out = make()
    stream = torch.cuda.Stream() if side else None
    wrong, got = [], out.clone()
    torch.cuda.synchronize()

    def work():
        try:
            call(got, stream)
        except Exception as e:
            wrong.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    call(out, None)
    assert wrong == [] and torch.equal(got, out)
