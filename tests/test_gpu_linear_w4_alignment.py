"""Products of the same numbers have the same bits wherever x's rows start."""
import numpy as np
import pytest
import torch

import expert_routing_moe_gb300 as moe
from _gpu import DEV
from test_gpu_linear_w4 import Weights, _bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K", [
    (3, 700, 1000), (9, 4000, 2048), (12, 20000, 600), (16, 15000, 1500), (20, 2048, 4096), (32, 2048, 4096), (32, 5120, 2048), (48, 1500, 3000), (64, 257, 2000),
    (65, 1027, 200), (65, 1027, 1200), (90, 6000, 700), (130, 2048, 2048), (300, 3000, 1000), (500, 300, 5000), (1000, 1500, 640)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bits_do_not_depend_on_where_rows_start(T, N, K, dtype):
    rng = np.random.default_rng(T + N + K)
    w = Weights(rng, N, K)
    x = _bf16(rng.normal(size=(T, K)))
    want = None
    for shift, ld in ((0, -(-K // 8) * 8), (1, -(-K // 8) * 8), (8, -(-K // 8) * 8 + 24), (0, K + 1 + K % 2), (3, K + 2)):
        buf = torch.full((T * ld + 16,), float("nan"), dtype=torch.bfloat16, device=DEV)
        on = buf[shift:shift + T * ld].view(T, ld)[:, :K]
        on.copy_(x)
        y = torch.empty(T, N, dtype=dtype, device=DEV)
        moe.moe_linear_w4(on, w.w, y)
        if want is None:
            want = y
        assert torch.equal(y, want)
