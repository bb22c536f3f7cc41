"""One key that draws attention among very many that get almost none."""
import math

import numpy as np
import pytest
import torch

import _kv4
import expert_routing_moe_gb300 as moe
from _gpu import DEV, assert_status_ok, status_tensor

pytestmark = pytest.mark.gpu
OTHERS = 100_000     # keys behind the first


@pytest.mark.parametrize("depth", [20.0, 25.2, 26.5, 28.0, 29.6, 31.4])
@pytest.mark.parametrize("D,n_q,new", [(64, 32, 1), (64, 64, 1), (128, 32, 1), (64, 32, 32), (128, 32, 32)])
def test_the_many_keep_their_share(D, n_q, new, depth):
    """The first key scores `depth` powers of two above all others, which alone have values, the largest that there are.
    The contexts name one page over and over, and there are as many of them as warps (or CTAs) that walk one each, so that
    a running maximum holds the first key while all others pass.

    The bound does not grow with the many's share: half a step of the bf16 output; 2^-11 for the probabilities' rounding,
    which all of them share; 2^-11 for 1563 pages' fp32 sums one after the other (up to 2^-23 each) and the exponentials; and
    2^-14 of the largest value for all that is lost far below the maximum."""
    n_kv = 4
    S = 304 if new == 1 else 38
    columns = -(-(OTHERS + 1) // 64)
    length = OTHERS + 1
    kc, ks, vc, vs = np.zeros((64, D), np.uint8), np.zeros((64, D // 16), np.uint8), np.full((64, D), 7, np.uint8), np.full((64, D // 16), 0x7E, np.uint8)
    vc[:, 1::2] |= 8                                     # -2688
    pages = np.zeros((2, n_kv, 64 * (D + D // 8)), np.uint8)
    for h in range(n_kv):
        _kv4.write_page(pages[1, h], D, kc, ks, vc, vs, 64)
    kc, ks, vc, vs = kc.copy(), ks.copy(), vc.copy(), vs.copy()
    kc[0, 0], ks[0, 0] = 7, 0x38                         # 6 * 1
    vc[0] = 0
    for h in range(n_kv):
        _kv4.write_page(pages[0, h], D, kc, ks, vc, vs, 64)
    table = torch.ones(S, columns, dtype=torch.int32, device=DEV)
    table[:, 0] = 0
    cache = moe.Kv4Cache(torch.from_numpy(pages).to(DEV), table, torch.full((S,), length, dtype=torch.int32, device=DEV), D)
    q = torch.zeros(S * new, n_q, D, device=DEV, dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    q[:, :, 1] = torch.randn(S * new, n_q, device=DEV)   # the keys have nothing there
    out, lse, st = torch.full_like(q, float("nan")), torch.zeros(S * new, n_q, device=DEV), status_tensor()
    moe.moe_attention_kv4(q, cache, torch.arange(S + 1, dtype=torch.int32, device=DEV) * new, out, depth * math.log(2) / 6, max_new=new, lse=lse, st=st)
    torch.cuda.synchronize()
    assert_status_ok(st)
    n = (length - new + torch.arange(new, dtype=torch.float64, device=DEV)).repeat(S)[:, None]    # keys behind the first that a row sees
    total = 1 + n * 2.0 ** -depth
    want = (2688 * n * 2.0 ** -depth / total)[:, :, None]
    sign = torch.where(torch.arange(D, device=DEV) % 2 == 0, 1.0, -1.0)
    err = (out.double() * sign - want).abs()
    tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -11) * want + 2.0 ** -14 * 2688
    assert (err <= tol).all(), "%.4g of the bound, out %.6g for %.6g" % (float((err / tol).max()), float(out[0, 0, 0]), float(want[0, 0, 0]))
    z = depth * math.log(2) + total.log()
    # roundings of the score's factors, and 1563 pages' sums added one after the other, each off by up to 2^-24
    assert ((lse.double() - z).abs() <= 2.0 ** -20 * z + 2.0 ** -13).all()
