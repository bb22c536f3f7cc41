"""A token whose position is outside the table: reported, and nothing of it written."""
import numpy as np
import pytest
import torch

import _kv4
import expert_routing_moe_gb300 as moe
from _gpu import DEV, assert_status_ok, status_tensor

pytestmark = pytest.mark.gpu
N_POS = 300


def _run(x, n_q, n_kv, D, rope, cache, starts):
    q = torch.full((x.shape[0], n_q, D), 7.0, dtype=x.dtype, device=DEV)
    k = torch.full((x.shape[0], n_kv, D), 7.0, dtype=x.dtype, device=DEV)
    w = torch.linspace(0.5, 1.5, D, device=DEV)
    st = status_tensor()
    moe.moe_qk_norm_rope(x, n_q, n_kv, q, k, w, w, rope=rope, cache=cache, q_start=starts, st=st)
    torch.cuda.synchronize()
    return q, k, st


def _expect(before, full, c, D, bad):
    """`full`'s bytes, but of the tokens `bad` [(sequence, place)] those of `before`."""
    out = full.copy()
    pkc, pks, pvc, pvs = _kv4.places(D)
    for s, place in bad:
        p, tok = c.table[s, place // 64], place % 64
        mask = np.zeros(full.shape[-1], np.uint8)
        mask[pkc[tok]] = mask[pks[tok]] = mask[pvs[tok]] = 0xFF
        mask[pvc[tok]] = 0xF0 if tok % 2 else 0x0F
        out[p] = (out[p] & ~mask) | (before[p] & mask)
    return out


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("axes,pairs", [(0, False), (1, True), (3, False), (3, True)])
@pytest.mark.parametrize("D,rot,dtype", [(128, 128, torch.bfloat16), (64, 32, torch.float32), (128, 64, torch.bfloat16)])
def test_nothing_of_the_token_is_written(D, rot, dtype, axes, pairs, many):
    rng = np.random.default_rng(D + rot + axes)
    lengths, new = ([201, 66, 40], [180, 66, 3]) if not many else ([264, 290, 64], [233, 290, 41])
    n_kv, n_q = 2, 3 if not many else 40
    T = sum(new)
    starts = np.concatenate([[0], np.cumsum(new)])
    c = _kv4.Cache(rng, lengths, n_kv, D)
    t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    cache = moe.Kv4Cache(t(c.bytes), t(c.table), torch.tensor(lengths, dtype=torch.int32, device=DEV), D, t(c.k_scale), t(c.v_scale))
    x = t(rng.normal(size=(T, (n_q + 2 * n_kv) * D))).to(dtype)
    qs = t(starts.astype(np.int32))
    table = t(rng.normal(size=(N_POS, rot // 2, 2)).astype(np.float32))
    axis = t((np.arange(rot // 2) * 3 // (rot // 2)).astype(np.uint8)) if axes == 3 else None
    place = np.concatenate([np.arange(l - n, l) for l, n in zip(lengths, new)])
    seq = np.repeat(np.arange(3), new)
    pos = rng.integers(0, N_POS, (max(axes, 1), T)).astype(np.int32)
    if axes == 0:                                       # places as positions, and a table that ends early
        pos[0] = place
    good = moe.Rope(table, t(pos), axis, pairs=pairs)
    q0, k0, st = _run(x, n_q, n_kv, D, good, cache, qs)
    assert_status_ok(st)
    full = cache.tensors[0].cpu().numpy()
    if axes == 0:
        cut = 61
        bad = place >= cut
        rope = moe.Rope(table[:cut].contiguous(), None, None, pairs=pairs)
    else:
        bad = rng.random(T) < 0.3
        bad[[0, T - 1]] = True
        bad[starts[1]:starts[1] + 4] = [False, True, True, False]
        worse = pos.copy()
        worse[rng.integers(0, axes, T)[bad], np.nonzero(bad)[0]] = rng.choice([-1, N_POS, 2 ** 31 - 1, -2 ** 31], int(bad.sum()))
        rope = moe.Rope(table, t(worse), axis, pairs=pairs)
    cache.tensors[0].copy_(t(c.bytes))
    q, k, st = _run(x, n_q, n_kv, D, rope, cache, qs)
    assert st.tolist()[0] == 3
    b = t(bad)
    assert torch.equal(q[~b], q0[~b]) and torch.equal(k[~b], k0[~b]) and (q[b] == 7).all() and (k[b] == 7).all()
    # (a last token at an even place clears the half byte behind it, which belongs to no token, when it is written)
    behind = [(s, l) for s, l in enumerate(lengths) if l % 2 and bad[starts[s + 1] - 1]]
    want = _expect(c.bytes, full, c, D, [(s, p) for s, p, n in zip(seq, place, bad) if n] + behind)
    assert np.array_equal(cache.tensors[0].cpu().numpy(), want)


def test_without_a_cache():
    T, D = 50, 64
    x = torch.randn(T, 4 * D, device=DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)[None].clone()
    table = torch.randn(T, D // 2, 2, device=DEV)
    q0, k0, st = _run(x, 2, 1, D, moe.Rope(table, pos), None, None)
    assert_status_ok(st)
    pos[0, 17] = T
    q, k, st = _run(x, 2, 1, D, moe.Rope(table, pos), None, None)
    assert st.tolist() == [3, T] and (q[17] == 7).all() and (k[17] == 7).all()
    q[17], k[17] = q0[17], k0[17]
    assert torch.equal(q, q0) and torch.equal(k, k0)


def test_an_axis_without_positions():
    T, D = 5, 64
    x = torch.randn(T, 4 * D, device=DEV)
    pos = torch.zeros(1, T, dtype=torch.int32, device=DEV)
    axis = torch.zeros(D // 2, dtype=torch.uint8, device=DEV)
    axis[-1] = 1
    q, k, st = _run(x, 2, 1, D, moe.Rope(torch.randn(9, D // 2, 2, device=DEV), pos, axis), None, None)
    assert st.tolist() == [3, -1] and (q == 7).all() and (k == 7).all()
