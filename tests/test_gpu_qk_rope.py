"""q/k norms, rotary positions and the append to the 4-bit cache on the GPU
against the numpy reference."""
import numpy as np
import pytest
import torch

import _kv4
import expert_routing_moe_gb300 as moe
from _gpu import DEV, assert_status_ok, status_tensor

pytestmark = pytest.mark.gpu
EPS = 1e-6


def _table(n_pos, rot):
    f = 1e4 ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(n_pos)[:, None] * f
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def _expected(x, n_q, n_kv, D, qw, kw, table, pos, axis, rot, pairs):
    """q and k rows in 64 bits, and for each number the sum of magnitudes its fp32 roundings scale with."""
    T = x.shape[0]
    x = x.astype(np.float64).reshape(T, n_q + 2 * n_kv, D)
    y = x[:, :n_q + n_kv].copy()
    for h in range(n_q + n_kv):
        w = qw if h < n_q else kw
        if w is not None:
            y[:, h] = y[:, h] / np.sqrt((y[:, h] ** 2).mean(-1, keepdims=True) + EPS) * w.astype(np.float64)
    size = np.abs(y)
    if rot:
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if pairs else (i, i + rot // 2)
        c, s = np.moveaxis(table.astype(np.float64)[pos[axis].T, i], -1, 0)[:, :, None]
        u, v = y[..., a].copy(), y[..., b].copy()
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
        size[..., a] = size[..., b] = np.abs(u) + np.abs(v)
    return y[:, :n_q], y[:, n_q:], x[:, n_q + n_kv:], size[:, :n_q], size[:, n_q:]


def _run(rng, T, n_q, n_kv, D, dtype, *, norm=True, rot=None, axes=1, pairs=False, cache=None, q_start=None, pos=None, k_out=True,
         pad=0, x=None, st=None):
    rot = D if rot is None else rot
    width = (n_q + 2 * n_kv) * D
    if x is None:
        x = rng.normal(size=(T, width)) * rng.uniform(0.2, 3, (T, 1))
    xt = torch.zeros(T, width + pad, dtype=dtype, device=DEV)
    xt[:, :width] = torch.from_numpy(x).to(DEV)
    xt = xt[:, :width]
    xv = xt.float().cpu().numpy()
    qw = kw = None
    if norm:
        qw, kw = (rng.uniform(0.5, 1.5, D).astype(np.float32) for _ in range(2))
    n_pos = 5000
    table = _table(n_pos, rot) if rot else None
    axis = rng.integers(0, axes, max(rot // 2, 1)) if axes > 1 else np.zeros(max(rot // 2, 1), int)
    if pos is None:
        pos = rng.integers(0, n_pos, (axes, T))
    rope = None
    if rot:
        rope = moe.Rope(torch.from_numpy(table).to(DEV), torch.from_numpy(pos.astype(np.int32)).to(DEV),
                        torch.from_numpy(axis.astype(np.uint8)).to(DEV) if axes > 1 else None, pairs=pairs)
    q = torch.full((T, n_q, D), float("nan"), dtype=dtype, device=DEV)
    k = torch.full((T, n_kv, D), float("nan"), dtype=dtype, device=DEV) if k_out else None
    own = st is None
    st = status_tensor() if own else st
    w = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
    moe.moe_qk_norm_rope(xt, n_q, n_kv, q, k, w(qw), w(kw), EPS, rope, cache, q_start, st)
    torch.cuda.synchronize()
    if own:
        assert_status_ok(st)
    exp = _expected(xv, n_q, n_kv, D, qw, kw, table, pos, axis, rot, pairs)
    return q, k, exp, xv


def _close(got, want, size, dtype):
    # the sum of squares: 12 roundings (half of them counts in its root); mean, eps, root, reciprocal, two products,
    # and a product and a sum of the rotation: 16 roundings of 2^-24 in all, scaled by |a| + |b|; then the output's own
    tol = 16 * 2.0 ** -24 * size + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) * np.abs(want) + 1e-30
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,n_q,n_kv,D", [(1, 32, 4, 128), (3, 14, 2, 64), (70, 5, 1, 128), (777, 8, 8, 64), (1100, 32, 4, 128), (1, 0, 1, 64)])
@pytest.mark.parametrize("pairs", [False, True])
def test_norm_and_rotation(dtype, T, n_q, n_kv, D, pairs):
    rng = np.random.default_rng(T * 7 + D)
    q, k, exp, _ = _run(rng, T, n_q, n_kv, D, dtype, axes=3, pairs=pairs, pad=64)
    if n_q:
        _close(q, exp[0], exp[3], dtype)
    _close(k, exp[1], exp[4], dtype)


@pytest.mark.parametrize("D,rot,norm,pairs", [(128, 64, True, False), (128, 96, False, False), (64, 32, True, True), (128, 0, True, False), (64, 0, False, False)])
def test_partial_rotation_and_no_norm(D, rot, norm, pairs):
    rng = np.random.default_rng(D + rot)
    q, k, exp, _ = _run(rng, 50, 6, 2, D, torch.float32, rot=rot, norm=norm, pairs=pairs)
    _close(q, exp[0], exp[3], torch.float32)
    _close(k, exp[1], exp[4], torch.float32)


def test_in_place():
    rng = np.random.default_rng(3)
    T, n_q, n_kv, D = 40, 8, 2, 128
    x = torch.randn(T, n_q + 2 * n_kv, D, device=DEV).bfloat16()
    w = torch.from_numpy(rng.uniform(0.5, 1.5, D).astype(np.float32)).to(DEV)
    rope = moe.Rope(torch.from_numpy(_table(64, D)).to(DEV), torch.arange(T, dtype=torch.int32, device=DEV)[None])
    q, k = torch.empty(T, n_q, D, device=DEV, dtype=torch.bfloat16), torch.empty(T, n_kv, D, device=DEV, dtype=torch.bfloat16)
    moe.moe_qk_norm_rope(x, n_q, n_kv, q, k, w, w, rope=rope)
    y = x.clone()
    moe.moe_qk_norm_rope(y, n_q, n_kv, y[:, :n_q], y[:, n_q:n_q + n_kv], w, w, rope=rope)
    assert torch.equal(y[:, :n_q], q) and torch.equal(y[:, n_q:n_q + n_kv], k) and torch.equal(y[:, n_q + n_kv:], x[:, n_q + n_kv:])


def _dev_cache(c):
    t = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
    return moe.Kv4Cache(t(c.bytes), t(c.table), torch.tensor(c.lengths, dtype=torch.int32, device=DEV), c.D, t(c.k_scale), t(c.v_scale))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n_kv,D", [(1, 128), (4, 128), (2, 64), (3, 64)])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("lengths,new", [([1], [1]), ([64], [1]), ([65, 3, 130], [1, 1, 1]), ([7, 200, 0, 65], [7, 131, 1, 2]),
                                         ([129, 64, 2], [66, 1, 0]), ([700], [601])])
def test_append_and_read(dtype, n_kv, D, pairs, lengths, new):
    """Values come back exactly as the reference's codes; keys within what their codes may be off; the
    tokens around them keep their bytes."""
    rng = np.random.default_rng(sum(lengths) + D + n_kv)
    c = _kv4.Cache(rng, lengths, n_kv, D)
    dc = _dev_cache(c)
    T, n_q = sum(new), 3
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q_start = torch.from_numpy(starts).to(DEV)
    q, k, exp, xv = _run(rng, T, n_q, n_kv, D, dtype, axes=3, pairs=pairs, cache=dc, q_start=q_start)
    _close(q, exp[0], exp[3], dtype)
    _close(k, exp[1], exp[4], dtype)
    kr, vr = (torch.full((T, n_kv, D), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    st = status_tensor()
    moe.moe_kv4_read(dc, q_start, kr, vr, st)
    torch.cuda.synchronize()
    assert_status_ok(st)
    vc, vs = _kv4.quantise(exp[2].astype(np.float32), c.v_scale[:, None])
    v_want = torch.from_numpy(_kv4.values(vc, vs, c.v_scale[:, None]).astype(np.float32)).bfloat16()
    got_v, got_k = vr.cpu(), kr.double().cpu().numpy()
    seq = np.searchsorted(starts, np.arange(T), "right") - 1
    place = np.array(lengths)[seq] - starts[seq + 1] + np.arange(T)
    there = place >= 0
    assert torch.equal(got_v[there], v_want[there]) and (got_v[~there] == 0).all()
    assert (got_k[~there] == 0).all()
    hs = c.k_scale.astype(np.float64)[:, None]
    top = np.repeat((np.abs(exp[1]) / hs).reshape(T, n_kv, D // 16, 16).max(-1), 16, -1)
    # half of the widest step (2) times a scale of at most (1 + 2^-4) top/6 (2^-10 where it is subnormal), bf16 rounding, fp32 noise
    tol = (top / 6 * (1 + 2.0 ** -4) + 6 * 2.0 ** -10) * hs + 2.0 ** -8 * np.abs(got_k) + 2.0 ** -18 * exp[4]
    assert (np.abs(got_k - exp[1]) <= tol)[there].all()
    # old tokens are what they were
    full = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32), device=DEV)
    L = sum(lengths)
    ka, va = (torch.empty(L, n_kv, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    moe.moe_kv4_read(dc, full, ka, va)
    ka, va = ka.float().cpu().numpy(), va.float().cpu().numpy()
    at = 0
    for s, n in enumerate(lengths):
        old = max(0, n - new[s])
        bf = lambda a: torch.from_numpy(a.astype(np.float32)).bfloat16().float().numpy()  # noqa: E731
        assert np.array_equal(ka[at:at + old], bf(c.k[s][:old])) and np.array_equal(va[at:at + old], bf(c.v[s][:old]))
        at += n
    # bytes of pages and tokens that the call has no business with
    host = dc.tensors[0].cpu().numpy()
    used = set(c.table[c.table >= 0].tolist())
    for p in range(host.shape[0]):
        if p not in used:
            assert np.array_equal(host[p], c.bytes[p])


def test_keys_without_norm_and_rotation_are_exact():
    rng = np.random.default_rng(9)
    c = _kv4.Cache(rng, [100, 31], 2, 128)
    dc = _dev_cache(c)
    q_start = torch.tensor([0, 50, 81], dtype=torch.int32, device=DEV)
    _, _, exp, _ = _run(rng, 81, 2, 2, 128, torch.float32, norm=False, rot=0, cache=dc, q_start=q_start)
    kr = torch.empty(81, 2, 128, dtype=torch.bfloat16, device=DEV)
    moe.moe_kv4_read(dc, q_start, kr, None)
    kc, ks = _kv4.quantise(exp[1].astype(np.float32), c.k_scale[:, None])
    want = torch.from_numpy(_kv4.values(kc, ks, c.k_scale[:, None]).astype(np.float32)).bfloat16()
    assert torch.equal(kr.cpu(), want)


def test_extreme_blocks():
    """Zero blocks, blocks beyond the largest scale, tiny ones, and a block with a single number."""
    D, n_kv = 64, 1
    x = np.zeros((6, 3 * D), np.float32)
    x[1] = 1e6
    x[2, :] = 1e-4
    x[3, 2 * D + 5] = 3.0
    x[4] = -0.0
    x[5, ::2] = -2.5e-3
    rng = np.random.default_rng(0)
    c = _kv4.Cache(rng, [6], n_kv, D, scales=False)
    dc = _dev_cache(c)
    qs = torch.tensor([0, 6], dtype=torch.int32, device=DEV)
    _, _, exp, _ = _run(rng, 6, 1, 1, D, torch.float32, norm=False, rot=0, cache=dc, q_start=qs, x=x)
    kr, vr = (torch.empty(6, 1, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    moe.moe_kv4_read(dc, qs, kr, vr)
    for got, y in ((kr, exp[1]), (vr, exp[2])):
        want = torch.from_numpy(_kv4.values(*_kv4.quantise(y.astype(np.float32), np.ones((1, 1))), 1.0).astype(np.float32)).bfloat16()
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("row,part", [(4, "k"), (4, "v"), (5, "v")])
def test_non_finite_is_reported_and_stored_as_zero(bad, row, part):
    rng = np.random.default_rng(1)
    D = 128
    x = rng.normal(size=(8, 3 * D))
    at = (1 if part == "k" else 2) * D + 17
    x[row, at] = bad
    c = _kv4.Cache(rng, [8], 1, D)
    dc = _dev_cache(c)
    qs = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    st = status_tensor()
    _run(rng, 8, 1, 1, D, torch.float32, norm=False, rot=0, cache=dc, q_start=qs, x=x, st=st)
    assert st.tolist() == [1, row]
    kr, vr = (torch.empty(8, 1, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    moe.moe_kv4_read(dc, qs, kr, vr)
    got = (kr if part == "k" else vr)[row, 0]
    assert torch.isfinite(kr).all() and torch.isfinite(vr).all() and got[17] == 0 and (got[:16] != 0).any()


def test_places_serve_as_positions_and_bad_indexes_are_reported():
    rng = np.random.default_rng(5)
    D, n_kv = 128, 2
    c = _kv4.Cache(rng, [70, 9], n_kv, D)
    dc = _dev_cache(c)
    qs = torch.tensor([0, 5, 14], dtype=torch.int32, device=DEV)
    x = torch.randn(14, 6 * D, device=DEV).bfloat16()
    table = torch.from_numpy(_table(80, D)).to(DEV)
    pos = torch.tensor([list(range(65, 70)) + list(range(9))], dtype=torch.int32, device=DEV)
    a, b = (torch.empty(14, 2, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    st = status_tensor()
    moe.moe_qk_norm_rope(x, 2, n_kv, a, rope=moe.Rope(table), cache=dc, q_start=qs, st=st)
    moe.moe_qk_norm_rope(x, 2, n_kv, b, rope=moe.Rope(table, pos), cache=dc, q_start=qs, st=st)
    assert st.tolist() == [0, 0] and torch.equal(a, b)
    # a position beyond the table
    pos[0, 3] = 80
    moe.moe_qk_norm_rope(x, 2, n_kv, b, rope=moe.Rope(table, pos), st=st)
    assert st.tolist() == [3, 80]
    # a page beyond the pool and an empty table entry: reported, nothing written
    for entry in (-1, dc.n_pages):
        st.zero_()
        dc.tensors[1][0, 1] = entry
        before = dc.tensors[0].clone()
        moe.moe_qk_norm_rope(x[:5], 2, n_kv, a[:5], rope=moe.Rope(table), cache=dc, q_start=torch.tensor([0, 5, 5], dtype=torch.int32, device=DEV), st=st)
        assert st.tolist() == [3, entry]
        assert torch.equal(dc.tensors[0], before)   # places 65..69 lie in the bad page


def test_other_stream_and_capture():
    rng = np.random.default_rng(6)
    D, n_kv, T = 128, 4, 3
    c = _kv4.Cache(rng, [66, 64, 10], n_kv, D)
    dc = _dev_cache(c)
    qs = torch.arange(4, dtype=torch.int32, device=DEV)
    x = torch.randn(T, (8 + 2 * n_kv) * D, device=DEV).bfloat16()
    rope = moe.Rope(torch.from_numpy(_table(80, D)).to(DEV))
    w = torch.ones(D, device=DEV)
    q = torch.empty(T, 8, D, dtype=torch.bfloat16, device=DEV)
    moe.moe_qk_norm_rope(x, 8, n_kv, q, q_weight=w, k_weight=w, rope=rope, cache=dc, q_start=qs)
    want, pages = q.clone(), dc.tensors[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        moe.moe_qk_norm_rope(x, 8, n_kv, q, q_weight=w, k_weight=w, rope=rope, cache=dc, q_start=qs)
    q.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q, want) and torch.equal(dc.tensors[0], pages)
