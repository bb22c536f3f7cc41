"""Attention over the 4-bit paged cache on the GPU against 64-bit numpy."""
import numpy as np
import pytest
import torch

import _kv4
import expert_routing_moe_gb300 as moe
from _gpu import DEV, assert_status_ok, status_tensor

pytestmark = pytest.mark.gpu


def _dev_cache(c):
    t = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
    return moe.Kv4Cache(t(c.bytes), t(c.table), torch.tensor(c.lengths, dtype=torch.int32, device=DEV), c.D, t(c.k_scale), t(c.v_scale))


def _ws(T, n_q, n_kv, D):
    return torch.zeros(moe.attention_kv4_workspace(T, n_q, n_kv, D), dtype=torch.uint8, device=DEV)


def _check(rng, lengths, new, n_q, n_kv, D, *, window=0, scales=True, size=1.0, pad=0, max_new=None, repeat=1):
    c = _kv4.Cache(rng, lengths, n_kv, D, scales=scales)
    dc = _dev_cache(c)
    T = sum(new)
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    q = torch.zeros(T, n_q * D + pad, dtype=torch.bfloat16, device=DEV)
    q[:, :n_q * D] = torch.from_numpy(rng.normal(size=(T, n_q * D)) * size).to(DEV)
    q = q[:, :n_q * D].unflatten(1, (n_q, D))
    out = torch.full((T, n_q * D + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
    ov = out[:, :n_q * D].unflatten(1, (n_q, D))
    lse = torch.full((T, n_q), float("nan"), device=DEV)
    scale = D ** -0.5
    ws, st = _ws(T, n_q, n_kv, D), status_tensor()
    seen = None
    for _ in range(repeat):
        moe.moe_attention_kv4(q, dc, torch.from_numpy(starts).to(DEV), ov, scale, max_new=max(new) if max_new is None else max_new,
                              window=window, lse=lse, workspace=ws, st=st)
        torch.cuda.synchronize()
        assert_status_ok(st)
        got = (ov.cpu(), lse.cpu())
        assert seen is None or (torch.equal(got[0], seen[0]) and torch.equal(got[1], seen[1]))   # the same bits each time
        seen = got
    if pad:
        assert torch.isnan(out[:, n_q * D:]).all()
    o, z, tol, tol_z = _kv4.attention(c, q.double().cpu().numpy(), starts, scale, window)
    err = np.abs(ov.double().cpu().numpy() - o)
    assert (err <= tol).all(), "out: %.3g of its bound" % float(np.nanmax(err / np.maximum(tol, 1e-30)))
    got_z = lse.double().cpu().numpy()
    empty = np.isneginf(z)
    assert np.array_equal(np.isneginf(got_z), empty) and (ov.float().cpu().numpy()[empty] == 0).all()
    assert (np.abs(got_z - z)[~empty] <= tol_z[~empty]).all()


HEADS = [(8, 1, 128), (32, 4, 128), (4, 4, 64), (14, 2, 64), (24, 2, 128), (20, 1, 64)]


@pytest.mark.parametrize("n_q,n_kv,D", HEADS)
@pytest.mark.parametrize("lengths", [[1], [63], [64], [65], [5, 0, 128, 700, 1], [3000]])
def test_single_tokens(n_q, n_kv, D, lengths):
    rng = np.random.default_rng(sum(lengths) + n_q)
    _check(rng, lengths, [1] * len(lengths), n_q, n_kv, D, repeat=2)


@pytest.mark.parametrize("n_q,n_kv,D", HEADS)
@pytest.mark.parametrize("lengths,new", [([70, 2, 300], [4, 2, 3]), ([5, 130, 64, 9], [5, 0, 7, 1])])
def test_drafts(n_q, n_kv, D, lengths, new):
    rng = np.random.default_rng(sum(lengths) + D)
    _check(rng, lengths, new, n_q, n_kv, D, pad=64)


@pytest.mark.parametrize("n_q,n_kv,D", HEADS)
@pytest.mark.parametrize("lengths,new", [([150], [150]), ([333, 64, 1, 200], [77, 64, 1, 40])])
def test_prompt_chunks(n_q, n_kv, D, lengths, new):
    rng = np.random.default_rng(sum(lengths) + 3 * D)
    _check(rng, lengths, new, n_q, n_kv, D, pad=8, repeat=2)


@pytest.mark.parametrize("window", [1, 50, 64, 129, 100000])
@pytest.mark.parametrize("n_q,n_kv,D,lengths,new", [(8, 1, 128, [400, 64, 3], [1, 1, 1]), (14, 2, 64, [260, 65], [4, 5]),
                                                    (8, 2, 128, [300, 90], [120, 90])])
def test_windows(window, n_q, n_kv, D, lengths, new):
    _check(np.random.default_rng(window), lengths, new, n_q, n_kv, D, window=window)


def test_large_and_small_scores():
    """Scores of some thousands (one key takes all) and of almost nothing."""
    _check(np.random.default_rng(1), [200, 90], [1, 2], 8, 1, 128, size=300.0)
    _check(np.random.default_rng(2), [200, 90], [1, 2], 8, 1, 128, size=1e-6, scales=False)
    _check(np.random.default_rng(3), [200], [80], 8, 1, 128, size=300.0)


def test_more_rows_than_the_bound_says():
    """max_new only chooses kernels."""
    for bound in (0, 1, 1000):
        _check(np.random.default_rng(4), [90, 5], [60, 2], 8, 2, 64, max_new=bound)


def test_rows_before_their_sequence():
    """More rows than tokens: the first rows see nothing."""
    _check(np.random.default_rng(5), [3, 0], [6, 40], 8, 2, 128)


@pytest.mark.parametrize("window", [0, 30])
def test_prompt_rows_before_their_sequence(window):
    """Whole blocks of a prompt's rows that see nothing, before, between and after ones that do."""
    _check(np.random.default_rng(15), [70, 3, 0, 500], [300, 6, 200, 400], 8, 2, 128, window=window, pad=8, repeat=2)


@pytest.mark.parametrize("n_q,n_kv,D,window", [(16, 2, 128, 0), (14, 2, 64, 40)])
def test_many_short_prompts(n_q, n_kv, D, window):
    """Several blocks of rows for each CTA, each with a few pages."""
    rng = np.random.default_rng(16 + window)
    new = [int(x) for x in rng.integers(1, 90, 120)]
    _check(rng, [x + int(rng.integers(0, 100)) for x in new], new, n_q, n_kv, D, window=window, repeat=2)


@pytest.mark.parametrize("new", [16, 17, 32, 33, 128, 129])
def test_rows_around_the_kernels_bounds(new):
    """Rows of a sequence on both sides of what goes to the one kernel or the other, alone and among others."""
    _check(np.random.default_rng(new), [200], [new], 8, 1, 128)
    _check(np.random.default_rng(new), [200, 150, 170], [new, 120, 1], 8, 1, 128, max_new=120)


def test_non_finite_queries_stay_in_their_rows():
    rng = np.random.default_rng(6)
    for new in (1, 100):
        c = _kv4.Cache(rng, [300, 200], 1, 128)
        dc = _dev_cache(c)
        q = torch.randn(2 * new, 8, 128, device=DEV).bfloat16()
        starts = torch.tensor([0, new, 2 * new], dtype=torch.int32, device=DEV)
        a, b = torch.empty_like(q), torch.empty_like(q)
        moe.moe_attention_kv4(q, dc, starts, a, 0.1, max_new=new)
        q[0, 3, 5] = float("nan")
        q[new, 0, 7] = float("inf")
        moe.moe_attention_kv4(q, dc, starts, b, 0.1, max_new=new)
        assert torch.isnan(b[0, 3]).all() and not torch.isfinite(b[new, 0]).all()
        b[0, 3], b[new, 0] = a[0, 3], a[new, 0]
        assert torch.equal(a, b)


def test_bad_indexes_are_reported_and_skipped():
    rng = np.random.default_rng(7)
    for new in (1, 90):
        c = _kv4.Cache(rng, [300, 200], 2, 128)
        dc = _dev_cache(c)
        q = torch.randn(2 * new, 8, 128, device=DEV).bfloat16()
        out = torch.zeros_like(q)
        starts = torch.tensor([0, new, 2 * new], dtype=torch.int32, device=DEV)
        for bad in (-1, dc.n_pages):
            st = status_tensor()
            dc.tensors[1][1, 1] = bad
            moe.moe_attention_kv4(q, dc, starts, out, 0.1, max_new=new, st=st)
            assert st.tolist()[0] == 3 and torch.isfinite(out).all()
        # a length beyond the table, rows beyond T, descending starts
        for lens, qs in (([300, 100000], [0, new, 2 * new]), ([300, 200], [0, new, 2 * new + 1]), ([300, 200], [new, 0, new])):
            st = status_tensor()
            dc.tensors[2].copy_(torch.tensor(lens, dtype=torch.int32))
            moe.moe_attention_kv4(q, dc, torch.tensor(qs, dtype=torch.int32, device=DEV), out, 0.1, max_new=new, st=st)
            assert st.tolist()[0] == 3


def test_far_pages():
    """A cache whose last pages lie beyond 2^32 bytes."""
    D, n_kv = 128, 4
    n = (1 << 32) // _kv4.page_bytes(n_kv, D) + 5
    rng = np.random.default_rng(8)
    c = _kv4.Cache(rng, [130], n_kv, D, spare=0)
    pages = torch.empty(n, n_kv, 9216, dtype=torch.uint8, device=DEV)
    pages[n - 3:] = torch.from_numpy(c.bytes).to(DEV)
    t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    table = torch.where(t(c.table) >= 0, t(c.table) + n - 3, -1).int()
    dc = moe.Kv4Cache(pages, table, torch.tensor([130], dtype=torch.int32, device=DEV), D, t(c.k_scale), t(c.v_scale))
    near = _dev_cache(c)
    for new in (1, 60):
        q = torch.randn(new, 32, D, device=DEV).bfloat16()
        a, b = torch.empty_like(q), torch.empty_like(q)
        starts = torch.tensor([0, new], dtype=torch.int32, device=DEV)
        moe.moe_attention_kv4(q, dc, starts, a, 0.1, max_new=new)
        moe.moe_attention_kv4(q, near, starts, b, 0.1, max_new=new)
        assert torch.equal(a, b)
    k = torch.empty(60, n_kv, D, dtype=torch.bfloat16, device=DEV)
    moe.moe_kv4_read(dc, starts, k, None)
    want = torch.from_numpy(c.k[0][70:].astype(np.float32)).bfloat16()
    assert torch.equal(k.cpu(), want)


def test_capture_follows_the_lengths():
    """A captured step attends over what the cache holds when it is replayed."""
    rng = np.random.default_rng(9)
    lengths = [200, 64, 31]
    c = _kv4.Cache(rng, lengths, 4, 128)
    dc = _dev_cache(c)
    q = torch.randn(3, 32, 128, device=DEV).bfloat16()
    starts = torch.arange(4, dtype=torch.int32, device=DEV)
    out, ws = torch.empty_like(q), _ws(3, 32, 4, 128)
    moe.moe_attention_kv4(q, dc, starts, out, 0.1, max_new=1, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_attention_kv4(q, dc, starts, out, 0.1, max_new=1, workspace=ws)
    for lens in ([200, 64, 31], [77, 1, 0], [129, 63, 30]):
        dc.tensors[2].copy_(torch.tensor(lens, dtype=torch.int32))
        want = torch.empty_like(q)
        moe.moe_attention_kv4(q, dc, starts, want, 0.1, max_new=1, workspace=ws)
        out.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_binding_refuses():
    rng = np.random.default_rng(10)
    dc = _dev_cache(_kv4.Cache(rng, [10], 2, 64))
    q = torch.randn(1, 4, 64, device=DEV).bfloat16()
    qs = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    with pytest.raises(moe.MoeError, match="q"):
        moe.moe_attention_kv4(q.float(), dc, qs, torch.empty_like(q), 0.1, max_new=1)
    with pytest.raises(moe.MoeError, match="q_start"):
        moe.moe_attention_kv4(q, dc, qs[:1], torch.empty_like(q), 0.1, max_new=1)
    with pytest.raises(moe.MoeError, match="out"):
        moe.moe_attention_kv4(q, dc, qs, torch.empty(2, 4, 64, device=DEV, dtype=torch.bfloat16), 0.1, max_new=1)
    with pytest.raises(moe.MoeError, match="strided"):
        moe.moe_attention_kv4(q.transpose(1, 2).contiguous().transpose(1, 2), dc, qs, torch.empty_like(q), 0.1, max_new=1)
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_attention_kv4(q, dc, qs, torch.empty_like(q), 0.1, max_new=1, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
