"""Calls at the edges between variants of the products in 4 bits, the weighing, the
verification and the eviction: many rows, many sequences, other streams."""
import numpy as np
import pytest
import torch

import _kv4
import _verify
import _w4
import expert_routing_moe_gb300 as moe
from _gpu import DEV, dev, host, status_tensor
from test_gpu_kv4_evict import Gpu, Host
from test_gpu_kv4_weigh import Case
from test_gpu_linear_w4 import EPS, Weights, _bf16, _check
from test_gpu_verify import _case

pytestmark = pytest.mark.gpu


def _place(a, dtype, shift, ld):
    """Rows `ld` numbers apart that start `shift` numbers into their memory, NaN between them."""
    T, V = a.shape
    buf = torch.full((T * ld + shift + 8,), float("nan"), dtype=dtype, device=DEV)
    out = buf[shift:shift + T * ld].view(T, ld)[:, :V]
    out.copy_(dev(a))
    return out


@pytest.mark.parametrize("S,V", [(70, 20003), (33, 50001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("by_model", [False, True])
def test_verification_of_many_rows(S, V, dtype, by_model):
    """Rows in many chunks; the drafting model's rows lie otherwise between 16-byte boundaries than the target's."""
    rng = np.random.default_rng(S)
    logits, tokens, uniform, q_start, draft, temp = _case(rng, S, 3, V, by_model, dtype)
    T = len(tokens)
    bad = {1: np.nan, 5: np.inf}                       # rows of sequences that then have no answer
    for s, v in bad.items():
        if q_start[s + 1] > q_start[s]:
            logits[q_start[s], V - 1] = v
    nothing = q_start[9]
    logits[nothing] = -np.inf
    st = status_tensor()
    acc, nxt, n_new = (torch.full((S,), -77, dtype=torch.int32, device=DEV) for _ in range(3))
    ws = torch.full((moe.verify_workspace(T, S, V),), 255, dtype=torch.uint8, device=DEV)
    moe.moe_verify_drafts(_place(logits, dtype, 1, V + 2), dev(tokens), dev(uniform), dev(q_start.astype(np.int32)), acc, nxt, n_new,
                          draft_logits=None if draft is None else _place(draft, dtype, 3, V + 5), temperature=dev(temp), workspace=ws, st=st)
    with np.errstate(invalid="ignore"):
        want = _verify.verify(logits, tokens, uniform, q_start, draft, temp)
    for g, w in zip((acc, nxt, n_new), want):
        assert np.array_equal(host(g), w)
    assert st.tolist()[0] == 1                         # not finite


@pytest.mark.parametrize("S", [303, 304, 305])
def test_verification_between_its_variants(S):
    rng = np.random.default_rng(S)
    V = 300
    c = [rng.normal(size=(S, V)).astype(np.float32) * 3, np.zeros(S, np.int32), rng.random(S).astype(np.float32), np.arange(S + 1), None, None]
    acc, nxt, n_new = (torch.full((S,), -77, dtype=torch.int32, device=DEV) for _ in range(3))
    moe.moe_verify_drafts(dev(c[0]), dev(c[1]), dev(c[2]), dev(c[3].astype(np.int32)), acc, nxt, n_new)
    for g, w in zip((acc, nxt, n_new), _verify.verify(*c)):
        assert np.array_equal(host(g), w)


def test_more_rows_than_a_sequence_may_have():
    c = Case(31, [100, 90], [5, 2], 8, 2, 64)
    good = host(c.run())
    for n, q_start in ((3, [0, 5, 7]), (200, [0, 300, 302])):
        c = Case(31, [400, 90], [q_start[1], 2], 8, 2, 64) if n > 3 else c
        good = host(c.run())
        c.max_new = n
        st = status_tensor()
        got = host(c.run(st=st))
        assert st.tolist() == [3, 0]
        assert np.array_equal(got[0], c.score[0]) and np.array_equal(got[1], good[1])


@pytest.mark.parametrize("lengths,rows,n_q,n_kv,D", [
    ([150], [3], 32, 16, 64), ([90, 200], [20, 4], 100, 1, 64), ([200], [30], 97, 1, 128), ([130], [3], 96, 1, 64), ([70] * 40, [1] * 40, 4, 2, 64), (list(range(300)), [1] * 300, 2, 1, 64),
    ([300] * 5, [32] * 5, 8, 1, 64), ([300] * 5, [31] * 5, 8, 1, 64), ([300] * 5, [16] * 5, 8, 1, 64), ([300] * 5, [15] * 5, 8, 1, 64), ([200, 70], [16, 15], 8, 1, 128)])
def test_weighing_of_other_shapes(lengths, rows, n_q, n_kv, D):
    """More key heads than one pass holds, groups beyond a tile, many sequences, rows at the limit of a variant."""
    rows = [min(r, n) for r, n in zip(rows, lengths)]
    Case(32, lengths, rows, n_q, n_kv, D).check()


@pytest.mark.parametrize("T,N,K", [
    (8, 4864, 130), (8, 4865, 130), (9, 14592, 130), (9, 14593, 130), (40, 14593, 200), (63, 257, 200), (64, 257, 200), (65, 257, 200), (66, 130, 137), (5, 14600, 8200),
    (96, 600, 72), (97, 600, 72), (191, 300, 130), (192, 300, 130), (193, 300, 130), (385, 129, 140)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_products_between_their_variants(T, N, K, dtype):
    rng = np.random.default_rng(T + N)
    w = Weights(rng, N, K)
    x = _bf16(rng.normal(size=(T, K)))
    y = torch.full((T, N), float("nan"), dtype=dtype, device=DEV)
    moe.moe_linear_w4(x.to(DEV), w.w, y)
    _check(y, _w4.linear(x.double().numpy(), w.ref, out_eps=EPS[dtype]), dtype)
    if dtype == torch.float32:
        before = y.double()
        moe.moe_linear_w4(x.to(DEV), w.w, y, accumulate=True)
        # twice the first sum, rounded once
        assert torch.equal(y, (2 * before).float())


def test_through_another_stream():
    """Each operator with `stream=`, while the current stream is another one and busy with something else."""
    rng = np.random.default_rng(33)
    side = torch.cuda.Stream()
    w = Weights(rng, 300, 200)
    x = _bf16(rng.normal(size=(70, 200))).to(DEV)
    want_y, got_y = (torch.empty(70, 300, device=DEV) for _ in range(2))
    moe.moe_linear_w4(x, w.w, want_y)
    c = Case(34, [500, 90], [70, 3], 8, 2, 64)
    q_start, lse, score = dev(c.q_start), dev(c.lse), dev(c.score)
    want_s = c.run()
    v = _case(rng, 7, 3, 2001, True, torch.float32)
    args = [dev(v[0]), dev(v[1]), dev(v[2]), dev(v[3].astype(np.int32))]
    outs = [torch.full((7,), -77, dtype=torch.int32, device=DEV) for _ in range(3)]
    draft, temp = dev(v[4]), dev(v[5])
    h = Host(rng, [300, 200], 2, 1, 64)
    g = Gpu(h)
    budget = dev(np.array([100, 150], np.int32))
    tiles = moe.Weight4.empty(300, 200, DEV)
    dense = torch.randn(300, 200, device=DEV)
    want_w = moe.Weight4.pack(dense)
    torch.cuda.synchronize()
    busy = torch.randn(2048, 2048, device=DEV)
    for _ in range(5):
        busy = busy @ busy
    moe.moe_linear_w4(x, w.w, got_y, stream=side)
    moe.moe_kv4_weigh(c.q_dev, c.cache, q_start, lse, score, c.scale, c.max_new, stream=side)
    moe.moe_verify_drafts(*args, *outs, draft_logits=draft, temperature=temp, stream=side)
    moe.moe_kv4_evict(g.pool, g.score, budget, 2, 3, g.ws, None, g.st, stream=side)
    moe.moe_w4_pack(dense, tiles, stream=side)
    side.synchronize()
    assert torch.equal(want_y, got_y) and torch.equal(want_s, score)
    for a, b in zip(outs, _verify.verify(*v)):
        assert np.array_equal(host(a), b)
    assert h.evict(host(budget), 2, 3) == (0, 0)
    g.same(h)
    assert torch.equal(tiles.tensors[0], want_w.tensors[0]) and torch.equal(tiles.tensors[1], want_w.tensors[1])


def test_two_evictions_at_once():
    """Pools of their own, each with its workspace, on two streams."""
    rng = np.random.default_rng(35)
    hosts = [Host(rng, [3000, 100, 900], 4, 2, 64, shared=[2], spare=30), Host(rng, [2500, 1800], 4, 2, 128)]
    gpus, streams = [Gpu(h) for h in hosts], [torch.cuda.Stream() for _ in hosts]
    for turn in range(3):
        budgets = [np.array([1500 - 400 * turn, 50, 300], np.int32), np.array([2000 - 500 * turn, 1000], np.int32)]
        on = [dev(b) for b in budgets]
        torch.cuda.synchronize()
        for g, b, s in zip(gpus, on, streams):
            moe.moe_kv4_evict(g.pool, g.score, b, 4, 20, g.ws, None, g.st, stream=s)
        torch.cuda.synchronize()
        for g, b, h in zip(gpus, budgets, hosts):
            assert h.evict(b, 4, 20) == (0, 0)
            g.same(h)


def test_a_short_status_is_refused():
    short = torch.zeros(1, dtype=torch.int32, device=DEV)
    w = Weights(np.random.default_rng(36), 20, 16)
    x, y = torch.zeros(1, 16, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 20, device=DEV)
    c = Case(36, [70], [1], 2, 1, 64)
    q_start, lse, score = dev(c.q_start), dev(c.lse), dev(c.score)
    one, f = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros(1, device=DEV)
    g = Gpu(Host(np.random.default_rng(36), [70], 1, 1, 64))
    before = g.len.clone()
    for stream in (None, torch.cuda.current_stream()):
        for call in (lambda: moe.moe_linear_w4(x, w.w, y, st=short, stream=stream),
                     lambda: moe.moe_w4_pack(torch.zeros(20, 16, device=DEV), w.w, st=short, stream=stream),
                     lambda: moe.moe_kv4_weigh(c.q_dev, c.cache, q_start, lse, score, 1.0, 1, st=short, stream=stream),
                     lambda: moe.moe_verify_drafts(torch.zeros(1, 9, device=DEV), one, f, q_start, one, one, st=short, stream=stream),
                     lambda: moe.moe_kv4_evict(g.pool, g.score, one, 0, 0, g.ws, st=short, stream=stream)):
            with pytest.raises(moe.MoeError, match="status"):
                call()
    assert torch.equal(g.len, before) and np.array_equal(host(score), c.score)


@pytest.mark.parametrize("T,N,K", [(9, 30000, 1024), (16, 40001, 600), (17, 9000, 1100), (33, 2049, 2100), (70, 300, 513), (24, 3000, 2047), (130, 2048, 4096), (64, 4000, 8000), (300, 515, 1290)])
def test_products_whose_tiles_are_shared(T, N, K):
    """Few tiles: a tile's columns in parts; with a bias and added to y, rows of x at any boundary."""
    rng = np.random.default_rng(T + N)
    w = Weights(rng, N, K)
    wide = torch.full((T, K + 3), float("nan"), dtype=torch.bfloat16, device=DEV)
    for shift in (0, 1):
        x = _bf16(rng.normal(size=(T, K)))
        if shift:
            on = wide[:, 1:K + 1]
            on.copy_(x)
        else:
            on = x.to(DEV)
        bias, y0 = rng.normal(size=N).astype(np.float32), rng.normal(size=(T, N)).astype(np.float32)
        y = dev(y0)
        moe.moe_linear_w4(on, w.w, y, bias=dev(bias), accumulate=True)
        _check(y, _w4.linear(x.double().numpy(), w.ref, bias.astype(np.float64), y0.astype(np.float64), 0.0), torch.float32)


def test_no_tokens():
    w = Weights(np.random.default_rng(37), 20, 16)
    y = torch.full((1, 20), 7.0, device=DEV)
    moe.moe_linear_w4(torch.zeros(0, 16, dtype=torch.bfloat16, device=DEV), w.w, y[:0])
    assert (y == 7).all()


def test_captured_calls_share_workspaces():
    """Two graphs of other sizes use one workspace in turn: verification of few and many rows, prompts weighed."""
    rng = np.random.default_rng(38)
    cases = [_case(rng, 3, 4, 5003, True, torch.float32), _case(rng, 200, 3, 401, False, torch.float32)]
    ws = torch.empty(max(moe.verify_workspace(len(c[1]), len(c[3]) - 1, c[0].shape[1]) for c in cases), dtype=torch.uint8, device=DEV)
    graphs = []
    for c in cases:
        S = len(c[3]) - 1
        on = [dev(c[0]), dev(c[1]), dev(c[2]), dev(c[3].astype(np.int32))]
        outs = [torch.zeros(S, dtype=torch.int32, device=DEV) for _ in range(3)]
        draft, temp = None if c[4] is None else dev(c[4]), dev(c[5])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_verify_drafts(*on, *outs, draft_logits=draft, temperature=temp, workspace=ws)
        graphs.append((graph, on, outs, draft, temp))
    weighed = [Case(39, [500, 90], [70, 30], 8, 2, 64), Case(40, [1100], [300], 4, 1, 128)]
    shared = max((c.ws for c in weighed), key=lambda t: t.numel())
    wanted, replays = [], []
    for c in weighed:
        wanted.append(c.run())
        c.ws = shared
        on = dev(c.score), dev(c.q_start), dev(c.lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_kv4_weigh(c.q_dev, c.cache, on[1], on[2], on[0], c.scale, c.max_new, workspace=c.ws)
        replays.append((graph, on))
    for turn in range(3):
        for c, (graph, on, outs, _, _) in zip(cases, graphs):
            u = rng.random(len(c[2])).astype(np.float32)
            on[2].copy_(dev(u))
            graph.replay()
            for g, want in zip(outs, _verify.verify(c[0], c[1], u, *c[3:])):
                assert np.array_equal(host(g), want)
        for c, want, (graph, on) in zip(weighed, wanted, replays):
            on[0].copy_(dev(c.score))
            graph.replay()
            assert torch.equal(on[0], want)


def test_a_page_twice_in_a_table():
    """A sequence whose table names a page twice (held twice): both are read before either place is made anew."""
    rng = np.random.default_rng(41)
    h = Host(rng, [256, 100], 2, 1, 64, spare=9)
    freed = h.table[0, 1]
    h.table[0, 1] = h.table[0, 0]
    h.ref[h.table[0, 0]], h.ref[freed] = 2, 0
    g = Gpu(h)
    g.evict([100, 50], 2, 3)
    assert h.evict([100, 50], 2, 3) == (0, 0) and g.st.tolist() == [0, 0]
    g.same(h)


@pytest.mark.parametrize("first", [59000, 118000])
def test_pages_far_into_a_large_pool(first):
    """Bytes beyond 2^31 and 2^32 of a pool: the same numbers as in a small one."""
    rng = np.random.default_rng(42)
    c = Case(43, [700, 90], [130, 2], 8, 4, 128)
    small = c.run()
    n, ids = int(c.pages.shape[0]), c.table.clone()
    page = c.pages[0].numel()
    big = torch.zeros(first + n, page, dtype=torch.uint8, device=DEV)
    assert (first + n) * page > 2 ** 31 * (1 if first < 100000 else 2)
    big[first:] = c.pages.view(n, page)
    table = torch.where(ids >= 0, ids + first, ids)
    c.cache = moe.Kv4Cache(big.view(first + n, *c.pages.shape[1:]), table, c.lens, 128, None if c.ref.k_scale is None else dev(c.ref.k_scale), None)
    assert torch.equal(c.run(), small)
    # eviction: the first pages are held by nobody, so free ones are low
    h = Host(rng, [300, 200], 1, 4, 128, spare=0)
    low = Gpu(h)
    held = h.table.copy()
    pages, ref = len(h.ref), np.zeros(first + len(h.ref), np.int32)
    far = Gpu(h)
    data = torch.zeros(1, first + pages, *h.data.shape[2:], dtype=torch.uint8, device=DEV)
    data[:, first:] = dev(h.data)
    ref[first:] = h.ref
    ref[:first] = 1
    far.pages, far.ref, far.table = data, dev(ref), dev(np.where(held >= 0, held + first, held).astype(np.int32))
    far.pool = moe.Kv4Pool(far.pages, far.table, far.len, far.ref, 128)
    far.ws = torch.empty(moe.kv4_evict_workspace(far.pool), dtype=torch.uint8, device=DEV)
    for g in (low, far):
        g.evict([130, 64], 2, 3)
        assert g.st.tolist() == [0, 0]
    assert torch.equal(low.len, far.len) and torch.equal(low.score, far.score) and torch.equal(low.pages, far.pages[:, first:])
    assert torch.equal(torch.where(low.table >= 0, low.table + first, low.table), far.table)


@pytest.mark.parametrize("lengths,rows", [([400, 300, 90], [200, 0, 2]), ([400, 300, 90, 70], [40, 1, 1, 1]), ([300] * 20, [100] + [1] * 19), ([300] * 20, [1] * 19 + [290])])
def test_prompts_and_single_tokens_in_one_call(lengths, rows):
    """Sequences of many and of few rows, where the many decide the kernel and where they do not; one that does not fit is reported."""
    c = Case(44, lengths, rows, 8, 2, 64)
    c.check()
    c.check(last=3, fresh=True)
    good = host(c.run())
    c.lens[0] = -1
    st = status_tensor()
    got = host(c.run(st=st))
    assert st.tolist() == [3, 0] and np.array_equal(got[0], c.score[0]) and np.array_equal(got[1:], good[1:])


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("temps", [(np.nan, 1.0, 1.0), (np.nan, 1.0, 0.0), (0.0, 1.0, 1.0), (1.0, 1.0, 0.0), (1.0, 0.0, 0.5)])
def test_starts_that_give_a_row_to_two_sequences(many, temps):
    """A bad q_start is reported; what its neighbours answer stays within their rows and the vocabulary."""
    rng = np.random.default_rng(45)
    V, extra = 700, 310 if many else 0
    T = 6 + extra
    logits, draft = (dev(rng.normal(size=(T, V)).astype(np.float32)) for _ in range(2))
    tokens, uniform = dev(rng.integers(0, V, T).astype(np.int32)), dev(rng.random(T).astype(np.float32))
    q_start = dev(np.array([0, 5, 2, 6] + list(range(7, 7 + extra)), np.int32))
    S = 3 + extra
    temp = dev(np.array(list(temps) + [1.0] * extra, np.float32))
    for model in (None, draft):
        acc, nxt, n_new = (torch.full((S,), -77, dtype=torch.int32, device=DEV) for _ in range(3))
        ws, st = torch.full((moe.verify_workspace(T, S, V),), 255, dtype=torch.uint8, device=DEV), status_tensor()
        moe.moe_verify_drafts(logits, tokens, uniform, q_start, acc, nxt, n_new, draft_logits=model, temperature=temp, workspace=ws, st=st)
        a, n = host(acc), host(nxt)
        assert st.tolist()[0] != 0 and a[1] == 0 and n[1] == -1
        assert ((a >= 0) & (a <= 4)).all() and ((n >= -1) & (n < V)).all()
        if extra:
            want = _verify.verify(host(logits)[6:], host(tokens)[6:], host(uniform)[6:], np.arange(extra + 1), None, np.ones(extra, np.float32))
            assert np.array_equal(a[3:], want[0]) and np.array_equal(n[3:], want[1])
