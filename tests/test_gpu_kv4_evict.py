"""Eviction on the GPU against the rules carried out one sequence at a time on the
host: every table, reference, score and byte is equal."""
import numpy as np
import pytest
import torch

import _kv4
import expert_routing_moe_gb300 as moe
from _gpu import DEV, dev, host, status_tensor

pytestmark = pytest.mark.gpu
PAGE = 64


class Host:
    """Tables, lengths, references, page contents and scores on the host."""

    def __init__(self, rng, lengths, layers, n_kv, D, columns=None, spare=4, shared=()):
        self.layers, self.n_kv, self.D = layers, n_kv, D
        self.len = np.array(lengths, np.int32)
        held = -(-self.len // PAGE)
        self.columns = max(held.max(), 1) + 1 if columns is None else columns
        n = int(held.sum()) + spare
        order = rng.permutation(n)
        self.table = np.full((len(lengths), self.columns), -1, np.int32)
        at = 0
        for s, k in enumerate(held):
            self.table[s, :k] = order[at:at + k]
            at += k
        self.ref = np.zeros(n, np.int32)
        self.ref[self.table[self.table >= 0]] = 1
        for s in shared:                     # sequences whose pages are held once more
            self.ref[self.table[s][self.table[s] >= 0]] += 1
        self.data = rng.integers(0, 256, (layers, n, n_kv, PAGE * (D + D // 8)), dtype=np.uint8)
        self.score = rng.random((len(lengths), self.columns * PAGE + 1)).astype(np.float32)
        self.kept = None

    def evict(self, budget, sinks, recent, width=None):
        """The rules of moe_kv4_evict; the status that it reports."""
        S = len(self.len)
        plans, drop, take = {}, [], []
        for s in range(S):
            n, b = int(self.len[s]), int(budget[s])
            if n < 0 or n > self.columns * PAGE:
                return 3, s
            if not 0 <= b < n:
                continue
            if sinks + recent > b or any(not 0 <= p < len(self.ref) for p in self.table[s, :-(-n // PAGE)]):
                return 3, s
        for s in range(S):
            n, b = int(self.len[s]), int(budget[s])
            if not 0 <= b < n:
                continue
            x = self.score[s, :n].astype(np.float64)
            x = np.where(np.isnan(x), -np.inf, x)
            nan = np.isnan(self.score[s, :n])
            middle = np.arange(sinks, n - recent)
            best = sorted(middle, key=lambda j: (-x[j], nan[j], j))[:b - sinks - recent]
            keep = np.zeros(n, bool)
            keep[:sinks] = keep[n - recent:] = True
            keep[best] = True
            plans[s] = np.nonzero(keep)[0]
        free = [p for p in range(len(self.ref)) if self.ref[p] == 0]
        writes = []
        for s, kept in plans.items():
            first = int(np.nonzero(np.r_[kept, -1] != np.arange(len(kept) + 1))[0][0]) // PAGE
            for c in range(first, -(-len(kept) // PAGE)):
                old = int(self.table[s, c])
                writes.append((s, c, old, self.ref[old] > 1))
        want = sum(w[3] for w in writes)
        if want > len(free):
            return 4, want - len(free)
        old_data, old_table, old_score = self.data.copy(), self.table.copy(), self.score.copy()
        kc, ks, vc, vs = _kv4.places(self.D)
        for s, c, old, shared in writes:
            page = free.pop(0) if shared else old
            if shared:
                drop.append(old)
                take.append(page)
                self.table[s, c] = page
            new = np.zeros_like(self.data[:, page])
            for i in range(PAGE):
                k = c * PAGE + i
                if k >= len(plans[s]):
                    break
                j = int(plans[s][k])
                src = old_data[:, old_table[s, j // PAGE]]
                o = j % PAGE
                new[..., kc[i]] = src[..., kc[o]]
                new[..., ks[i]] = src[..., ks[o]]
                new[..., vs[i]] = src[..., vs[o]]
                new[..., vc[i]] |= ((src[..., vc[o]] >> (4 * (o & 1))) & 15) << (4 * (i & 1))
            self.data[:, page] = new
        for s, kept in plans.items():
            n = int(self.len[s])
            for c in range(-(-len(kept) // PAGE), -(-n // PAGE)):
                drop.append(int(old_table[s, c]))
                self.table[s, c] = -1
            self.score[s, :n] = 0
            self.score[s, :len(kept)] = old_score[s, kept]
            self.len[s] = len(kept)
        for p in drop:
            self.ref[p] -= 1
        for p in take:
            self.ref[p] = 1
        if width is not None:
            self.kept = np.full((S, width), -1, np.int32)
            for s in range(S):
                k = plans.get(s, np.arange(self.len[s]))[:width]
                self.kept[s, :len(k)] = k
        return 0, 0


class Gpu:
    def __init__(self, h):
        self.table, self.len, self.ref, self.pages, self.score = dev(h.table), dev(h.len), dev(h.ref), dev(h.data), dev(h.score)
        self.pool = moe.Kv4Pool(self.pages, self.table, self.len, self.ref, h.D)
        self.ws = torch.full((moe.kv4_evict_workspace(self.pool),), 255, dtype=torch.uint8, device=DEV)
        self.st = status_tensor()

    def evict(self, budget, sinks, recent, kept=None):
        moe.moe_kv4_evict(self.pool, self.score, dev(np.asarray(budget, np.int32)), sinks, recent, self.ws, kept, self.st)

    def same(self, h):
        for mine, theirs, what in ((self.len, h.len, "len"), (self.table, h.table, "table"), (self.ref, h.ref, "ref"), (self.score, h.score, "score"), (self.pages, h.data, "pages")):
            assert np.array_equal(host(mine), theirs, equal_nan=what == "score"), what


def _both(h, budget, sinks, recent, width=50):
    g = Gpu(h)
    kept = torch.full((len(h.len), width), -9, dtype=torch.int32, device=DEV)
    g.evict(budget, sinks, recent, kept)
    code = h.evict(budget, sinks, recent, width)
    assert g.st.tolist() == list(code)
    g.same(h)
    if code[0] == 0:
        assert np.array_equal(host(kept), h.kept)
    else:
        assert (kept == -9).all()
    return g


@pytest.mark.parametrize("D,n_kv,layers", [(64, 1, 1), (64, 3, 2), (128, 2, 3)])
@pytest.mark.parametrize("lengths,budget,sinks,recent", [
    ([1], [0], 0, 0), ([2], [1], 0, 1), ([64], [63], 0, 0), ([65], [64], 4, 10), ([130, 0, 64], [65, 0, 64], 1, 1), ([200, 300, 17], [100, -1, 30], 4, 20),
    ([1000], [200], 70, 64), ([1500, 700, 129, 5], [1000, 64, 128, 4], 0, 0), ([900, 900], [0, 899], 0, 0), ([300, 600], [299, 100], 50, 50), ([2000], [150], 150, 0),
    ([2000], [150], 0, 150), ([2000], [150], 100, 50)])
@pytest.mark.parametrize("shared", [False, True])
def test_equals_the_rules(D, n_kv, layers, lengths, budget, sinks, recent, shared):
    rng = np.random.default_rng(sum(lengths) + D)
    h = Host(rng, lengths, layers, n_kv, D, spare=40 if shared else 0, shared=range(0, len(lengths), 2) if shared else ())
    if shared and len(lengths) > 1:          # some pages are shared, some not
        h.ref[h.table[1][h.table[1] >= 0][::2]] += 3
    _both(h, budget, sinks, recent)


def test_again_and_again():
    """Growing and evicting in turn, scores of every kind."""
    rng = np.random.default_rng(1)
    h = Host(rng, [500, 333, 64, 1000, 0], 2, 2, 64, columns=20, spare=30)
    for step in range(6):
        kind = step % 3
        if kind == 1:
            h.score[:] = rng.integers(0, 3, h.score.shape)                                 # many equal ones
        elif kind == 2:
            h.score[:] = rng.choice(np.array([np.nan, np.inf, -np.inf, -1, -0.0, 0.0, 1e-40, 3], np.float32), h.score.shape)
        budget = [int(n) - int(rng.integers(0, 90)) for n in h.len]     # a negative one: it stays
        sinks = 2 if all(b < 0 or b >= 7 for b in budget) else 0
        _both(h, budget, sinks, 5 if sinks else 0)


def test_a_nan_is_lowest_and_equal_ones_go_by_place():
    rng = np.random.default_rng(2)
    h = Host(rng, [70], 1, 1, 64)
    h.score[0, :70] = 1
    h.score[0, [3, 60]] = np.nan
    h.score[0, [5, 6]] = -np.inf
    h.score[0, [8, 9]] = [-0.0, 0.0]
    _both(h, [66], 0, 0, 70)
    assert h.kept[0].tolist() == [j for j in range(70) if j not in (3, 5, 6, 60)] + [-1] * 4
    h = Host(rng, [70], 1, 1, 64)
    h.score[0, :70] = 1
    _both(h, [10], 0, 0, 10)
    assert h.kept[0].tolist() == list(range(10))


def test_long_sequence():
    rng = np.random.default_rng(3)
    h = Host(rng, [20000, 5000], 1, 1, 64)
    _both(h, [9000, 4999], 4, 100, 9000)


def test_many_sequences():
    rng = np.random.default_rng(4)
    lengths = rng.integers(0, 200, 1500)
    h = Host(rng, lengths, 1, 1, 64, spare=200, shared=range(0, 1500, 40))
    _both(h, np.where(rng.random(1500) < 0.3, -1, rng.integers(10, 150, 1500)), 3, 7)


def test_all_or_nothing():
    rng = np.random.default_rng(5)
    h = Host(rng, [300, 200], 2, 1, 64, spare=2, shared=[0])
    _both(h, [190, 100], 0, 0)                            # three free pages wanted, two there
    assert h.ref.max() == 2 and h.len.tolist() == [300, 200]
    _both(h, [128, 100], 0, 0)                            # two will do
    h = Host(rng, [300, 200], 2, 1, 64)
    for budget, sinks, recent in (([299, 99], 50, 50), ([299, 99], 2 ** 31 - 1, 2 ** 31 - 1)):
        _both(h, budget, sinks, recent)                   # below sinks + recent: of the second (or both)
    for bad in (-1, 9999, len(h.ref)):
        keep = h.table[1, 3]
        h.table[1, 3] = bad
        g = Gpu(h)
        g.evict([100, 100], 0, 0)
        assert g.st.tolist() == [3, 1]
        g.same(h)
        h.table[1, 3] = keep
    for bad in (-1, h.columns * PAGE + 1, 2 ** 31 - 1):
        keep = h.len[0]
        h.len[0] = bad
        g = Gpu(h)
        g.evict([100, 100], 0, 0)
        assert g.st.tolist() == [3, 0]
        g.same(h)
        h.len[0] = keep
    _both(h, [100, 100], 4, 4)


def test_two_sequences_that_share_pages():
    """A fork: both evict, and neither sees the other's writes."""
    rng = np.random.default_rng(6)
    h = Host(rng, [256, 256, 100], 2, 2, 64, spare=12)
    h.ref[h.table[1, :4]] = 0
    h.table[1, :4] = h.table[0, :4]
    h.ref[h.table[0, :4]] = 2
    _both(h, [130, 70, 50], 1, 2)


def test_captured_with_a_shared_workspace():
    """Two graphs on pools of different sizes use one workspace in turn."""
    rng = np.random.default_rng(7)
    hosts = [Host(rng, [300, 500], 2, 1, 64, spare=3), Host(rng, [100, 90, 700, 64], 1, 2, 128, spare=9)]
    gpus = [Gpu(h) for h in hosts]
    ws = max((g.ws for g in gpus), key=lambda w: w.numel())
    budgets = [dev(np.array([200, 200], np.int32)), dev(np.array([50, 90, 300, 10], np.int32))]
    graphs = []
    for g, b in zip(gpus, budgets):
        g.ws = ws
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_kv4_evict(g.pool, g.score, b, 2, 3, ws, None, g.st)
        graphs.append(graph)
    for turn in range(3):
        for g, h, b, graph in zip(gpus, hosts, budgets, graphs):
            b.sub_(10 * turn).clamp_(min=5)
            graph.replay()
            assert h.evict(host(b), 2, 3) == (0, 0)
            g.same(h)
            assert g.st.tolist() == [0, 0]


def test_binding_refuses():
    h = Host(np.random.default_rng(8), [100], 1, 1, 64)
    g = Gpu(h)
    budget = dev(np.array([10], np.int32))
    with pytest.raises(moe.MoeError, match="score"):
        moe.moe_kv4_evict(g.pool, g.score[:, :191], budget, 0, 0, g.ws)
    with pytest.raises(moe.MoeError, match="budget"):
        moe.moe_kv4_evict(g.pool, g.score, dev(np.array([1, 2], np.int32)), 0, 0, g.ws)
    with pytest.raises(moe.MoeError, match="kept"):
        moe.moe_kv4_evict(g.pool, g.score, budget, 0, 0, g.ws, torch.zeros(2, 4, dtype=torch.int32, device=DEV))
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_kv4_evict(g.pool, g.score, budget, 0, 0, g.ws[:64])
    with pytest.raises(moe.MoeError, match="invalid"):
        moe.moe_kv4_evict(g.pool, g.score, budget, -1, 0, g.ws)
    g.same(h)
