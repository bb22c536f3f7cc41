"""The cache's pages on the GPU against the rules carried out one sequence at
a time on the host."""
import numpy as np
import pytest
import torch

import expert_routing_moe_gb300 as moe
from _gpu import DEV, status_tensor

pytestmark = pytest.mark.gpu
PAGE = 64


class Book:
    """Tables, lengths, references and page contents on the host."""

    def __init__(self, S, columns, n_pages, layers, page_bytes, rng):
        self.table = np.full((S, columns), -1, np.int32)
        self.len = np.zeros(S, np.int32)
        self.ref = np.zeros(n_pages, np.int32)
        self.data = rng.integers(0, 256, (layers, n_pages, page_bytes), dtype=np.uint8)

    def reserve(self, n_new):
        """The rules of moe_kv4_reserve; the status word that it reports."""
        S, columns = self.table.shape
        for s in range(S):
            if self.len[s] + int(n_new[s]) > columns * PAGE:
                return 3
        grows = [s for s in range(S) if n_new[s] > 0 and self.len[s] % PAGE]
        last = {s: int(self.table[s, self.len[s] // PAGE]) for s in grows}
        copies = []
        for s in grows:
            sharers = [x for x in grows if last[x] == last[s]]
            if self.ref[last[s]] > 1 and not (len(sharers) == self.ref[last[s]] and s == sharers[-1]):
                copies.append(s)
        need = {s: -(-(self.len[s] + n_new[s]) // PAGE) - -(-self.len[s] // PAGE) if n_new[s] > 0 else 0 for s in range(S)}
        free = [p for p in range(len(self.ref)) if self.ref[p] == 0]
        if len(copies) + sum(need.values()) > len(free):
            return 4
        drop = []
        for s in range(S):
            if s in copies:
                p = free.pop(0)
                self.data[:, p] = self.data[:, last[s]]
                drop.append(last[s])
                self.ref[p] = 1
                self.table[s, self.len[s] // PAGE] = p
            held = -(-self.len[s] // PAGE)
            for c in range(need[s]):
                p = free.pop(0)
                self.ref[p] = 1
                self.table[s, held + c] = p
            after = max(0, int(self.len[s]) + int(n_new[s]))
            for c in range(-(-after // PAGE), held):
                drop.append(int(self.table[s, c]))
                self.table[s, c] = -1
            self.len[s] = after
        for p in drop:
            self.ref[p] -= 1
        return 0

    def assign(self, parent):
        table, length = self.table.copy(), self.len.copy()
        for s, p in enumerate(parent):
            if p == s:
                continue
            for g in table[s][table[s] >= 0]:
                self.ref[g] -= 1
            self.table[s] = table[p] if p >= 0 else -1
            self.len[s] = length[p] if p >= 0 else 0
            for g in self.table[s][self.table[s] >= 0]:
                self.ref[g] += 1

    def compact(self):
        n = int((self.ref != 0).sum())
        src = [p for p in range(n, len(self.ref)) if self.ref[p]]
        dst = [p for p in range(n) if not self.ref[p]]
        for a, b in zip(src, dst):
            self.data[:, b] = self.data[:, a]
            self.ref[b], self.ref[a] = self.ref[a], 0
            self.table[self.table == a] = b
        return n


class Gpu:
    def __init__(self, b, D, n_kv):
        t = lambda a: torch.from_numpy(a.copy()).to(DEV)  # noqa: E731
        self.table, self.len, self.ref = t(b.table), t(b.len), t(b.ref)
        self.pages = t(b.data).view(b.data.shape[0], b.data.shape[1], n_kv, -1)
        self.pool = moe.Kv4Pool(self.pages, self.table, self.len, self.ref, D)
        self.ws = torch.zeros(moe.kv4_pool_workspace(self.pool), dtype=torch.uint8, device=DEV)
        self.st = status_tensor()

    def same(self, b):
        torch.cuda.synchronize()
        assert np.array_equal(self.table.cpu().numpy(), b.table)
        assert np.array_equal(self.len.cpu().numpy(), b.len)
        assert np.array_equal(self.ref.cpu().numpy(), b.ref)
        assert np.array_equal(self.pages.cpu().numpy().reshape(b.data.shape), b.data)


def _vec(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("S,columns,n_pages,layers,n_kv,D", [(1, 3, 4, 1, 1, 64), (7, 9, 40, 3, 2, 64), (64, 17, 300, 2, 4, 128),
                                                             (1500, 5, 5000, 1, 1, 64)])
def test_a_day_in_the_life(S, columns, n_pages, layers, n_kv, D):
    """Random growing, truncating, forking, freeing and packing; every step equals the host's."""
    rng = np.random.default_rng(S)
    b = Book(S, columns, n_pages, layers, n_kv * PAGE * (D + D // 8), rng)
    g = Gpu(b, D, n_kv)
    for step in range(12):
        kind = ["reserve", "assign", "reserve", "compact"][step % 4]
        if kind == "reserve":
            room = columns * PAGE - b.len
            add = np.minimum(rng.integers(0, 90, S), room)
            if step:
                add = np.where(rng.random(S) < 0.3, -rng.integers(0, 130, S), add)
            add = np.where(rng.random(S) < 0.2, 0, add).astype(np.int32)
            g.st.zero_()
            moe.moe_kv4_reserve(g.pool, _vec(add), g.ws, g.st)
            assert g.st.tolist()[0] == b.reserve(add)
        elif kind == "assign":
            parent = np.where(rng.random(S) < 0.4, rng.integers(-1, S, S), np.arange(S))
            moe.moe_kv4_assign(g.pool, _vec(parent), g.st)
            b.assign(parent)
        else:
            live = torch.zeros(1, dtype=torch.int32, device=DEV)
            moe.moe_kv4_compact(g.pool, live, g.ws, g.st)
            assert int(live) == b.compact()
        g.same(b)
        assert (b.ref >= 0).all()


def _filled(lengths, columns, n_pages, rng, layers=2):
    b = Book(len(lengths), columns, n_pages, layers, PAGE * 72, rng)
    assert b.reserve(np.array(lengths)) == 0
    return b


def test_copy_on_write_rules():
    rng = np.random.default_rng(1)
    b = _filled([100, 0, 0, 0, 64], 4, 20, rng)
    b.assign(np.array([0, 0, 0, 0, 4]))
    g = Gpu(b, 64, 1)
    assert b.ref[b.table[0, 1]] == 4
    # two of four sharers grow: both copy
    add = np.array([1, 1, 0, 0, 1])
    moe.moe_kv4_reserve(g.pool, _vec(add), g.ws, g.st)
    assert b.reserve(add) == 0
    g.same(b)
    # the two that are left: the first copies, the last keeps
    last = b.table[3, 1]
    add = np.array([0, 0, 1, 30, 0])
    moe.moe_kv4_reserve(g.pool, _vec(add), g.ws, g.st)
    assert b.reserve(add) == 0
    g.same(b)
    assert b.table[3, 1] == last and b.table[2, 1] != last
    # a reference of the caller's own keeps the page from changing
    p = b.table[3, 2 if b.len[3] > 128 else 1]
    b.ref[p] += 1
    g.ref[int(p)] += 1
    add = np.array([0, 0, 0, 1, 0])
    moe.moe_kv4_reserve(g.pool, _vec(add), g.ws, g.st)
    assert b.reserve(add) == 0
    g.same(b)
    assert b.ref[p] == 1


def test_all_or_nothing():
    rng = np.random.default_rng(2)
    b = _filled([100, 60, 0], 3, 5, rng)
    g = Gpu(b, 64, 1)
    moe.moe_kv4_reserve(g.pool, _vec([-100, 0, 192]), g.ws, g.st)      # 3 wanted, 2 free (those of the call itself do not count)
    assert g.st.tolist() == [4, 1]
    g.same(b)
    g.st.zero_()
    moe.moe_kv4_reserve(g.pool, _vec([1, 1, 193]), g.ws, g.st)         # beyond the table
    assert g.st.tolist() == [3, 2]
    g.same(b)
    g.st.zero_()
    moe.moe_kv4_reserve(g.pool, _vec([2147483647, 0, 0]), g.ws, g.st)
    assert g.st.tolist() == [3, 0]
    g.same(b)
    # a table that names a page outside the pool
    keep = int(g.table[0, 1])
    for bad in (-1, 5, 1 << 30):
        for add in ([1, 1, 1], [-80, 0, 1]):
            g.table[0, 1] = bad
            g.st.zero_()
            moe.moe_kv4_reserve(g.pool, _vec(add), g.ws, g.st)
            assert g.st.tolist() == [3, 0]
            g.table[0, 1] = keep
            g.same(b)
    # and the workspace is as good as new
    g.st.zero_()
    moe.moe_kv4_reserve(g.pool, _vec([1, -60, 5]), g.ws, g.st)
    assert g.st.tolist() == [0, 0] and b.reserve(np.array([1, -60, 5])) == 0
    g.same(b)


def test_assign_cycles_and_bad_parents():
    rng = np.random.default_rng(3)
    b = _filled([70, 130, 10, 0], 4, 12, rng)
    g = Gpu(b, 64, 1)
    for parent in ([1, 2, 0, 3], [3, 3, 3, 3], [0, 1, 2, -1]):
        moe.moe_kv4_assign(g.pool, _vec(parent), g.st)
        b.assign(np.array(parent))
        g.same(b)
    assert g.st.tolist() == [0, 0]
    moe.moe_kv4_assign(g.pool, _vec([-2, 1, 4, 3]), g.st)
    assert g.st.tolist()[0] == 3
    g.same(b)


def test_compact_edges():
    rng = np.random.default_rng(4)
    b = _filled([0, 0], 2, 7, rng)                  # nothing in use
    g = Gpu(b, 64, 1)
    moe.moe_kv4_compact(g.pool, None, g.ws, g.st)
    g.same(b)
    b = _filled([128, 65], 2, 4, rng)               # all in use
    g = Gpu(b, 64, 1)
    moe.moe_kv4_compact(g.pool, None, g.ws, g.st)
    g.same(b)
    # only the last page, held outside any table
    b = Book(1, 1, 3000, 1, PAGE * 72, rng)
    b.ref[2999] = 5
    g = Gpu(b, 64, 1)
    live = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_kv4_compact(g.pool, live, g.ws, g.st)
    assert int(live) == b.compact() == 1 and b.ref[0] == 5
    g.same(b)


def test_capture():
    rng = np.random.default_rng(5)
    b = _filled([100, 30, 64], 4, 30, rng)
    g = Gpu(b, 64, 1)
    add, parent = _vec([1, 1, 1]), _vec([0, 0, 2])
    # the replays below count, the calls that warm up do not
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_kv4_assign(g.pool, parent, g.st)
        moe.moe_kv4_reserve(g.pool, add, g.ws, g.st)
        moe.moe_kv4_compact(g.pool, None, g.ws, g.st)
    for _ in range(3):
        graph.replay()
        b.assign(np.array([0, 0, 2]))
        assert b.reserve(np.array([1, 1, 1])) == 0
        b.compact()
        g.same(b)


def test_binding_refuses():
    rng = np.random.default_rng(6)
    g = Gpu(_filled([10], 2, 4, rng), 64, 1)
    with pytest.raises(moe.MoeError, match="n_new"):
        moe.moe_kv4_reserve(g.pool, _vec([1, 2]), g.ws)
    with pytest.raises(moe.MoeError, match="parent"):
        moe.moe_kv4_assign(g.pool, _vec([0]).long())
    with pytest.raises(moe.MoeError, match="workspace"):
        moe.moe_kv4_compact(g.pool, None, g.ws[:16])
