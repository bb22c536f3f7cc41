"""Steps that are only tried: snapshot, restore and release of the pages."""
import pytest
import torch

import expert_routing_moe_gb300 as moe
from _gpu import DEV

pytestmark = pytest.mark.gpu
NKV, D, COLS = 2, 64, 4


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Server:
    def __init__(self, lengths, n_pages):
        self.g = torch.Generator(device=DEV).manual_seed(len(lengths))
        self.S = len(lengths)
        self.pages = moe.KvPages(1, n_pages, NKV, D, self.S, COLS * 64, DEV)
        self.cache = self.pages.layer(0)
        self.grow(lengths)

    def grow(self, n_new):
        """Room for n_new tokens (negative: fewer) and random ones appended."""
        self.pages.reserve(_i32(n_new))
        new = [max(0, n) for n in n_new]
        T = sum(new)
        if T:
            x = torch.randn(T, 2 * NKV * D, generator=self.g, device=DEV).bfloat16()
            starts = _i32([sum(new[:i]) for i in range(self.S + 1)])
            moe.moe_qk_norm_rope(x, 0, NKV, None, cache=self.cache, q_start=starts, st=self.pages.status)

    def read(self):
        """Every sequence's tokens, and the tables."""
        n = self.pages.seq_len.tolist()
        k, v = (torch.empty(max(1, sum(n)), NKV, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        moe.moe_kv4_read(self.cache, _i32([sum(n[:i]) for i in range(self.S + 1)]), k, v, self.pages.status)
        assert self.pages.device_status() == (0, 0)
        return n, k, v, self.pages.book.clone()


def _same(a, b):
    return a[0] == b[0] and all(torch.equal(x, y) for x, y in zip(a[1:], b[1:]))


STEPS = {
    "grow": lambda s: s.grow([3, 1, 70]),
    "drop one, fork another": lambda s: (s.pages.assign(_i32([0, 0, 2])), s.grow([2, 1, 1]), s.grow([1, 1, 60])),
    "drop all and start again": lambda s: (s.pages.assign(_i32([-1, -1, -1])), s.grow([130, 64, 20])),
    "truncate and grow": lambda s: (s.grow([-40, -90, -5]), s.grow([60, 80, 3])),
}


@pytest.mark.parametrize("step", list(STEPS))
@pytest.mark.parametrize("lengths", [[100, 93, 64], [33, 128, 1]])
def test_restore_brings_back_every_token(step, lengths):
    s = Server(lengths, 24)
    before = s.read()
    saved = s.pages.snapshot()
    STEPS[step](s)
    s.pages.restore(saved)
    assert _same(s.read(), before)
    # and the server goes on as one that never tried
    other = Server(lengths, 24)
    other.g.set_state(s.g.get_state())
    s.grow([1, 66, 2])
    other.grow([1, 66, 2])
    assert _same(s.read(), other.read())


def test_nested_trials():
    s = Server([70, 40, 10], 24)
    first = s.read()
    a = s.pages.snapshot()
    STEPS["drop one, fork another"](s)
    second = s.read()
    b = s.pages.snapshot()
    STEPS["drop all and start again"](s)
    s.pages.restore(b)
    got = s.read()
    assert _same(got[:3], second[:3]) and torch.equal(s.pages.page_table.flatten(), second[3][:3 * COLS])
    s.pages.restore(a)
    assert _same(s.read(), first)


def test_release_keeps_the_step():
    s = Server([100, 93, 64], 24)
    saved = s.pages.snapshot()
    STEPS["drop one, fork another"](s)
    kept = s.read()
    with pytest.raises(moe.MoeError, match="snapshot"):
        s.pages.compact()
    s.pages.release(saved)
    assert _same(s.read()[:3], kept[:3])
    # every page is held by the entries that name it, and by nothing else
    table = s.pages.page_table[s.pages.page_table >= 0].long()
    assert torch.equal(s.pages.ref, torch.bincount(table, minlength=24).int())
    live = int(s.pages.compact())
    assert live == table.unique().numel() and _same(s.read()[:3], kept[:3])


def test_a_table_with_pages_outside_the_pool():
    s = Server([10, 0, 0], 4)
    s.pages.page_table[1, 0], s.pages.page_table[2, 1] = 4, 1 << 30
    saved = s.pages.snapshot()
    assert s.pages.ref.tolist() == [2, 0, 0, 0]
    s.pages.restore(saved)
    assert s.pages.ref.tolist() == [1, 0, 0, 0]


def test_a_snapshot_ends_once_and_in_order():
    s = Server([70, 40, 10], 24)
    first = s.read()
    a, b = s.pages.snapshot(), s.pages.snapshot()
    for end in (s.pages.restore, s.pages.release):
        with pytest.raises(moe.MoeError, match="last one first"):
            end(a)
    s.pages.release(b)
    with pytest.raises(moe.MoeError, match="once"):
        s.pages.release(b)
    s.pages.restore(a)
    assert _same(s.read(), first) and int(s.pages.compact()) == 4
