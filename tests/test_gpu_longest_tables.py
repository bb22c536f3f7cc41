"""Tables of as many tokens as there can be, 64 less than 2^31: every entry names one page, so that what is
read fits the device."""
import numpy as np
import pytest
import torch

import _kv4
import expert_routing_moe_gb300 as moe
from _gpu import DEV, dev, host, status_tensor

pytestmark = pytest.mark.gpu
PAGE, D = 64, 64
COLUMNS = 2 ** 25 - 1
TOKENS = COLUMNS * PAGE


def _moved(page, kept):
    """Bytes of the page of tokens that had the places `kept` of sequences whose every page is `page`."""
    kc, ks, vc, vs = _kv4.places(D)
    new = np.zeros_like(page)
    for i, j in enumerate(np.asarray(kept) % PAGE):
        new[kc[i]], new[ks[i]], new[vs[i]] = page[kc[j]], page[ks[j]], page[vs[j]]
        new[vc[i]] |= ((page[vc[j]] >> np.uint8(4 * (j & 1))) & np.uint8(15)) << np.uint8(4 * (i & 1))
    return new


@pytest.mark.parametrize("end", [False, True])
def test_eviction(end):
    """Most of the longest sequence goes, or some of its last tokens."""
    if torch.cuda.mem_get_info()[0] < 30e9:
        pytest.skip("needs 30 GB")
    rng = np.random.default_rng(end)
    data = rng.integers(0, 256, (1, 10, 1, PAGE * (D + D // 8)), dtype=np.uint8)
    pages = dev(data)
    table = torch.full((1, COLUMNS), 2, dtype=torch.int32, device=DEV)
    length = torch.full((1,), TOKENS, dtype=torch.int32, device=DEV)
    ref = torch.zeros(10, dtype=torch.int32, device=DEV)
    ref[2] = COLUMNS
    pool = moe.Kv4Pool(pages, table, length, ref, D)
    score = torch.zeros(1, TOKENS, device=DEV)
    if end:
        sinks, recent, gone = TOKENS - 300, 100, 100
        best = np.sort(rng.choice(np.arange(sinks, TOKENS - recent), 200 - gone, replace=False))
        budget = TOKENS - gone
    else:
        sinks, recent, budget = 70, 70, 200
        best = np.unique(np.r_[rng.integers(70, TOKENS - 70, 58), 70, TOKENS - 71])
        assert len(best) == 60
    score[0, dev(best)] = 1 + torch.arange(len(best), device=DEV, dtype=torch.float32)
    ws, st = torch.empty(moe.kv4_evict_workspace(pool), dtype=torch.uint8, device=DEV), status_tensor()
    moe.moe_kv4_evict(pool, score, torch.full((1,), budget, dtype=torch.int32, device=DEV), sinks, recent, ws, None, st)
    assert st.tolist() == [0, 0] and length.tolist() == [budget]
    # the kept places from page `first` on, where the table changes
    first = (sinks + int((best != sinks + np.arange(len(best))).argmax())) // PAGE if end else 1
    tail = np.r_[np.arange(first * PAGE, sinks), best, np.arange(TOKENS - recent, TOKENS)]
    n = -(-len(tail) // PAGE)
    names = [p for p in range(10) if p != 2][:n]
    assert host(table[0, first:first + n]).tolist() == names and (table[0, :first] == 2).all() and (table[0, first + n:] == -1).all()
    want = np.zeros(10, np.int32)
    want[2], want[names] = first, 1
    assert np.array_equal(host(ref), want)
    got = host(pages)[0, :, 0]
    for i, p in enumerate(names):
        assert np.array_equal(got[p], _moved(data[0, 2, 0], tail[i * PAGE:(i + 1) * PAGE]))
    left = [p for p in range(10) if p not in names]
    assert np.array_equal(got[left], data[0, left, 0])
    at = sinks + torch.arange(len(best), device=DEV)
    assert torch.equal(score[0, at], 1 + torch.arange(len(best), device=DEV, dtype=torch.float32))
    assert int(torch.count_nonzero(score)) == len(best)


def test_weighing():
    if torch.cuda.mem_get_info()[0] < 30e9:
        pytest.skip("needs 30 GB")
    rng = np.random.default_rng(2)
    ref = _kv4.Cache(rng, [PAGE], 1, D, False)
    page = int(ref.table[0, 0])
    pages, q = dev(ref.bytes), torch.randn(1, 2, D, device=DEV).bfloat16()
    q_start, lse = dev(np.array([0, 1], np.int32)), torch.full((1, 2), 3.0, device=DEV)

    def run(columns, length):
        table = torch.full((1, columns), page, dtype=torch.int32, device=DEV)
        cache = moe.Kv4Cache(pages, table, torch.full((1,), length, dtype=torch.int32, device=DEV), D, None, None)
        score, st = torch.zeros(1, columns * PAGE, device=DEV), status_tensor()
        moe.moe_kv4_weigh(q, cache, q_start, lse, score, 0.125, 1, st=st)
        assert st.tolist() == [0, 0]
        return score

    one = run(1, PAGE)
    assert (one > 0).all()
    score = run(COLUMNS, TOKENS)
    assert bool((score.view(COLUMNS, PAGE) == one).all())
