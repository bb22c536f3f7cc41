"""KvPages.assign with scores: each sequence's scores are those of the tokens that it has."""
import pytest
import torch

import expert_routing_moe_gb300 as moe
from _gpu import DEV

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _pages(**kw):
    pages = moe.KvPages(1, 12, 2, 64, 3, 128, DEV, evicts=True)
    pages.reserve(_i32([100, 30, 7]))
    pages.score.copy_(torch.arange(1, 3 * 128 + 1, device=DEV).view(3, 128))
    return pages


@pytest.mark.parametrize("parent,source", [([1, 0, 0], [1, 0, 0]), ([3, 0, 0], [0, 0, 0]), ([2, -2, 1], [2, 1, 1]), ([2 ** 31 - 1, 2, 0], [0, 2, 0]), ([-2 ** 31, 0, 5], [0, 0, 2])])
@pytest.mark.parametrize("side", [False, True])
def test_a_refused_parent_keeps_its_own_sequence_alone(parent, source, side):
    """`source`: what each sequence becomes; the others move where one parent is refused."""
    pages = _pages()
    score, lens, table = pages.score.clone(), pages.seq_len.clone(), pages.page_table.clone()
    stream = torch.cuda.Stream() if side else None
    torch.cuda.synchronize()
    pages.assign(_i32(parent), stream)
    torch.cuda.synchronize()
    assert pages.seq_len.tolist() == lens[source].tolist() and torch.equal(pages.page_table, table[source])
    assert torch.equal(pages.score, score[source])
    assert (pages.device_status()[0] != 0) == any(not -1 <= p < 3 for p in parent)
