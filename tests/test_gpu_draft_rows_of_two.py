"""Verification where bad starts give rows to two sequences that are far apart in the
batch: the rows are the first one's, at every call, and the other one has an answer
only if it takes them in the same way."""
import numpy as np
import pytest
import torch

import _verify
import expert_routing_moe_gb300 as moe
from _gpu import DEV, dev, host, status_tensor

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,extra", [(700, 0), (40000, 0), (700, 400), (40000, 60)])
@pytest.mark.parametrize("between", [1, 40, 700])
@pytest.mark.parametrize("temps", [(1.0, 1.0), (0.0, 0.0), (0.5, 1.0), (0.0, 1.0), (1.0, 0.0), (np.nan, 1.0), (np.nan, 0.0), (1.0, np.nan)])
@pytest.mark.parametrize("by_model", [False, True])
def test_the_first_sequence_has_the_rows(V, extra, between, temps, by_model):
    rng = np.random.default_rng(V + extra + between)
    T = 6 + extra
    logits = (rng.normal(size=(T, V)) * 3).astype(np.float32)
    draft = logits + rng.normal(size=(T, V)).astype(np.float32)
    tokens, uniform = draft.argmax(1).astype(np.int32), rng.random(T).astype(np.float32)
    tokens[1:] = tokens[:-1].copy()
    # rows 0 .. 4, a sequence that ends before it starts, empty ones, rows 2 .. 5, then one each
    q_start = np.array([0, 5] + [2] * between + [6] + list(range(7, 7 + extra)), np.int32)
    S, other = len(q_start) - 1, 1 + between
    temp = np.ones(S, np.float32)
    temp[0], temp[other] = temps
    of = lambda a, b, t: [int(v[0]) for v in _verify.verify(logits[a:b], tokens[a:b], uniform[a:b], [0, b - a], draft[a:b] if by_model else None, [t])]  # noqa: E731
    want0, want_other = of(0, 5, temps[0]), of(2, 6, temps[1])
    if temps[0] != temps[1]:
        want_other = [0, -1, -3]
    rest = _verify.verify(logits[6:], tokens[6:], uniform[6:], np.arange(extra + 1), draft[6:] if by_model else None, np.ones(extra)) if extra else None
    on = [dev(a) for a in (logits, tokens, uniform, q_start)]
    model, temp = dev(draft) if by_model else None, dev(temp)
    for _ in range(10):
        outs = [torch.full((S,), -77, dtype=torch.int32, device=DEV) for _ in range(3)]
        st = status_tensor()
        ws = torch.full((moe.verify_workspace(T, S, V),), 255, dtype=torch.uint8, device=DEV)
        moe.moe_verify_drafts(*on, *outs, draft_logits=model, temperature=temp, workspace=ws, st=st)
        got = [host(o) for o in outs]
        assert st.tolist()[0] != 0
        assert [int(g[0]) for g in got] == want0 and [int(g[other]) for g in got] == want_other
        assert (got[0][1:other] == 0).all() and (got[1][1:other] == -1).all()
        if extra:
            for g, w in zip(got, rest):
                assert np.array_equal(g[other + 1:], w)
