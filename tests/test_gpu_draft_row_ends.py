"""Verification with a drafting model's logits whose rows have large numbers beside
them: neither what lies between rows nor a neighbouring row's first numbers is drawn."""
import numpy as np
import pytest
import torch

import _verify
import expert_routing_moe_gb300 as moe
from _gpu import DEV, dev, host, status_tensor

pytestmark = pytest.mark.gpu


def _rows(a, dtype, shift, pad, beside):
    """Rows that start `shift` numbers into their memory, `pad` numbers apart, `beside` everywhere else."""
    T, V = a.shape
    buf = torch.full((T * (V + pad) + shift + 16,), beside, dtype=dtype, device=DEV)
    out = buf[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V]
    out.copy_(dev(a))
    return out


def _check(logits, draft, tokens, uniform, q_start, temp, dtype, target_at, draft_at, beside):
    """Answers equal the definition's; `_at`: (shift, pad) of the rows."""
    S, T, V = len(q_start) - 1, *logits.shape
    outs = [torch.full((S,), -77, dtype=torch.int32, device=DEV) for _ in range(3)]
    st = status_tensor()
    moe.moe_verify_drafts(_rows(logits, dtype, *target_at, beside), dev(tokens), dev(uniform), dev(np.asarray(q_start, np.int32)), *outs,
                          draft_logits=_rows(draft, dtype, *draft_at, beside), temperature=dev(temp), st=st)
    got, want = [host(o) for o in outs], _verify.verify(logits, tokens, uniform, q_start, draft, temp)
    assert (want[0] < np.diff(q_start) - 1).any()              # a draft is refused, so that max(p - q, 0) is drawn from
    assert ((got[1] >= 0) & (got[1] < V)).all()
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert st.tolist() == [0, 0]


def _case(rng, S, V, dtype, low=0.0):
    """Sequences of three rows whose first draft the target hardly takes."""
    T = 3 * S
    logits = rng.normal(size=(T, V)) + low
    draft = logits + 0.3 * rng.normal(size=(T, V))
    tokens = rng.integers(0, V, T)
    for s in range(S):
        draft[3 * s, tokens[3 * s + 1]] = draft[3 * s].max() + 1
        logits[3 * s, tokens[3 * s + 1]] = logits[3 * s].min() - 1
    logits, draft = (torch.from_numpy(a.astype(np.float32)).to(dtype).float().numpy() for a in (logits, draft))
    return logits, draft, tokens.astype(np.int32), rng.uniform(0.2, 1, T).astype(np.float32), np.arange(S + 1) * 3


@pytest.mark.parametrize("S,V", [(1, 5), (2, 101), (3, 5003), (90, 3001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("temperature,above", [(0.02, 4.0), (0.02, 40.0), (0.05, 10.0), (0.1, 20.0), (0.1, 4.0), (1.0, 200.0)])
def test_large_numbers_between_rows(S, V, dtype, temperature, above):
    rng = np.random.default_rng(S + V)
    logits, draft, tokens, uniform, q_start = _case(rng, S, V, dtype)
    beside = float(max(logits.max(), draft.max()) + above)
    temp = np.full(S, temperature, np.float32)
    # the rows of both tensors begin alike between 16-byte boundaries, then otherwise
    for target_at, draft_at in (((3, 2), (3, 2)), ((1, 4), (2, 3)), ((0, 1), (7, 1))):
        _check(logits, draft, tokens, uniform, q_start, temp, dtype, target_at, draft_at, beside)


@pytest.mark.parametrize("S,V", [(2, 7), (3, 1001), (120, 2003)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("temperature", [0.02, 0.1])
def test_large_numbers_in_the_next_row(S, V, dtype, temperature):
    """Rows without anything between them, each far above the one before."""
    rng = np.random.default_rng(S + V)
    logits, draft, tokens, uniform, q_start = _case(rng, S, V, dtype)
    up = (np.arange(3 * S) % 7 * 16.0)[:, None].astype(np.float32)
    logits, draft = (torch.from_numpy(a + up).to(dtype).float().numpy() for a in (logits, draft))
    temp = np.full(S, temperature, np.float32)
    for shift in (0, 1):
        _check(logits, draft, tokens, uniform, q_start, temp, dtype, (0, 0), (shift, 0), -5.0)


@pytest.mark.parametrize("S,V", [(1, 6), (3, 1000), (90, 3001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("temperature", [0.02, 0.1])
def test_rows_of_negative_numbers(S, V, dtype, temperature):
    """Zero would be far above every logit; the rows of both tensors begin otherwise between 16-byte boundaries."""
    rng = np.random.default_rng(S + V)
    logits, draft, tokens, uniform, q_start = _case(rng, S, V, dtype, low=-30.0)
    for target_at, draft_at in (((0, 0), (1, 0)), ((3, 0), (2, 5)), ((2, 1), (2, 1))):
        _check(logits, draft, tokens, uniform, q_start, np.full(S, temperature, np.float32), dtype, target_at, draft_at, 0.0)
