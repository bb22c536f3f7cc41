"""Verification of drafted tokens on the GPU: every decision equals the plain
implementation's (tests/_verify.py), whose whole numbers do not depend on an order."""
import math

import numpy as np
import pytest
import torch

import _verify
import expert_routing_moe_gb300 as moe
from _gpu import DEV, dev, host, status_tensor

pytestmark = pytest.mark.gpu


def _run(logits, tokens, uniform, q_start, draft=None, temperature=None, dtype=torch.float32, shift=0, pad=0, st=None, ws=None):
    """Through the binding; rows start `shift` numbers into their memory and have `pad` numbers between them."""
    def place(a):
        T, V = a.shape
        buf = torch.full((T * (V + pad) + shift + 8,), float("nan"), dtype=dtype, device=DEV)
        out = buf[shift:shift + T * (V + pad)].view(T, V + pad)[:, :V]
        out.copy_(dev(a))
        return out
    S = len(q_start) - 1
    acc, nxt, n_new = (torch.full((S,), -77, dtype=torch.int32, device=DEV) for _ in range(3))
    moe.moe_verify_drafts(place(logits), dev(np.asarray(tokens, np.int32)), dev(np.asarray(uniform, np.float32)), dev(np.asarray(q_start, np.int32)), acc, nxt, n_new,
                          draft_logits=None if draft is None else place(draft),
                          temperature=None if temperature is None else dev(np.asarray(temperature, np.float32)), workspace=ws, st=st)
    return host(acc), host(nxt), host(n_new)


def _case(rng, S, most, V, by_model, dtype, near=0.5, idle=0.15):
    counts = [0 if rng.random() < idle else int(rng.integers(1, most + 2)) for _ in range(S)]
    q_start = np.concatenate([[0], np.cumsum(counts)])
    T = max(int(q_start[-1]), 1)
    logits = rng.normal(size=(T, V)) * 3
    draft = logits + near * rng.normal(size=(T, V))
    hide = rng.random((T, V)) < 0.2
    hide[np.arange(T), rng.integers(0, V, T)] = False
    logits = np.where(hide, -np.inf, logits)
    if dtype == torch.bfloat16:
        logits, draft = (torch.from_numpy(a.astype(np.float32)).to(dtype).float().numpy() for a in (logits, draft))
    logits, draft = logits.astype(np.float32), draft.astype(np.float32)
    tokens = np.zeros(T, np.int32)
    tokens[1:] = (draft + rng.gumbel(size=(T, V))).argmax(1)[:-1]
    temp = rng.choice([0.0, 0.5, 1.0, 1.7], S).astype(np.float32)
    return logits, tokens, rng.random(T).astype(np.float32), q_start, draft if by_model else None, temp


@pytest.mark.parametrize("S,most,V", [(1, 0, 1), (1, 4, 7), (5, 3, 100), (40, 6, 333), (3, 7, 5003), (2, 3, 32000), (2, 2, 70001), (300, 2, 17)])
@pytest.mark.parametrize("by_model", [False, True])
@pytest.mark.parametrize("dtype,shift,pad", [(torch.float32, 0, 0), (torch.float32, 1, 3), (torch.bfloat16, 0, 1), (torch.bfloat16, 3, 0)])
def test_equals_the_definition(S, most, V, by_model, dtype, shift, pad):
    rng = np.random.default_rng(S * 100 + V + by_model)
    for near in (0.1, 1.5):
        c = _case(rng, S, most, V, by_model, dtype, near)
        st = status_tensor()
        got = _run(*c, dtype=dtype, shift=shift, pad=pad, st=st)
        want = _verify.verify(*c)
        for g, w in zip(got, want):
            assert np.array_equal(g, w)
        assert st.tolist() == [0, 0]


def test_without_temperature_or_n_new():
    rng = np.random.default_rng(1)
    logits, tokens, u, q_start, draft, _ = _case(rng, 6, 3, 50, True, torch.float32)
    want = _verify.verify(logits, tokens, u, q_start, draft)
    acc, nxt = (torch.empty(6, dtype=torch.int32, device=DEV) for _ in range(2))
    moe.moe_verify_drafts(dev(logits), dev(tokens), dev(u), dev(q_start.astype(np.int32)), acc, nxt, draft_logits=dev(draft))
    assert np.array_equal(host(acc), want[0]) and np.array_equal(host(nxt), want[1])


def test_ends_of_the_uniform_numbers():
    """0 and the largest number below 1 draw the first and the last token that can be; numbers outside count as the nearest."""
    rng = np.random.default_rng(2)
    V = 1000
    row = np.full((1, V), -np.inf, np.float32)
    can = np.sort(rng.choice(V, 50, replace=False))
    row[0, can] = rng.normal(size=50)
    for u, want in ((0.0, can[0]), (1 - 2.0 ** -24, can[-1]), (1.0, can[-1]), (5.0, can[-1]), (-1.0, can[0]), (math.nan, can[0])):
        assert _run(row, [0], [u], [0, 1])[1][0] == want


def test_greedy_takes_the_first_of_equals():
    row = np.zeros((3, 9000), np.float32)
    row[0, [700, 8999]] = 5
    row[1, 4] = row[1, 5] = 1
    assert [int(v[0]) for v in _run(row, [0, 700, 4], [0.5] * 3, [0, 3], temperature=[0.0])] == [2, 0, 0]
    assert [int(v[0]) for v in _run(row, [0, 8999, 4], [0.5] * 3, [0, 3], temperature=[0.0])] == [0, 700, -2]
    assert [int(v[0]) for v in _run(row, [0, 700, 5], [0.5] * 3, [0, 3], temperature=[2.0 ** -61])] == [1, 4, -1]


def test_same_distributions_accept_all():
    """q = p: u q < p for every u below 1."""
    rng = np.random.default_rng(3)
    logits = rng.normal(size=(33, 400)).astype(np.float32)
    tokens = np.r_[0, rng.integers(0, 400, 32)].astype(np.int32)
    assert _run(logits, tokens, np.full(33, 1 - 2.0 ** -24), [0, 33], draft=logits)[0][0] == 32


def test_disjoint_distributions_accept_none():
    logits, draft = np.full((2, 64), -np.inf, np.float32), np.full((2, 64), -np.inf, np.float32)
    logits[:, :32], draft[:, 32:] = 0, 0
    acc, nxt, n_new = _run(logits, [0, 40], [0.999, 0.0], [0, 2], draft=draft)
    assert (acc[0], n_new[0]) == (0, -1) and nxt[0] == 31


def test_many_drafts():
    """More drafts than a CTA has threads."""
    rng = np.random.default_rng(4)
    T, V = 1300, 12
    logits = np.full((T, V), -np.inf, np.float32)
    path = rng.integers(0, V, T)
    logits[np.arange(T), path] = 1.0
    tokens = np.r_[0, path[:-1]].astype(np.int32)
    for stop in (None, 1, 700, 1298):
        t = tokens.copy()
        if stop is not None:
            t[stop + 1 if stop < 1298 else 1299] ^= 1
        acc, nxt, _ = _run(logits, t, np.full(T, 0.3), [0, T])
        n = T - 1 if stop is None else int(np.nonzero(t != tokens)[0][0]) - 1
        assert acc[0] == n and nxt[0] == path[n]


@pytest.mark.parametrize("by_model", [False, True])
def test_bad_inputs_are_reported_and_stay_alone(by_model):
    rng = np.random.default_rng(5)
    logits, tokens, u, q_start, draft, temp = _case(rng, 8, 3, 90, by_model, torch.float32, idle=0)
    temp[:] = 1
    q_start = np.arange(9) * 3
    T = 24
    logits, draft0 = rng.normal(size=(T, 90)).astype(np.float32), rng.normal(size=(T, 90)).astype(np.float32)
    tokens, u = rng.integers(0, 90, T).astype(np.int32), rng.random(T).astype(np.float32)
    draft = draft0 if by_model else None
    good = _verify.verify(logits, tokens, u, q_start, draft, temp)

    def check(code, details, s, **kw):
        a = dict(logits=logits, tokens=tokens, uniform=u, q_start=q_start, draft=draft, temperature=temp)
        a.update(kw)
        st = status_tensor()
        got = _run(**a, st=st)
        assert st.tolist()[0] == code and st.tolist()[1] in details
        assert (got[0][s], got[1][s]) == (0, -1)
        keep = np.arange(8) != s
        for g, w in zip(got, good):
            assert np.array_equal(g[keep], w[keep])

    for value in (math.nan, math.inf):
        x = logits.copy()
        x[3 * 2 + 1, 50] = value
        check(1, [7], 2, logits=x)
    x = logits.copy()
    x[8] = -np.inf
    check(1, [8], 2, logits=x)
    for bad in (-1, 90, 2 ** 31 - 1):
        t = tokens.copy()
        t[10] = bad
        check(3, [10], 3, tokens=t)
    for bad in (-0.5, math.nan, math.inf):
        t = temp.copy()
        t[5] = bad
        check(1, [-6], 5, temperature=t)
    if by_model:
        x = draft.copy()
        x[13, 0] = math.nan
        check(1, [T + 13], 4, draft=x)
        x = draft.copy()
        x[14, 0] = math.nan                # a sequence's last row is not read
        st = status_tensor()
        assert np.array_equal(_run(logits, tokens, u, q_start, x, temp, st=st)[1], good[1]) and st.tolist() == [0, 0]
    # rows that no sequence has are not read, and a bad range is reported
    x = logits.copy()
    x[21:] = math.nan
    q = q_start.copy()
    q[8] = 21
    got = _run(logits=x, tokens=tokens, uniform=u, q_start=q, draft=draft, temperature=temp, st=(st := status_tensor()))
    assert st.tolist() == [0, 0] and [int(v[7]) for v in got] == [0, -1, 0]
    for end in (25, 20, -3):
        q = q_start.copy()
        q[8] = end
        got = _run(logits=logits, tokens=tokens, uniform=u, q_start=q, draft=draft, temperature=temp, st=(st := status_tensor()))
        assert st.tolist() == [3, 7] and [int(v[7]) for v in got] == [0, -1, 0]
        assert np.array_equal(got[1][:7], good[1][:7])


def test_captured_and_replayed():
    rng = np.random.default_rng(6)
    c = _case(rng, 9, 4, 2001, True, torch.bfloat16)
    S, T = 9, len(c[1])
    bf = lambda a: dev(a).to(torch.bfloat16)  # noqa: E731
    logits, draft, tokens, u = bf(c[0]), bf(c[4]), dev(c[1]), dev(c[2])
    q_start, temp = dev(c[3].astype(np.int32)), dev(c[5])
    outs = [torch.empty(S, dtype=torch.int32, device=DEV) for _ in range(3)]
    ws = torch.empty(moe.verify_workspace(T, S, 2001), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_verify_drafts(logits, tokens, u, q_start, *outs, draft_logits=draft, temperature=temp, workspace=ws)
    for _ in range(4):
        u.copy_(dev(rng.random(T).astype(np.float32)))
        ws.fill_(255)                      # it holds nothing between calls
        graph.replay()
        want = _verify.verify(c[0], c[1], host(u), c[3], c[4], c[5])
        for g, w in zip(outs, want):
            assert np.array_equal(host(g), w)


def test_distribution_of_the_first_token():
    """8000 sequences of one distribution: the token after the newest is distributed as the target's, whatever the drafts were
    drawn from (the counts' chi-square statistic, of 7 degrees of freedom, is above 55.9 once in 1e9)."""
    rng = np.random.default_rng(7)
    V, S = 8, 8000
    p_l, q_l = rng.normal(size=V).astype(np.float32), rng.normal(size=V).astype(np.float32)
    p = np.exp(p_l.astype(np.float64))
    p /= p.sum()
    q = np.exp(q_l.astype(np.float64))
    q /= q.sum()
    tokens = np.zeros(2 * S, np.int32)
    tokens[1::2] = rng.choice(V, S, p=q)
    u = rng.random(2 * S).astype(np.float32)
    acc, nxt, _ = _run(np.tile(p_l, (2 * S, 1)), tokens, u, np.arange(S + 1) * 2, draft=np.tile(q_l, (2 * S, 1)))
    first = np.where(acc == 1, tokens[1::2], nxt)
    count = np.bincount(first, minlength=V)
    assert ((count - S * p) ** 2 / (S * p)).sum() < 55.9


def test_binding_refuses():
    i32 = dict(dtype=torch.int32, device=DEV)
    a = [torch.zeros(4, 10, device=DEV), torch.zeros(4, **i32), torch.zeros(4, device=DEV), torch.zeros(3, **i32), torch.zeros(2, **i32), torch.zeros(2, **i32)]

    def call(i, t, **kw):
        b = list(a)
        if i is not None:
            b[i] = t
        moe.moe_verify_drafts(*b, **kw)

    for i, t, match in ((0, torch.zeros(4, 10, 1, device=DEV), "logits"), (0, torch.zeros(4, 10, device=DEV).half(), "dtype"), (1, a[1][:3], "tokens"),
                        (1, a[1].long(), "tokens"), (2, a[2][:3], "uniform"), (3, a[3][:2], "q_start"), (5, a[5][:1], "next_token")):
        with pytest.raises(moe.MoeError, match=match):
            call(i, t)
    with pytest.raises(moe.MoeError, match="draft_logits"):
        call(None, None, draft_logits=a[0].bfloat16())
    with pytest.raises(moe.MoeError, match="temperature"):
        call(None, None, temperature=torch.zeros(3, device=DEV))
    with pytest.raises(moe.MoeError, match="n_new"):
        call(None, None, n_new=torch.zeros(3, **i32))
    with pytest.raises(moe.MoeError, match="workspace"):
        call(None, None, workspace=torch.zeros(16, dtype=torch.uint8, device=DEV))
