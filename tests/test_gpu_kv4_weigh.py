"""The attention weight that cached tokens draw, on the GPU against the
definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

import _kv4
import expert_routing_moe_gb300 as moe
from _gpu import DEV, assert_status_ok, dev, host, status_tensor

pytestmark = pytest.mark.gpu
PAGE = 64


def _reference(cache, q, lse, q_start, scale, window, last, score, fresh):
    """(score, bound of its error).  A score's product is off by at most 2^-20 of its magnitudes' sum (as in the
    attention); its difference to lse by 2^-23 of both; the exponential by 2^-21; and a sum of n terms, in any
    order, by n 2^-24 of it (all terms are positive), of which half a step is the last addition's."""
    T, n_q, D = q.shape
    G = n_q // cache.n_kv
    out, tol = score.astype(np.float64).copy(), np.zeros(score.shape)
    for s, length in enumerate(cache.lengths):
        q0, n = q_start[s], q_start[s + 1] - q_start[s]
        if n == 0 or length == 0:
            continue
        new = max(0, length - n)
        if fresh:
            out[s, new:length] = 0
        terms = np.zeros(length)
        for i in range(max(0, n - last) if last else 0, n):
            p = length - n + i
            lo = max(0, p - window + 1) if window else 0
            if p < 0:
                continue
            k = cache.k[s][lo:p + 1]
            for h in range(n_q):
                z = float(lse[q0 + i, h])
                if z == -math.inf:
                    continue
                kh = k[:, h // G]
                x = kh @ q[q0 + i, h] * scale
                off = np.abs(kh) @ np.abs(q[q0 + i, h]) * abs(scale) * 2.0 ** -20
                w = np.exp(x - z)
                out[s, lo:p + 1] += w
                tol[s, lo:p + 1] += w * (np.expm1(off + 2.0 ** -22 * (np.abs(x) + abs(z))) + 2.0 ** -21)
                terms[lo:p + 1] += 1
        tol[s, :length] += (terms + 2) * 2.0 ** -24 * np.abs(out[s, :length]) + 2.0 ** -24 * np.abs(score[s, :length]) + 1e-30
    return out, tol


class Case:
    def __init__(self, seed, lengths, rows, n_q, n_kv, D, scales=True, pad_rows=0, stride=0):
        rng = np.random.default_rng(seed)
        self.ref = _kv4.Cache(rng, lengths, n_kv, D, scales)
        self.q_start = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
        T = int(self.q_start[-1]) + pad_rows
        self.q = torch.from_numpy(rng.normal(size=(T, n_q, D)).astype(np.float32)).to(torch.bfloat16)
        self.scale = D ** -0.5
        self.rng, self.max_new, self.T, self.n_q = rng, max(list(rows) + [0]), T, n_q
        r = self.ref
        self.pages, self.table, self.lens = dev(r.bytes), dev(r.table), dev(np.array(r.lengths, np.int32))
        self.cache = moe.Kv4Cache(self.pages, self.table, self.lens, D, None if r.k_scale is None else dev(r.k_scale), None)
        # lse as attention gives it
        _, self.lse, _, _ = _kv4.attention(r, self.q.double().numpy(), self.q_start.tolist(), self.scale)
        self.lse = self.lse.astype(np.float32)
        self.score = (rng.random((len(lengths), r.columns * PAGE + 3)) * 2).astype(np.float32)
        wide = torch.zeros(T, n_q * D + stride, dtype=torch.bfloat16, device=DEV)
        self.q_dev = wide[:, :n_q * D].unflatten(1, (n_q, D))
        self.q_dev.copy_(self.q)
        self.ws = torch.full((max(moe.kv4_weigh_workspace(self.cache, T, n_q), 256),), 255, dtype=torch.uint8, device=DEV)

    def run(self, window=0, last=0, fresh=False, lse=None, st=None, score=None):
        out = dev(self.score) if score is None else score
        moe.moe_kv4_weigh(self.q_dev, self.cache, dev(self.q_start), dev(self.lse if lse is None else lse), out, self.scale, self.max_new, window, last, fresh,
                          self.ws, st)
        return out

    def check(self, window=0, last=0, fresh=False, lse=None):
        st = status_tensor()
        if window and lse is None:
            _, lse, _, _ = _kv4.attention(self.ref, self.q.double().numpy(), self.q_start.tolist(), self.scale, window)
            lse = lse.astype(np.float32)
        got = host(self.run(window, last, fresh, lse, st)).astype(np.float64)
        want, tol = _reference(self.ref, self.q.double().numpy(), self.lse if lse is None else lse, self.q_start, self.scale, window, last, self.score, fresh)
        err = np.abs(got - want)
        assert (err <= tol).all(), "worst error / bound %.2f at %s" % (np.max(err / (tol + 1e-300)), np.unravel_index(np.argmax(err - tol), err.shape))
        assert_status_ok(st)


@pytest.mark.parametrize("lengths,rows,n_q,n_kv,D", [
    ([1], [1], 1, 1, 64), ([64], [1], 8, 2, 128), ([65, 63, 0, 200], [1, 1, 1, 1], 16, 2, 64), ([130, 7], [3, 7], 14, 2, 64), ([300], [300], 8, 1, 128),
    ([500, 33], [40, 20], 12, 4, 64), ([1000, 0, 129, 64], [1, 0, 4, 2], 6, 3, 128), ([90, 700], [90, 130], 4, 4, 64), ([700], [257], 20, 2, 128),
    ([3, 5000], [1, 2], 2, 2, 64)])
def test_equals_the_definition(lengths, rows, n_q, n_kv, D):
    c = Case(sum(lengths), lengths, rows, n_q, n_kv, D, scales=D == 64)
    c.check()
    c.check(fresh=True)


@pytest.mark.parametrize("window,last,fresh", [(1, 0, False), (63, 0, False), (64, 0, True), (100, 0, False), (5000, 0, False), (0, 1, False), (0, 30, True),
                                               (0, 500, False), (50, 16, True), (2147483647, 3, False)])
def test_windows_and_last_rows(window, last, fresh):
    Case(11, [400, 129, 77, 0], [150, 9, 77, 2], 8, 2, 64).check(window, last, fresh)


def test_strided_queries_and_rows_of_no_sequence():
    c = Case(12, [100, 260], [5, 100], 6, 2, 128, pad_rows=9, stride=16)
    c.check()
    c.q_dev[105:] = float("nan")
    c.check()


def test_rows_before_their_sequence_and_rows_that_see_nothing():
    c = Case(13, [3, 70], [10, 8], 4, 2, 64)       # seven of the first's rows have a place below 0
    assert (c.lse[:7] == -np.inf).all()
    c.check()
    c.check(last=9)
    # rows whose lse says that they see nothing add nothing, whatever is in them
    lse = c.lse.copy()
    lse[12] = -np.inf
    c.check(lse=lse)
    c.q_dev[12] = float("nan")
    out = c.run(lse=lse)
    assert out.isfinite().all()


def test_other_sums_than_one():
    """With another lse the weights are what the definition says, above 1 and far below the smallest float among them."""
    c = Case(14, [200], [20], 8, 2, 128)
    c.check(lse=c.lse - 3)
    c.check(lse=c.lse + 40)
    out = c.run(lse=np.full_like(c.lse, np.inf))
    assert np.array_equal(host(out), c.score)


def test_two_layers_share_a_score():
    a, b = Case(15, [150, 80], [4, 2], 8, 2, 64), Case(15, [150, 80], [4, 2], 8, 2, 64)
    out = a.run(fresh=True)
    one = host(out).copy()
    b.run(score=out)
    two = host(out)
    assert np.allclose(two[0, 146:150], 2 * one[0, 146:150], rtol=1e-6) and np.array_equal(two[0, 150:], a.score[0, 150:])


def test_sum_over_the_tokens_is_the_rows():
    """Every row that sees something gives each of its heads a weight of 1 in all."""
    c = Case(16, [900, 300], [64, 1], 8, 2, 128)
    got = host(c.run()) - c.score
    assert abs(got[0].sum() - 64 * 8) < 1e-2 and abs(got[1].sum() - 8) < 1e-3


def test_long_context_and_many_pages():
    c = Case(17, [9000], [2], 8, 1, 64)
    c.check()
    c.check(window=4000)


def test_bad_pages_lengths_and_starts():
    c = Case(18, [200, 200, 200], [2, 2, 2], 4, 2, 64)
    good = host(c.run())
    for bad in (-1, 1 << 30, int(c.pages.shape[0])):
        keep = int(c.table[1, 2])
        c.table[1, 2] = bad
        st = status_tensor()
        got = host(c.run(st=st))
        assert st.tolist() == [3, bad]
        assert np.array_equal(got[1, :128], good[1, :128]) and np.array_equal(got[1, 128:], np.where(np.arange(got.shape[1] - 128) < 64, c.score[1, 128:], good[1, 128:]))
        assert np.array_equal(got[[0, 2]], good[[0, 2]])
        c.table[1, 2] = keep
    for bad in (-5, c.table.shape[1] * 64 + 1, 2 ** 31 - 1):
        c.lens[1] = bad
        st = status_tensor()
        got = host(c.run(st=st))
        assert st.tolist() == [3, 1] and np.array_equal(got[1], c.score[1]) and np.array_equal(got[[0, 2]], good[[0, 2]])
        c.lens[1] = 200
    keep = c.q_start.copy()
    for bad in ([0, 2, 1, 6], [0, 2, 100, 6], [0, -3, 4, 6]):
        c.q_start = np.array(bad, np.int32)
        st = status_tensor()
        c.run(st=st)
        assert st.tolist()[0] == 3
    c.q_start = keep
    assert np.array_equal(host(c.run()), good)


@pytest.mark.parametrize("lengths,rows", [([500, 90], [3, 1]), ([700, 400], [300, 150])])
def test_same_bits_in_a_graph_and_on_two_streams(lengths, rows):
    c = Case(19, lengths, rows, 8, 2, 128)
    want = c.run()
    out, start, lse = dev(c.score), dev(c.q_start), dev(c.lse)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_kv4_weigh(c.q_dev, c.cache, start, lse, out, c.scale, c.max_new, workspace=c.ws)
    for _ in range(3):
        out.copy_(first)
        graph.replay()
        assert torch.equal(out, want)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, spaces = [first.clone() for _ in range(2)], [torch.zeros_like(c.ws) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, w in zip(streams, outs, spaces):
            with torch.cuda.stream(s):
                o.copy_(first)
            moe.moe_kv4_weigh(c.q_dev, c.cache, start, lse, o, c.scale, c.max_new, workspace=w, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_binding_refuses():
    c = Case(20, [100], [2], 4, 2, 64)
    q_start, lse, score = dev(c.q_start), dev(c.lse), dev(c.score)
    with pytest.raises(moe.MoeError, match="lse"):
        moe.moe_kv4_weigh(c.q_dev, c.cache, q_start, lse[:1], score, 1.0, 2)
    with pytest.raises(moe.MoeError, match="score"):
        moe.moe_kv4_weigh(c.q_dev, c.cache, q_start, lse, score[:, :127], 1.0, 2)
    with pytest.raises(moe.MoeError, match="score"):
        moe.moe_kv4_weigh(c.q_dev, c.cache, q_start, lse, score.double(), 1.0, 2)
    with pytest.raises(moe.MoeError, match="q:"):
        moe.moe_kv4_weigh(c.q_dev[..., :32], c.cache, q_start, lse, score, 1.0, 2)
    with pytest.raises(moe.MoeError, match="q_start"):
        moe.moe_kv4_weigh(c.q_dev, c.cache, q_start[:1], lse, score, 1.0, 2)
    with pytest.raises(moe.MoeError, match="invalid"):
        moe.moe_kv4_weigh(c.q_dev, c.cache, q_start, lse, score, float("nan"), 2)
    moe.moe_kv4_weigh(c.q_dev, c.cache, q_start, lse, score, c.scale, 2)      # a workspace of the call's own
    assert torch.equal(score, c.run())
