"""The numpy references of the weights in 4 bits, of the drafts' verification and
of the eviction against closed forms, and the host side of the operators' entry
points: sizes and refusals.  No GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import __graft_entry__ as entry
import _kv4
import _verify
import _w4
import expert_routing_moe_gb300 as moe
from expert_routing_moe_gb300 import _abi as abi

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails its host-side checks
ODD = ctypes.c_void_p((1 << 20) + 8)
BYTE = ctypes.c_void_p((1 << 20) + 1)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    entry.build()
    return abi.load()


# ---- weights in 4 bits ----
@pytest.mark.parametrize("N,K", [(1, 1), (128, 128), (130, 200), (256, 129)])
def test_layout_places_are_a_partition(N, K):
    half, j, sc = _w4.places(N, K)
    bits = np.zeros(_w4.n_bytes(N, K) * 8, int)
    for jj, at in enumerate(_w4.BITS):
        for b in at:
            np.add.at(bits, half[j == jj] * 8 + b, 1)
    assert bits.max() == 1 and bits.sum() == 4 * N * K
    scale = np.zeros(_w4.n_bytes(N, K), int)
    np.add.at(scale, sc, 1)
    assert (bits.reshape(-1, 8).sum(1)[scale > 0] == 0).all() and scale.max() <= 16
    assert len(np.unique(sc)) == N * -(-K // 16)


def test_first_codes_are_shift_and_mask():
    """A code's bits, taken as a bf16 with the sign and the low exponent bits that the layout puts there, are the code's value times 2^-126."""
    for code in range(16):
        for j, shift in ((0, 0), (1, 3), (2, 6)):
            word = sum(((code >> (3 - i)) & 1) << b for i, b in enumerate(_w4.BITS[j]))
            half = (word << shift) & 0x81C0
            v = torch.tensor([half if half < 0x8000 else half - 0x10000], dtype=torch.int16).view(torch.bfloat16).double().item()
            assert v * 2.0 ** 126 == _kv4.GRID[code & 7] * (-1 if code & 8 else 1)


def test_quantised_weights_are_near():
    rng = np.random.default_rng(0)
    w = (rng.normal(size=(40, 250)) * rng.uniform(0.001, 3, (40, 1))).astype(np.float32)
    w[3] = 0
    v = _w4.values(*_w4.quantise(w))
    pad = np.zeros((40, 256))
    pad[:, :250] = np.abs(w)
    top = np.repeat(pad.reshape(40, 16, 16).max(-1), 16, -1)[:, :250]
    # steps are at most 2 in units of a block's scale, which is top/6 to within 2^-4, or half a step of the smallest scale (2^-10 row scales)
    row = np.abs(w).max(1, keepdims=True) / 2688
    assert (np.abs(v - w) <= top / 6 * (1 + 2.0 ** -4) + 6 * 2.0 ** -10 * row + 1e-30).all()
    assert (v[3] == 0).all()


# ---- verification ----
def test_weights_are_powers():
    rng = np.random.default_rng(1)
    row = (rng.normal(size=5000) * 8).astype(np.float32)
    for temp in (1.0, 0.3, 5.0):
        w = _verify.weights(row, np.float32(_verify.LOG2E / np.float32(temp))).astype(np.float64)
        true = np.exp((row.astype(np.float64) - row.max()) / temp)
        true = np.maximum(true, 2.0 ** -60)
        # the exponent is off by 3 roundings of at most 2^-24 of itself (at most 60 ln 2), the series by 2^-22
        assert (np.abs(w / true - 1) <= 2.0 ** -21 + 3 * 2.0 ** -24 * np.abs(np.log(true)) * 1.01).all()
    assert _verify.weights(row, np.float32(1)).max() == 1


@pytest.mark.parametrize("by_model", [False, True])
def test_first_token_is_distributed_as_the_target(by_model):
    """P(x) = q(x) min(1, p(x)/q(x)) + P(refused) max(p - q, 0)(x) / sum, from the reference's own decisions, is p(x)."""
    rng = np.random.default_rng(2)
    V = 6
    logits = rng.normal(size=(2, V)).astype(np.float32) * 2
    draft = rng.normal(size=(2, V)).astype(np.float32) * 2 if by_model else None
    p = np.exp(logits[0].astype(np.float64))
    p /= p.sum()
    q = np.exp(draft[0].astype(np.float64)) if by_model else np.eye(V)[3]
    q /= q.sum()
    grid = (np.arange(2000) + 0.5) / 2000
    got = np.zeros(V)
    for x in range(V):
        if q[x] == 0:
            continue
        tokens = np.array([0, x], np.int32)
        accepted = np.array([_verify.verify(logits, tokens, np.array([0.5, u], np.float32), [0, 2], draft)[0][0] for u in grid])
        share = accepted.mean()
        assert abs(share - min(1, p[x] / q[x])) <= 1 / 2000
        got[x] += q[x] * share
        if share < 1:
            nxt = [_verify.verify(logits, tokens, np.array([u, 1 - 2.0 ** -24], np.float32), [0, 2], draft)[1][0] for u in grid]
            got += q[x] * (1 - share) * np.bincount(nxt, minlength=V) / 2000
    assert np.abs(got - p).max() <= 3 / 2000


def test_verify_by_hand():
    big = np.full((3, 4), -math.inf, np.float32)
    big[0, 1] = big[1, 2] = big[2, 3] = 0
    u = np.zeros(3, np.float32)
    assert [int(v[0]) for v in _verify.verify(big, np.array([0, 1, 2]), u, [0, 3])] == [2, 3, 0]
    assert [int(v[0]) for v in _verify.verify(big, np.array([0, 1, 3]), u, [0, 3])] == [1, 2, -1]
    assert [int(v[0]) for v in _verify.verify(big, np.array([0, 0, 2]), u, [0, 3])] == [0, 1, -2]


# ---- sizes and refusals ----
def test_sizes(lib):
    assert moe.w4_bytes(1, 1) == 9216 and moe.w4_bytes(129, 128) == 2 * 9216 and moe.w4_bytes(0, 5) == 0
    assert moe.w4_bytes(1 << 24, 1 << 24) == (1 << 34) * 9216
    assert moe.verify_workspace(0, 4, 10) == 0 and moe.verify_workspace(7, 2, 10) > 0 and moe.verify_workspace(-1, 2, 10) == 0
    assert lib.moe_kv4_evict_workspace(3, 10, 40) >= 3 * 10 * 64 * 4 and lib.moe_kv4_evict_workspace(-1, 10, 40) == 0
    assert lib.moe_kv4_weigh_workspace(3, 10, 4, 3, 128, 8) == 0      # heads do not divide


def _cache(pages=FAKE, table=FAKE, lens=FAKE, n_pages=8, max_pages=4, S=2, n_kv=2, D=128):
    return abi._Kv4CacheParams(pages, table, lens, None, None, n_pages, max_pages, S, n_kv, D)


def _pool(pages=FAKE, table=FAKE, lens=FAKE, ref=FAKE, layers=2, n_pages=8, max_pages=4, S=2, bytes_=2 * 9216):
    return abi._Kv4PoolParams(pages, 8 * bytes_, bytes_, table, lens, ref, layers, n_pages, max_pages, S)


def _w4p(tiles=FAKE, scale=FAKE, N=64, K=64):
    return abi._W4Params(tiles, scale, N, K)


BAD, UNSUPPORTED, WORKSPACE = -1, -2, -4


def _weigh(lib, cache=None, **kw):
    a = dict(q=FAKE, ld_q=512, T=4, n_q=4, q_start=FAKE, max_new=2, lse=FAKE, scale=0.1, window=0, last=0, score=FAKE, ld_score=256, fresh=0,
             ws=FAKE, bytes_=BIG)
    a.update(kw)
    c = _cache() if cache is None else cache
    return lib.moe_kv4_weigh(a["q"], a["ld_q"], a["T"], a["n_q"], ctypes.byref(c), a["q_start"], a["max_new"], a["lse"], a["scale"], a["window"], a["last"],
                             a["score"], a["ld_score"], a["fresh"], a["ws"], a["bytes_"], None, None)


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(q=None)), (BAD, dict(q=ODD)), (BAD, dict(ld_q=511)), (BAD, dict(ld_q=516)), (BAD, dict(T=-1)), (BAD, dict(n_q=3)), (BAD, dict(n_q=0)),
    (BAD, dict(q_start=None)), (BAD, dict(max_new=-1)), (BAD, dict(lse=None)), (BAD, dict(scale=math.nan)), (BAD, dict(scale=math.inf)),
    (BAD, dict(window=-1)), (BAD, dict(last=-1)), (BAD, dict(score=None)), (BAD, dict(ld_score=255)),
    (UNSUPPORTED, dict(n_q=2048, ld_q=BIG)), (UNSUPPORTED, dict(cache=_cache(D=96))), (UNSUPPORTED, dict(cache=_cache(max_pages=1 << 25))),
    (BAD, dict(cache=_cache(pages=ODD))), (BAD, dict(cache=_cache(table=None)))])
def test_weigh_refuses(lib, want, kw):
    assert _weigh(lib, **kw) == want


def test_weigh_nothing_to_do(lib):
    assert _weigh(lib, T=0, q=None, lse=None, score=None) == 0 and _weigh(lib, cache=_cache(S=0)) == 0


def _evict(lib, pool=None, **kw):
    a = dict(D=128, score=FAKE, ld_score=256, budget=FAKE, sinks=0, recent=0, kept=None, ld_kept=0, ws=FAKE, bytes_=BIG)
    a.update(kw)
    p = _pool() if pool is None else pool
    return lib.moe_kv4_evict(ctypes.byref(p), a["D"], a["score"], a["ld_score"], a["budget"], a["sinks"], a["recent"], a["kept"], a["ld_kept"], a["ws"], a["bytes_"],
                             None, None)


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(score=None)), (BAD, dict(ld_score=255)), (BAD, dict(budget=None)), (BAD, dict(sinks=-1)), (BAD, dict(recent=-1)),
    (BAD, dict(kept=FAKE, ld_kept=-1)), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(bytes_=100)), (BAD, dict(ws=ODD)), (UNSUPPORTED, dict(D=96)),
    (BAD, dict(pool=_pool(bytes_=9216 + 4608))), (BAD, dict(pool=_pool(ref=None))), (UNSUPPORTED, dict(pool=_pool(S=5000))),
    (UNSUPPORTED, dict(pool=_pool(max_pages=1 << 25), ld_score=BIG))])
def test_evict_refuses(lib, want, kw):
    assert _evict(lib, **kw) == want


def test_evict_nothing_to_do(lib):
    assert _evict(lib, pool=_pool(S=0), score=None) == 0


def _linear(lib, w=None, **kw):
    a = dict(x=FAKE, ld_x=64, T=2, bias=None, y=FAKE, dtype=0, ld_y=64, add=0)
    a.update(kw)
    p = _w4p() if w is None else w
    return lib.moe_linear_w4(a["x"], a["ld_x"], a["T"], ctypes.byref(p), a["bias"], a["y"], a["dtype"], a["ld_y"], a["add"], None, None)


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(x=None)), (BAD, dict(x=BYTE)), (BAD, dict(ld_x=63)), (BAD, dict(T=-1)), (BAD, dict(y=None)), (BAD, dict(y=BYTE)), (BAD, dict(dtype=2)),
    (BAD, dict(ld_y=63)), (BAD, dict(dtype=1, add=1)), (UNSUPPORTED, dict(T=(1 << 20) + 1)), (BAD, dict(w=_w4p(tiles=None))), (BAD, dict(w=_w4p(tiles=ODD))),
    (BAD, dict(w=_w4p(N=0))), (BAD, dict(w=_w4p(K=0))), (UNSUPPORTED, dict(w=_w4p(N=(1 << 24) + 1)))])
def test_linear_refuses(lib, want, kw):
    assert _linear(lib, **kw) == want


def test_linear_nothing_to_do(lib):
    assert _linear(lib, T=0, x=None, y=None) == 0


@pytest.mark.parametrize("want,args", [(BAD, dict(w=None)), (BAD, dict(ld=63)), (BAD, dict(dtype=7)), (BAD, dict(out=_w4p(scale=None))), (BAD, dict(out=_w4p(tiles=ODD)))])
def test_pack_refuses(lib, want, args):
    a = dict(w=FAKE, dtype=0, ld=64, out=_w4p())
    a.update(args)
    assert lib.moe_w4_pack(a["w"], a["dtype"], a["ld"], ctypes.byref(a["out"]), None, None) == want


def _verify_call(lib, **kw):
    a = dict(logits=FAKE, dtype=0, ld=100, T=5, V=100, tokens=FAKE, uniform=FAKE, q_start=FAKE, S=2, draft=None, ld_draft=0, temperature=None, accepted=FAKE,
             next=FAKE, n_new=None, ws=FAKE, bytes_=BIG)
    a.update(kw)
    return lib.moe_verify_drafts(a["logits"], a["dtype"], a["ld"], a["T"], a["V"], a["tokens"], a["uniform"], a["q_start"], a["S"], a["draft"], a["ld_draft"],
                                 a["temperature"], a["accepted"], a["next"], a["n_new"], a["ws"], a["bytes_"], None, None)


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(logits=None)), (BAD, dict(logits=BYTE)), (BAD, dict(dtype=3)), (BAD, dict(ld=99)), (BAD, dict(T=-1)), (BAD, dict(V=0)), (BAD, dict(tokens=None)),
    (BAD, dict(uniform=None)), (BAD, dict(q_start=None)), (BAD, dict(S=-1)), (BAD, dict(draft=FAKE, ld_draft=99)), (BAD, dict(draft=BYTE, ld_draft=100)),
    (BAD, dict(accepted=None)), (BAD, dict(next=None)), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(bytes_=16)), (BAD, dict(ws=ODD)),
    (UNSUPPORTED, dict(T=(1 << 16) + 1)), (UNSUPPORTED, dict(V=(1 << 20) + 1, ld=BIG)), (UNSUPPORTED, dict(S=16385))])
def test_verify_refuses(lib, want, kw):
    assert _verify_call(lib, **kw) == want


def test_verify_nothing_to_do(lib):
    assert _verify_call(lib, S=0, q_start=None, accepted=None) == 0


def test_binding_refuses_host_tensors(lib):
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    with pytest.raises(moe.MoeError, match="tiles"):
        moe.Weight4(torch.zeros(9216, dtype=torch.uint8), 4, 4)
    with pytest.raises(moe.MoeError, match="tiles: expected 18432 bytes"):
        moe.Weight4(torch.zeros(9216, dtype=torch.uint8), 129, 4)
    with pytest.raises(moe.MoeError, match="logits"):
        moe.moe_verify_drafts(torch.zeros(2, 5), torch.zeros(2, dtype=i32), torch.zeros(2), torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(1, dtype=i32))
    with pytest.raises(moe.MoeError, match="dtype"):
        moe.moe_w4_pack(torch.zeros(4, 4, dtype=torch.float16), None)
    assert bf is not f32
