"""The numpy reference of the 4-bit cache against closed forms, and the host
side of its entry points: page sizes, workspaces, refusals.  No GPU."""
import ctypes

import numpy as np
import pytest
import torch

import __graft_entry__ as entry
import _kv4
import expert_routing_moe_gb300 as moe
from expert_routing_moe_gb300 import _abi as abi

FAKE = ctypes.c_void_p(1 << 20)   # never dereferenced: every call below fails its host-side checks
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    entry.build()
    return abi.load()


def test_e4m3_grid_matches_torch():
    b = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(b, _kv4.E4M3)


@pytest.mark.parametrize("x,c", [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6), (5.1, 7),
                                 (0.2501, 1), (6.0, 7)])
def test_ties_go_to_the_even_code(x, c):
    assert _kv4.round_to(_kv4.GRID, np.array([x]))[0] == c


@pytest.mark.parametrize("D", [64, 128])
def test_layout_places_are_a_partition(D):
    kc, ks, vc, vs = _kv4.places(D)
    count = np.zeros(64 * (D + D // 8), int)
    for p in (kc, vc):
        np.add.at(count, p.ravel(), 1)
    assert set(count[np.unique(kc)]) == {2} and set(count[np.unique(vc)]) == {2}   # two codes a byte
    for p in (ks, vs):
        np.add.at(count, p.ravel(), 2)
    assert (count == 2).all()


@pytest.mark.parametrize("D", [64, 128])
def test_write_page_equals_token_by_token(D):
    rng = np.random.default_rng(1)
    c = lambda w, hi: rng.integers(0, hi, (64, w), dtype=np.uint8)  # noqa: E731
    kc, ks, vc, vs = c(D, 16), c(D // 16, 127), c(D, 16), c(D // 16, 127)
    a = rng.integers(0, 256, 64 * (D + D // 8), dtype=np.uint8)
    b = a.copy()
    for n in (64, 37):
        _kv4.write_page(a, D, kc, ks, vc, vs, n)
        for t in range(n):
            _kv4.write_token(b, t, D, kc[t], ks[t], vc[t], vs[t])
        assert np.array_equal(a, b)


def test_block_error_is_within_half_a_step():
    rng = np.random.default_rng(2)
    y = (rng.normal(size=(500, 64)) * rng.uniform(0.1, 20, (500, 1))).astype(np.float32)
    c, s = _kv4.quantise(y, np.ones(500)[:, None])
    v = _kv4.values(c, s, np.ones(500)[:, None])
    top = np.repeat(np.abs(y.reshape(500, 4, 16)).max(-1), 16, -1)
    # steps are at most 2 (between 4 and 6) in units of a scale of at most (1 + 2^-4) top/6
    assert (np.abs(v - y) <= top / 6 * (1 + 2.0 ** -4)).all()


def test_sizes(lib):
    assert moe.kv4_page_bytes(4, 128) == 4 * 9216 and moe.kv4_page_bytes(2, 64) == 2 * 4608
    assert moe.kv4_page_bytes(4, 96) == 0 and moe.kv4_page_bytes(0, 128) == 0
    assert moe.attention_kv4_workspace(32, 32, 4, 128) > 0
    assert moe.attention_kv4_workspace(32, 32, 5, 128) == 0      # heads do not divide
    assert lib.moe_kv4_pool_workspace(64, 100) >= 100 * 8 and lib.moe_kv4_pool_workspace(-1, 4) == 0
    assert "pages" in abi.status_string(abi.MOE_DEV_NO_PAGES, True)


def _cache(pages=FAKE, table=FAKE, lens=FAKE, n_pages=8, max_pages=4, S=2, n_kv=2, D=128):
    return abi._Kv4CacheParams(pages, table, lens, None, None, n_pages, max_pages, S, n_kv, D)


def _rope(table=FAKE, positions=FAKE, rot=128, n_pos=16, axes=1):
    return abi._RopeParams(table, positions, None, n_pos, rot, axes, 0)


def test_qk_norm_rope_rejects(lib):
    f = lib.moe_qk_norm_rope

    def call(x=FAKE, dt=1, ld=(4 + 4) * 128, T=4, nq=4, nkv=2, D=128, eps=1e-6, rope=None, qo=FAKE, ldq=512, ko=None, ldk=0,
             cache=None, qs=FAKE, w=None):
        return f(x, dt, ld, T, nq, nkv, D, w, None, eps, None if rope is None else ctypes.byref(rope), qo, ldq, ko, ldk,
                 None if cache is None else ctypes.byref(cache), qs, None, None)

    assert call(T=0) == 0                                   # nothing to do
    assert call(T=-1) == -1
    assert call(dt=2) == -1                                 # dtype
    assert call(D=96, ld=8 * 96) == -2                      # head size
    assert call(nkv=0) == -1
    assert call(nq=1021, ld=1025 * 128, ldq=1021 * 128) == -2   # too many heads
    assert call(eps=-1.0) == -1 and call(eps=float("nan")) == -1 and call(eps=float("inf")) == -1
    assert call(x=None) == -1 and call(x=ODD) == -1
    assert call(ld=8 * 128 - 8) == -1                       # rows overlap
    assert call(ld=8 * 128 + 4) == -1                       # rows off 16 bytes
    assert call(qo=None) == -1 and call(qo=ODD) == -1 and call(ldq=504) == -1
    assert call(ko=ODD, ldk=256) == -1 and call(ko=FAKE, ldk=128) == -1
    assert call(w=ODD) == -1
    assert call(rope=_rope(rot=160)) == -1 and call(rope=_rope(rot=0)) == -1
    assert call(rope=_rope(rot=48)) == -2                   # rot % 32
    assert call(rope=_rope(table=None)) == -1 and call(rope=_rope(table=ODD)) == -1 and call(rope=_rope(n_pos=0)) == -1
    assert call(rope=_rope(axes=0)) == -1
    assert call(rope=_rope(positions=None)) == -1           # places come from a cache
    assert call(cache=_cache(), qs=None) == -1
    assert call(cache=_cache(n_kv=4)) == -1 and call(cache=_cache(D=64)) == -1
    assert call(cache=_cache(pages=None)) == -1 and call(cache=_cache(pages=ODD)) == -1
    assert call(cache=_cache(S=20000)) == -2


def test_attention_rejects(lib):
    f = lib.moe_attention_kv4
    need = moe.attention_kv4_workspace(4, 8, 2, 128)

    def call(q=FAKE, ldq=1024, T=4, nq=8, cache=None, qs=FAKE, mx=1, scale=0.1, win=0, o=FAKE, ldo=1024, ws=FAKE, nb=None):
        c = _cache() if cache is None else cache
        return f(q, ldq, T, nq, ctypes.byref(c), qs, mx, scale, win, o, ldo, None, ws, need if nb is None else nb, None, None)

    assert call(T=0) == 0 and call(cache=_cache(S=0)) == 0
    assert f(FAKE, 1024, 4, 8, None, FAKE, 1, 0.1, 0, FAKE, 1024, None, FAKE, need, None, None) == -1   # no cache
    assert call(nq=7, ldq=1024) == -1                       # heads do not divide
    assert call(nq=0) == -1 and call(T=-1) == -1 and call(mx=-1) == -1 and call(win=-1) == -1
    assert call(scale=float("nan")) == -1 and call(scale=float("inf")) == -1
    assert call(qs=None) == -1
    assert call(q=None) == -1 and call(q=ODD) == -1 and call(ldq=1016) == -1 and call(ldq=1028) == -1
    assert call(o=None) == -1 and call(o=ODD) == -1 and call(ldo=1016) == -1
    assert call(ws=None) == -4 and call(nb=need - 1) == -4
    assert call(ws=ctypes.c_void_p((1 << 20) + 16)) == -1
    assert call(cache=_cache(D=32)) == -2 and call(cache=_cache(n_kv=0)) == -1 and call(cache=_cache(lens=None)) == -1


def test_read_rejects(lib):
    f = lib.moe_kv4_read
    c = _cache()
    assert f(None, FAKE, 4, FAKE, FAKE, None, None) == -1
    assert f(ctypes.byref(c), None, 4, FAKE, FAKE, None, None) == -1
    assert f(ctypes.byref(c), FAKE, -1, FAKE, FAKE, None, None) == -1
    assert f(ctypes.byref(c), FAKE, 4, ODD, FAKE, None, None) == -1
    assert f(ctypes.byref(c), FAKE, 4, None, None, None, None) == 0
    assert f(ctypes.byref(c), FAKE, 0, FAKE, FAKE, None, None) == 0


def test_pool_calls_reject(lib):
    def pool(pages=FAKE, stride=1 << 20, pb=9216, table=FAKE, lens=FAKE, ref=FAKE, layers=2, n=16, mp=4, S=3):
        return abi._Kv4PoolParams(pages, stride, pb, table, lens, ref, layers, n, mp, S)

    need = lib.moe_kv4_pool_workspace(3, 16)
    calls = [lambda p, ws=FAKE, nb=need, v=FAKE: lib.moe_kv4_reserve(ctypes.byref(p), v, ws, nb, None, None),
             lambda p, ws=FAKE, nb=need, v=FAKE: lib.moe_kv4_assign(ctypes.byref(p), v, None, None),
             lambda p, ws=FAKE, nb=need, v=FAKE: lib.moe_kv4_compact(ctypes.byref(p), v, ws, nb, None, None)]
    for f in calls:
        for bad in (dict(S=-1), dict(n=-1), dict(mp=-1), dict(layers=0), dict(pb=0), dict(pb=100), dict(stride=8), dict(table=None),
                    dict(lens=None), dict(ref=None), dict(pages=None), dict(pages=ODD)):
            assert f(pool(**bad)) == -1, bad
        assert f(pool(S=4097)) == -2
    for f in (calls[0], calls[2]):
        assert f(pool(), ws=None) == -4 and f(pool(), nb=need - 1) == -4
        assert f(pool(), ws=ctypes.c_void_p((1 << 20) + 16)) == -1
    assert calls[0](pool(), v=None) == -1 and calls[1](pool(), v=None) == -1
    assert calls[0](pool(S=0)) == 0 and calls[1](pool(S=0)) == 0


def test_binding_checks_shapes():
    cpu = torch.zeros(2, 2, 64 * 144, dtype=torch.uint8)
    with pytest.raises(moe.MoeError, match="CUDA"):
        moe.Kv4Cache(cpu, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 128)
    with pytest.raises(moe.MoeError, match="expected"):
        moe.Kv4Cache(cpu, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 64)
    with pytest.raises(moe.MoeError, match="rot/2"):
        moe.Rope(torch.zeros(4, 64))
    with pytest.raises(moe.MoeError, match="n_layers"):
        moe.Kv4Pool(cpu, torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 128)
