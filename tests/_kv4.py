"""The 4-bit paged cache and the operators on it in plain numpy, written from
the definitions in include/moe_gb300.h: values in 64 bits, bytes one by one."""
from __future__ import annotations

import numpy as np

PAGE, BLOCK = 64, 16
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
F32 = np.float32


def page_bytes(n_kv, D):
    return n_kv * PAGE * (D + D // 8)


def e4m3_values():
    """All e4m3 numbers >= 0 by their byte (0x7f is NaN)."""
    b = np.arange(127)
    e, m = b >> 3, b & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


E4M3 = e4m3_values()


def round_to(grid, x):
    """Index of the nearest member of an ascending grid, ties to the even index."""
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantise(y, hs):
    """Codes [..., D] and scale bytes [..., D/16] of y (fp32), each step rounded to fp32."""
    z = (y.astype(F32) * (F32(1) / np.asarray(hs, F32))).astype(F32)
    b = z.reshape(z.shape[:-1] + (z.shape[-1] // BLOCK, BLOCK))
    top = np.minimum((np.abs(b).max(-1) * F32(1 / 6)).astype(F32), F32(448))
    s = round_to(E4M3, top.astype(np.float64)).astype(np.uint8)
    sv = E4M3[s].astype(F32)
    r = np.where(sv > 0, F32(1) / np.where(sv > 0, sv, F32(1)), F32(0)).astype(F32)
    m = (b * r[..., None]).astype(F32)
    c = round_to(GRID, np.minimum(np.abs(m), 6).astype(np.float64)).astype(np.uint8)
    c |= ((m < 0).astype(np.uint8) << 3)
    return c.reshape(z.shape), s


def values(codes, scales, hs):
    """c * s * hs in 64 bits."""
    c = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return c * np.repeat(E4M3[scales], BLOCK, -1) * np.asarray(hs, np.float64)


def places(D):
    """Byte (within a head's part of a page) of every key code, key scale, value code
    and value scale, from the layout's definition."""
    tok = np.arange(PAGE)[:, None]
    i, b = np.arange(D)[None], np.arange(D // BLOCK)[None]
    o = 0
    kc = o + tok * (D // 2) + i // 2
    o += PAGE * D // 2
    R = D // 64
    ks = o + (((b // R) * 8 + tok % 8) * 8 + tok // 8) * R + b % R
    o += PAGE * D // 16
    j, U = tok // 2, D // 8
    vc = o + (((j // 4) * 8 + i // U) * 4 + j % 4) * U + i % U
    o += PAGE * D // 2
    vs = o + ((b * 4 + j % 4) * 8 + j // 4) * 2 + tok % 2
    return kc, ks, vc, vs


def write_token(page, tok, D, kc, ks, vc, vs):
    """One token of one head into its part of a page (uint8 vector)."""
    pkc, pks, pvc, pvs = places(D)
    i = np.arange(D)
    for e in i:
        sh = 4 * (e & 1)
        at = pkc[tok, e]
        page[at] = (page[at] & (0xF0 >> sh)) | (kc[e] << sh)
        sh = 4 * (tok & 1)
        at = pvc[tok, e]
        page[at] = (page[at] & (0xF0 >> sh)) | (vc[e] << sh)
    page[pks[tok]] = ks
    page[pvs[tok]] = vs


def write_page(page, D, kc, ks, vc, vs, n):
    """The first n tokens of a head's part of a page; the rest keeps its bytes.  kc, vc [64][D], ks, vs [64][D/16]."""
    pkc, pks, pvc, pvs = places(D)
    page[pkc[:n, 0::2]] = kc[:n, 0::2] | (kc[:n, 1::2] << 4)
    page[pks[:n]] = ks[:n]
    even = np.arange(0, n, 2)
    low = vc[even]
    high = np.where((even + 1 < n)[:, None], vc[np.minimum(even + 1, PAGE - 1)], page[pvc[even]] >> 4)
    page[pvc[even]] = low | (high << 4)
    page[pvs[:n]] = vs[:n]


class Cache:
    """A random cache on the host: keys/values of `lengths` tokens, pages in a random order, and
    junk (NaN scales among it) wherever no token was written."""

    def __init__(self, rng, lengths, n_kv, D, scales=True, spare=2, extra_columns=1, outliers=True):
        self.n_kv, self.D, self.lengths = n_kv, D, list(lengths)
        S = len(lengths)
        pages = [-(-n // PAGE) for n in lengths]
        total = sum(pages) + spare
        self.columns = max(pages + [0]) + extra_columns
        order = rng.permutation(total)
        self.table = np.full((S, self.columns), -1, np.int32)
        self.k_scale = rng.uniform(0.3, 3, n_kv).astype(F32) if scales else None
        self.v_scale = rng.uniform(0.3, 3, n_kv).astype(F32) if scales else None
        self.bytes = rng.integers(0, 256, (total, n_kv, PAGE * (D + D // 8)), dtype=np.uint8)
        _, pks, _, pvs = places(D)
        self.bytes[:, :, pks] = np.where(rng.random((total, n_kv) + pks.shape) < 0.5, 0x7F, 0xFF).astype(np.uint8)
        self.bytes[:, :, pvs] = np.where(rng.random((total, n_kv) + pvs.shape) < 0.5, 0x7F, 0xFF).astype(np.uint8)
        self.k, self.v = [], []
        at = 0
        for s, n in enumerate(lengths):
            self.table[s, :pages[s]] = order[at:at + pages[s]]
            at += pages[s]
            k = rng.normal(size=(n, n_kv, D)) * rng.uniform(0.5, 1.5, D)
            v = rng.normal(size=(n, n_kv, D)) * rng.uniform(0.2, 3, (n, 1, 1))
            if outliers and n:
                k[0] *= 3
            hk = (self.k_scale if scales else np.ones(n_kv, F32))[:, None]
            hv = (self.v_scale if scales else np.ones(n_kv, F32))[:, None]
            kc, ks = quantise(k.astype(F32), hk)
            vc, vs = quantise(v.astype(F32), hv)
            self.k.append(values(kc, ks, hk))
            self.v.append(values(vc, vs, hv))
            for p in range(pages[s]):
                m = min(PAGE, n - p * PAGE)
                for h in range(n_kv):
                    pad = [np.concatenate([x[p * PAGE:p * PAGE + m, h], np.zeros((PAGE - m, x.shape[-1]), np.uint8)])
                           for x in (kc, ks, vc, vs)]
                    write_page(self.bytes[self.table[s, p], h], D, *pad, m)


def attention(cache, q, q_start, scale, window=0):
    """(out, lse, error bound of out, of lse) in 64 bits.  q [T][n_q][D] float64 (bf16 values).

    The bounds: a score is a sum of D exact products of fp16 numbers added in fp32, off by at most
    2^-20 of the sum of their magnitudes (a few roundings or truncations of 2^-23 for each 16 products);
    a probability is off by that (as an exponent), 2^-20 for the exponential and 2^-11 for its
    rounding to fp16 (2^-25 where it is subnormal); sums of fp32 add 2^-18; the output is rounded to bf16."""
    T, n_q, D = q.shape
    G = n_q // cache.n_kv
    out, lse = np.zeros((T, n_q, D)), np.full((T, n_q), -np.inf)
    tol, tol_lse = np.zeros((T, n_q, D)), np.zeros((T, n_q))
    for s, length in enumerate(cache.lengths):
        q0, n = q_start[s], q_start[s + 1] - q_start[s]
        for i in range(n):
            p = length - n + i
            lo = max(0, p - window + 1) if window else 0
            if p < 0:
                continue
            k, v = cache.k[s][lo:p + 1], cache.v[s][lo:p + 1]
            for h in range(n_q):
                kh, vh = k[:, h // G], v[:, h // G]
                x = kh @ q[q0 + i, h] * scale
                off = (np.abs(kh) @ np.abs(q[q0 + i, h])).max() * abs(scale) * 2.0 ** -20
                m = x.max()
                e = np.exp(x - m)
                l = e.sum()
                o = e @ vh / l
                size = e @ np.abs(vh) / l
                out[q0 + i, h], lse[q0 + i, h] = o, m + np.log(l)
                rel = 2.0 ** -11 + 2 * off + 2.0 ** -18
                tiny = 2.0 ** -25 * np.abs(vh).sum(0) / l
                tol[q0 + i, h] = 2.0 ** -8 * np.abs(o) + rel * size + (2 * off + 2.0 ** -18) * np.abs(o) + tiny
                tol_lse[q0 + i, h] = 2 * off + 2.0 ** -18 + 2.0 ** -22 * abs(lse[q0 + i, h])
    return out, lse, tol, tol_lse
