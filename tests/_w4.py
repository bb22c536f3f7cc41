"""Weights in 4 bits in plain numpy, written from the definitions in
include/moe_gb300.h: values in 64 bits, bits one by one."""
from __future__ import annotations

import numpy as np

import _kv4

F32 = np.float32
BITS = ((15, 8, 7, 6), (12, 5, 4, 3), (9, 2, 1, 0), (14, 13, 11, 10))


def n_bytes(N, K):
    return -(-N // 128) * -(-K // 128) * 9216


def places(N, K):
    """For every (n, k): byte of its half word, index j of its code in it; and the byte of its scale."""
    n, k = np.arange(N)[:, None], np.arange(K)[None]
    kt = -(-K // 128)
    base = ((n // 128) * kt + k // 128) * 9216
    r, kk = n % 128, k % 128
    c = kk // 32
    half = base + (r // 8) * 512 + c * 128 + ((r % 8) ^ (2 * c)) * 16 + kk % 32 // 8 * 4 + kk % 2 * 2
    return half, np.broadcast_to(kk % 8 // 2, half.shape), base + 8192 + r * 8 + kk // 16


def pack_codes(codes, scales):
    """Tiles of codes [N][K] and scale bytes [N][ceil(K/16)]."""
    N, K = codes.shape
    half, j, sc = places(N, K)
    out = np.zeros(n_bytes(N, K), np.uint8)
    words = out.view(np.uint16)
    for jj, bits in enumerate(BITS):
        at = half[j == jj] // 2
        c = codes[j == jj].astype(np.uint16)
        for i, to in enumerate(bits):
            np.bitwise_or.at(words, at, ((c >> (3 - i)) & 1).astype(np.uint16) << np.uint16(to))
    out[sc] = np.repeat(scales, 16, 1)[:, :K]
    return out


def quantise(w):
    """(codes, scale bytes, row scales) of w [N][K] fp32 by the rules of moe_w4_pack."""
    N, K = w.shape
    z = np.zeros((N, -(-K // 16) * 16), F32)
    z[:, :K] = np.where(np.isfinite(w), w, 0)
    hs = (np.abs(z).max(1) * F32(1 / 2688)).astype(F32)
    hs = np.where(hs >= F32(2.0 ** -100), hs, F32(1))
    codes, scales = _kv4.quantise(z, hs[:, None])
    return codes[:, :K], scales, hs


def values(codes, scales, hs):
    K = codes.shape[1]
    c = _kv4.GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return c * np.repeat(_kv4.E4M3[scales], 16, 1)[:, :K] * np.asarray(hs, np.float64)[:, None]


def linear(x, w, bias=None, y0=None, out_eps=0.0):
    """(y, bound of its error) in 64 bits.  Products are exact; each of the K/16 accumulating tensor-core steps rounds
    or truncates once, by at most 2^-23 of a sum no larger than the products' magnitudes, as do up to 16 joins; the row's scale,
    bias and residual round by 2^-24 each; then the output's own rounding of half a step."""
    y = x @ w.T
    size = np.abs(x) @ np.abs(w).T
    tol = size * ((x.shape[1] / 16 + 16) * 2.0 ** -23)
    for extra in (bias, y0):
        if extra is not None:
            y = y + extra
            tol = tol + 2.0 ** -24 * (np.abs(extra) + np.abs(y))
    return y, tol + np.abs(y) * (2.0 ** -23 + out_eps / 2) + 1e-38
