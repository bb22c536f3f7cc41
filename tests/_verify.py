"""Verification of drafted tokens in plain numpy, from the definition in
include/moe_gb300.h: one sequence at a time."""
from __future__ import annotations

import math

import numpy as np

F32 = np.float32
LOG2E = F32(float.fromhex("0x1.715476p+0"))
C = [F32(math.log(2) ** i / math.factorial(i)) for i in range(7)]


def weights(row, it):
    """w of every token of a row (fp32)."""
    m = row.max()
    with np.errstate(over="ignore"):
        t = np.maximum(((row - m).astype(F32) * it).astype(F32), F32(-60))
    n = np.rint(t)
    f = (t - n).astype(F32)
    p = np.full_like(t, C[6])
    for c in C[5::-1]:      # a product of two fp32 numbers is exact in fp64
        p = (p.astype(np.float64) * f + float(c)).astype(F32)
    return np.ldexp(p, n.astype(np.int32)).astype(F32)


def units(w):
    return np.rint(w.astype(np.float64) * 2.0 ** 42).astype(np.int64)


def verify(logits, tokens, uniform, q_start, draft=None, temperature=None):
    """(accepted, next, n_new) of every sequence."""
    out = []
    for s in range(len(q_start) - 1):
        r0, r1 = int(q_start[s]), int(q_start[s + 1])
        n = r1 - r0
        if n == 0:
            out.append((0, -1, 0))
            continue
        temp = F32(1) if temperature is None else F32(temperature[s])
        rows = logits[r0:r1].astype(F32)
        V = rows.shape[1]
        bad = not (temp >= 0 and np.isfinite(temp)) or not np.isfinite(rows.max(1)).all()
        drafts = tokens[r0 + 1:r1]
        bad = bad or ((drafts < 0) | (drafts >= V)).any()
        greedy = not bad and temp < F32(2.0 ** -60)
        d_rows = None
        if draft is not None and not greedy:
            d_rows = draft[r0:r1 - 1].astype(F32)
            bad = bad or (len(d_rows) and not np.isfinite(d_rows.max(1)).all())
        if bad:
            out.append((0, -1, -(n - 1)))
            continue
        if greedy:
            j = 0
            while j < n - 1 and tokens[r0 + j + 1] == rows[j].argmax():
                j += 1
            out.append((j, int(rows[j].argmax()), j - (n - 1)))
            continue
        it = F32(LOG2E / temp)
        j = 0
        while j < n - 1:
            x = int(tokens[r0 + j + 1])
            W = units(weights(rows[j], it))
            p = float(W[x]) / float(W.sum())
            q = 1.0
            if d_rows is not None:
                Q = units(weights(d_rows[j], it))
                q = float(Q[x]) / float(Q.sum())
            if not float(uniform[r0 + j + 1]) * q < p:
                break
            j += 1
        w = weights(rows[j], it)
        W = units(w)
        R = W
        if j < n - 1:
            if d_rows is None:
                R = W.copy()
                R[tokens[r0 + j + 1]] = 0
            else:
                wq = weights(d_rows[j], it)
                ip, iq = F32(2.0 ** 42 / float(W.sum())), F32(2.0 ** 42 / float(units(wq).sum()))
                R = units(np.maximum((w * ip).astype(F32) - (wq * iq).astype(F32), F32(0)))
            if R.sum() == 0:
                R = W
        total = int(R.sum())
        at = max(0, min(int(math.floor(float(uniform[r0]) * float(total))), total - 1))
        out.append((j, int(np.searchsorted(R.cumsum(), at, side="right")), j - (n - 1)))
    return tuple(np.array(c, np.int32) for c in zip(*out))
