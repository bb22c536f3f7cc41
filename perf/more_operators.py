"""Operators around the 4-bit cache of a decoder that serves, as cases to be timed and compared.

Four operators: products with weights in 4 bits ("linear"), the verification of
drafted tokens ("verify"), the attention weight that every cached token has
drawn ("weigh"), and the eviction of the tokens that drew least ("evict").
`run` computes them in plain torch where `own` is false and through
expert_routing_moe_gb300 where it is true.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64     # tokens of a page
BLOCK = 16    # numbers that share a scale
TILE = 128    # rows and columns of a tile of weights
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
LOG2E = float.fromhex("0x1.715476p+0")   # log2(e), nearest fp32
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    # 32 query heads over 4 cached heads of 128 numbers, and a hidden size of 2048, unless a case says otherwise
    big = {"hq": 32, "hk": 4, "d": 128}
    small = {"hq": 14, "hk": 2, "d": 64}
    return [
        # one user's next token, the projection to queries, keys and values: latency alone
        {"name": "linear-1", "op": "linear", "t": 1, "n": 5120, "k": 2048, "out": "bf16", "bias": False, "add": False},
        # a decode batch, the projection back, added to the residual
        {"name": "linear-32", "op": "linear", "t": 32, "n": 2048, "k": 4096, "out": "f32", "bias": False, "add": True},
        # the output head for a token and its four drafts
        {"name": "linear-head", "op": "linear", "t": 5, "n": 128001, "k": 2048, "out": "f32", "bias": False, "add": False},
        # a prompt chunk of odd length
        {"name": "linear-2001", "op": "linear", "t": 2001, "n": 5120, "k": 2048, "out": "bf16", "bias": True, "add": False},
        # one user, drafts looked up in the prompt (no distribution of their own)
        {"name": "verify-1", "op": "verify", "seqs": 1, "drafts": 4, "v": 32000, "dtype": "f32", "by_model": False, "idle": 0},
        # a batch whose drafts a small model sampled, an odd vocabulary
        {"name": "verify-32", "op": "verify", "seqs": 32, "drafts": 4, "v": 128001, "dtype": "bf16", "by_model": True, "idle": 2},
        # a decode batch of 32 ragged contexts
        {"name": "weigh-32", "op": "weigh", "seqs": 32, "new": 1, "ctx": 8192, **big, "window": 0, "last": 0, "idle": 2},
        # one user with a long document
        {"name": "weigh-long", "op": "weigh", "seqs": 1, "new": 1, "ctx": 131071, **big, "window": 0, "last": 0, "idle": 0},
        # prompt chunks of a small model, of which the last 64 rows count
        {"name": "weigh-last", "op": "weigh", "seqs": 6, "new": 500, "ctx": 9001, **small, "window": 0, "last": 64, "idle": 1},
        # a whole prompt, all of its rows
        {"name": "weigh-8192", "op": "weigh", "seqs": 1, "new": 8192, "ctx": 8192, **big, "window": 0, "last": 0, "idle": 0},
        # one user's long context cut to a quarter, in 48 layers
        {"name": "evict-1", "op": "evict", "seqs": 1, "ctx": 32001, "budget": 8192, "layers": 48, "hk": 4, "d": 128, "sinks": 4, "recent": 256},
        # a batch, each over its budget by a different amount or not at all
        {"name": "evict-32", "op": "evict", "seqs": 32, "ctx": 6000, "budget": 2000, "layers": 8, "hk": 4, "d": 128, "sinks": 4, "recent": 100},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    heads = rng.choice([(32, 4, 128), (14, 2, 64), (16, 16, 64), (8, 1, 128), (20, 2, 128), (12, 4, 64)])
    shape = {"hq": heads[0], "hk": heads[1], "d": heads[2]}
    op = rng.choice(["linear", "linear", "verify", "weigh", "weigh", "evict"])
    if op == "linear":
        t = _spread(rng, 1, 2000)
        k = 64 * _spread(rng, 2, 125) if rng.random() < 0.8 else _spread(rng, 100, 8000)
        n = _spread(rng, 100, min(128000, 260_000_000 // k, 20_000_000_000 // (k * t)))
        out = rng.choice(["bf16", "f32"])
        return {"op": op, "t": t, "n": n, "k": k, "out": out, "bias": rng.random() < 0.4, "add": out == "f32" and rng.random() < 0.5}
    if op == "verify":
        v, drafts = _spread(rng, 500, 150000), rng.randint(0, 7)
        by_model = rng.random() < 0.6
        seqs = _spread(rng, 1, max(1, min(64, 30_000_000 // (v * (1 + drafts) * (2 if by_model else 1)))))
        return {"op": op, "seqs": seqs, "drafts": drafts, "v": v, "dtype": rng.choice(["bf16", "f32"]), "by_model": by_model, "idle": rng.randint(0, min(3, seqs - 1))}
    if op == "weigh":
        kind = rng.choice(["step", "draft", "chunk"])
        seqs = _spread(rng, 1, 64) if kind != "chunk" else rng.randint(1, 4)
        new = 1 if kind == "step" else rng.randint(2, 7) if kind == "draft" else _spread(rng, 16, 2000)
        ctx = new + _spread(rng, 1, 16000 if kind == "chunk" else min(100000, 400000 // seqs))
        if kind == "chunk":
            seqs = max(1, min(seqs, 32_000_000 // (new * ctx)))
        return {"op": op, "seqs": seqs, "new": new, "ctx": ctx, **shape, "window": _spread(rng, 100, 4000) if rng.random() < 0.2 else 0,
                "last": _spread(rng, 1, 128) if kind == "chunk" and rng.random() < 0.5 else 0, "idle": rng.randint(0, min(3, seqs - 1))}
    layers = rng.choice([8, 24, 48])
    ctx = _spread(rng, 100, 30000)
    seqs = _spread(rng, 1, max(1, min(64, 1_500_000 // (layers * ctx))))
    budget = max(30, int(ctx * rng.uniform(0.1, 0.9)))
    sinks = rng.choice([0, 4, 70 if budget > 200 else 1])
    return {"op": op, "seqs": seqs, "ctx": ctx, "budget": budget, "layers": layers, "hk": heads[1], "d": heads[2], "sinks": sinks,
            "recent": rng.randint(0, (budget - sinks) // 2)}


# ---------------------------------------------------------------------------
# The sizes that a case stands for: from the case alone, so that its work is known.
# ---------------------------------------------------------------------------
def _sizes(case):
    """(new tokens, cached tokens with them) of each sequence; idle ones have one row and nothing cached."""
    rng = random.Random(case["seqs"] * 1000003 + case["ctx"] * 31 + case["new"])
    new, length = [], []
    for i in range(case["seqs"]):
        n = case["new"] if i == 0 or case["new"] == 1 else rng.randint(max(1, case["new"] // 3), case["new"])
        m = case["ctx"] if i == 0 else max(n, _spread(rng, 1, case["ctx"]))
        if 0 < i <= case["idle"]:
            n, m = 1, 0
        new.append(n)
        length.append(m)
    return new, length


def _drafts(case):
    """Drafted tokens of each sequence; -1 for a sequence without rows."""
    rng = random.Random(case["seqs"] * 7 + case["v"] + case["drafts"])
    return [-1 if 0 < i <= case["idle"] else case["drafts"] if i == 0 else rng.randint(case["drafts"] // 2, case["drafts"]) for i in range(case["seqs"])]


def _held(case):
    """(tokens, budget) of each sequence; -1: it is left as it is."""
    rng = random.Random(case["seqs"] + 13 * case["ctx"])
    out = []
    for i in range(case["seqs"]):
        n = case["ctx"] if i == 0 else rng.randint(max(1, case["ctx"] // 4), case["ctx"])
        out.append((n, -1 if i % 8 == 5 else case["budget"]))
    return out


def _columns(case):
    """Columns of a page table: a page more than the longest sequence has."""
    return -(-case["ctx"] // PAGE) + 1


def _counted(case):
    """Visible (query, key) pairs that count, and cached tokens that some such query sees."""
    pairs = seen = 0
    for n, m in zip(*_sizes(case)):
        if m == 0:
            continue
        first = m - (min(n, case["last"]) if case["last"] else n)   # place of the first row that counts
        w = case["window"] or m
        full = max(0, m - max(first, w - 1))                        # rows whose window is full
        pairs += full * w + sum(p + 1 for p in range(first, min(m, w - 1)))
        seen += m - max(0, first - w + 1)
    return pairs, seen


def work(case):
    if case["op"] == "linear":
        t, n, k = case["t"], case["n"], case["k"]
        out = t * n * (2 if case["out"] == "bf16" else 8 if case["add"] else 4)
        return {"bytes": n * k * 9 // 16 + n * (8 if case["bias"] else 4) + t * k * 2 + out, "flops": 2 * t * n * k}
    if case["op"] == "verify":
        rows, judged = sum(d + 1 for d in _drafts(case)), sum(max(0, d) for d in _drafts(case))
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": (rows + (judged if case["by_model"] else 0)) * case["v"] * size + rows * 8 + case["seqs"] * 16, "flops": 0}
    if case["op"] == "weigh":
        pairs, seen = _counted(case)
        new, length = _sizes(case)
        rows = sum(min(n, case["last"]) if case["last"] else n for n in new)
        keys = seen * case["hk"] * (case["d"] // 2 + case["d"] // 16)
        return {"bytes": keys + rows * case["hq"] * (2 * case["d"] + 4) + 8 * seen, "flops": 2 * case["d"] * case["hq"] * pairs}
    moved = read = 0
    for n, b in _held(case):
        if 0 <= b < n:
            moved += b - case["sinks"] // PAGE * PAGE   # the first tokens stay where they are
            read += n
    return {"bytes": 2 * moved * case["layers"] * case["hk"] * (case["d"] + case["d"] // 8) + 4 * read + 8 * moved, "flops": 0}


# ---------------------------------------------------------------------------
# Numbers in 4 bits (e2m1) with an 8-bit scale (e4m3) for every 16 of them
# ---------------------------------------------------------------------------
def _quantise(z):
    """Codes and scale bytes of the blocks of 16 along the last axis of z (fp32)."""
    b = z.unflatten(-1, (-1, BLOCK))
    s = (b.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    r = s.float()
    m = b * torch.where(r > 0, 1 / r, torch.zeros_like(r)).unsqueeze(-1)
    a = m.abs()
    c = torch.zeros_like(a, dtype=torch.uint8)
    for edge, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += a >= edge if up else a > edge     # to the nearest of E2M1, ties to the even code
    return (c | ((m < 0).byte() << 3)).flatten(-2), s.view(torch.uint8)


def _lut(dev):
    return torch.tensor(E2M1 + tuple(-x for x in E2M1), device=dev)


# Weights [n][k] lie in tiles of 128 rows and 128 columns, 9216 bytes each, [tiles of rows][tiles of columns]: the codes of
# row r, column 32 c + i at byte (r/8)*512 + c*128 + ((r%8) ^ (2c))*16 + i/8*4, where eight codes share a word, the even ones of
# them in its lower half; then the scales of row r, block b at 8192 + r*8 + b.  What lies beyond n or k is zero.
# Bits of a half, of the codes (sign, three bits of magnitude) j = 0 .. 3 in it:
_BITS = ((15, 8, 7, 6), (12, 5, 4, 3), (9, 2, 1, 0), (14, 13, 11, 10))


def _pack_weights(codes, scales):
    n, k = codes.shape
    nt, kt = -(-n // TILE), -(-k // TILE)
    dev = codes.device
    full = torch.zeros(nt * TILE, kt * TILE, dtype=torch.uint8, device=dev)
    full[:n, :k] = codes
    full = full.view(nt, 16, 8, kt, 4, 4, 4, 2)                                                  # ..., word, j, half
    low, high = torch.zeros_like(full[..., 0, :]), torch.zeros_like(full[..., 0, :])             # bytes of a half
    for j, bits in enumerate(_BITS):
        for i, to in enumerate(bits):
            bit = (full[..., j, :] >> (3 - i)) & 1
            low, high = (low, high | (bit << (to - 8))) if to >= 8 else (low | (bit << to), high)
    full = torch.stack([low, high], -1).flatten(-3).permute(0, 3, 1, 4, 2, 5)                    # [nt][kt][16][c][8][16 bytes]
    place = torch.arange(8, device=dev) ^ (2 * torch.arange(4, device=dev)[:, None])             # [c][place] -> row
    full = torch.gather(full, 4, place[:, :, None].expand(nt, kt, 16, 4, 8, 16))
    s = torch.zeros(nt * TILE, kt * 8, dtype=torch.uint8, device=dev)
    s[:n, :scales.shape[1]] = scales
    s = s.view(nt, TILE, kt, 8).permute(0, 2, 1, 3).reshape(nt, kt, 1024)
    return torch.cat([full.reshape(nt, kt, 8192), s], -1).contiguous()


def _unpack_weights(tiles, n, k):
    """The weights as fp32 values, without the rows' own scales."""
    nt, kt, _ = tiles.shape
    dev = tiles.device
    place = torch.arange(8, device=dev) ^ (2 * torch.arange(4, device=dev)[:, None])             # [c][row] -> place, its own inverse
    b = torch.gather(tiles[..., :8192].reshape(nt, kt, 16, 4, 8, 16), 4, place[:, :, None].expand(nt, kt, 16, 4, 8, 16))
    b = b.reshape(nt, kt, 16, 4, 8, 4, 2, 2)                                                     # ..., word, half, byte
    codes = []
    for bits in _BITS:
        c = torch.zeros_like(b[..., 0])
        for i, to in enumerate(bits):
            c |= ((b[..., to // 8] >> (to % 8)) & 1) << (3 - i)
        codes.append(c)
    b = torch.stack(codes, -2).flatten(-2)                                                       # j, half -> eight codes
    b = b.permute(0, 2, 4, 1, 3, 5, 6).reshape(nt * TILE, kt * TILE)[:n, :k]
    s = tiles[..., 8192:].reshape(nt, kt, TILE, 8).permute(0, 2, 1, 3).reshape(nt * TILE, kt * 8).contiguous()
    s = s.view(torch.float8_e4m3fn).float().repeat_interleave(BLOCK, -1)[:n, :k]
    return _lut(dev)[b.int()] * s


# A page of one head of the cache: the keys' codes and scales, the values' codes and scales.
#   keys     byte tok*(d/2) + i/2, the even i in the low half
#   scales   of token g + 8 i (g < 8), block b = t*(d/64) + r (t < 4): ((t*8 + g)*8 + i)*(d/64) + r
#   values   of tokens 2j and 2j + 1 (low and high half), number e = g*(d/8) + u: (((j/4)*8 + g)*4 + j%4)*(d/8) + u
#   scales   of token 2j + h, block b: ((b*4 + j%4)*8 + j/4)*2 + h
def _pack_pages(kc, ks, vc, vs):
    """Codes [n][64][heads][d] and scale bytes [n][64][heads][d/16] as pages [n][heads][bytes]."""
    n, _, h, d = kc.shape
    kc, ks, vc, vs = (t.permute(0, 2, 1, 3) for t in (kc, ks, vc, vs))
    k = kc.reshape(n, h, PAGE, d // 2, 2)
    k = k[..., 0] | (k[..., 1] << 4)
    s = ks.reshape(n, h, 8, 8, 4, d // 64).permute(0, 1, 4, 3, 2, 5)
    v = vc.reshape(n, h, PAGE // 2, 2, d)
    v = (v[:, :, :, 0] | (v[:, :, :, 1] << 4)).reshape(n, h, 8, 4, 8, d // 8).permute(0, 1, 2, 4, 3, 5)
    w = vs.reshape(n, h, 8, 4, 2, d // 16).permute(0, 1, 5, 3, 2, 4)
    return torch.cat([t.reshape(n, h, -1) for t in (k, s, v, w)], -1).contiguous()


def _split_pages(pages, d):
    """The inverse of _pack_pages: codes [n][64][heads][d] and scale bytes [n][64][heads][d/16] of keys, then of values."""
    n, h, _ = pages.shape
    a, b = PAGE * d // 2, PAGE * d // 16
    k, s, v, w = pages.split([a, b, a, b], -1)
    k = torch.stack([k & 15, k >> 4], -1).reshape(n, h, PAGE, d)
    s = s.reshape(n, h, 4, 8, 8, d // 64).permute(0, 1, 4, 3, 2, 5).reshape(n, h, PAGE, d // 16)
    v = v.reshape(n, h, 8, 8, 4, d // 8).permute(0, 1, 2, 4, 3, 5).reshape(n, h, PAGE // 2, 1, d)
    v = torch.cat([v & 15, v >> 4], 3).reshape(n, h, PAGE, d)
    w = w.reshape(n, h, d // 16, 4, 8, 2).permute(0, 1, 4, 3, 5, 2).reshape(n, h, PAGE, d // 16)
    return tuple(t.permute(0, 2, 1, 3) for t in (k, s, v, w))


def _keys(pages, d):
    """Keys [n][64][heads][d] in fp32, without the heads' own scales."""
    n, h, _ = pages.shape
    a, b = PAGE * d // 2, PAGE * d // 16
    k, s = pages[..., :a], pages[..., a:a + b]
    k = torch.stack([k & 15, k >> 4], -1).reshape(n, h, PAGE, d)
    s = s.reshape(n, h, 4, 8, 8, d // 64).permute(0, 1, 4, 3, 2, 5).reshape(n, h, PAGE, d // 16).contiguous()
    return (_lut(pages.device)[k.int()] * s.view(torch.float8_e4m3fn).float().repeat_interleave(BLOCK, -1)).permute(0, 2, 1, 3)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _starts(new, dev):
    return torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=dev)


def _page_tables(held, columns, order):
    """Tables whose pages are taken from `order`, in turn; -1 where a sequence has none."""
    table = np.full((len(held), columns), -1, np.int32)
    at = 0
    for i, n in enumerate(held):
        k = -(-n // PAGE)
        table[i, :k] = order[at:at + k]
        at += k
    return table, at


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(int(seed))
    r = np.random.RandomState(int(seed) % (1 << 32))
    normal = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    unit = lambda *s: torch.rand(*s, generator=g, device=dev)  # noqa: E731
    noise = lambda *s: torch.randint(0, 256, s, generator=g, device=dev, dtype=torch.uint8)  # noqa: E731
    s = {"case": dict(case)}
    if case["op"] == "linear":
        t, n, k = case["t"], case["n"], case["k"]
        w = torch.zeros(n, -(-k // BLOCK) * BLOCK, device=dev)
        w[:, :k] = normal(n, k) * (0.02 * (0.5 + unit(n, 1)))
        s["row_scale"] = (w.abs().amax(-1) / 2688).clamp(min=1e-30)
        codes, scales = _quantise(w / s["row_scale"][:, None])
        s["tiles"] = _pack_weights(codes[:, :k], scales)
        # normed activations with a few strong channels
        x = normal(t, k) * (0.5 + unit(k)) * (1 + 20 * (unit(k) < 0.005))
        s["x"] = x.to(torch.bfloat16)
        s["bias"] = normal(n) * 0.1 if case["bias"] else None
        s["y"] = torch.empty(t, n, dtype=DTYPES[case["out"]], device=dev)
        s["y0"] = normal(t, n) if case["add"] else None      # the residual that is added to
        return s
    if case["op"] == "verify":
        drafts, v = _drafts(case), case["v"]
        t, n_seq = sum(d + 1 for d in drafts), case["seqs"]
        # logits as a head gives them: a broad bulk and a few strong candidates; the drafting model's are near them
        logits = 2.5 * normal(t, v) + 6 * (unit(t, v) < 3 / v) * (1 + unit(t, v))
        other = logits + 0.7 * normal(t, v)
        # rows of a grammar that allows a part of the vocabulary
        masked = unit(t, 1) < 0.1
        hidden = masked & (unit(1, v) < 0.6)
        hidden[:, 7 % v] = False
        s["logits"] = logits.masked_fill_(hidden, -math.inf).to(DTYPES[case["dtype"]])
        # three settings a batch: greedy, cool and plain sampling
        temp = torch.tensor([(0.7, 1.0, 0.0)[i % 3] for i in range(n_seq)], device=dev)
        count = torch.tensor([d + 1 for d in drafts], device=dev)
        row_temp = temp.repeat_interleave(count)
        pick = other / row_temp.clamp(min=0.05)[:, None] - (-unit(t, v).clamp(min=1e-20).log()).log()
        tokens = torch.zeros(t, dtype=torch.int32, device=dev)
        tokens[1:] = pick[:-1].argmax(-1).int()      # a row's token was drafted from the row before
        s.update(tokens=tokens, uniform=unit(t), temperature=temp, q_start=_starts([d + 1 for d in drafts], dev),
                 draft_logits=other.to(DTYPES[case["dtype"]]) if case["by_model"] else None, rows=t)
        s.update({name: torch.empty(n_seq, dtype=torch.int32, device=dev) for name in ("accepted", "next", "n_new")})
        return s
    if case["op"] == "weigh":
        new, length = _sizes(case)
        h, d, columns = case["hk"], case["d"], _columns(case)
        total = sum(-(-n // PAGE) for n in length)
        table, _ = _page_tables(length, columns, r.permutation(total + 3))
        # keys with a few strong channels; what no token has written yet is whatever the memory held
        k = normal(total + 3, PAGE, h, d) * (0.6 + 1.4 * unit(d))
        codes, scales = _quantise(k)
        written = torch.zeros(total + 3, PAGE, dtype=torch.bool, device=dev)
        at = torch.arange(columns * PAGE, device=dev).reshape(columns, PAGE)
        table = torch.from_numpy(table).to(dev)
        for i, m in enumerate(length):
            n_pages = -(-m // PAGE)
            written[table[i, :n_pages].long()] = at[:n_pages] < m
        there = written[:, :, None, None]
        codes, scales = torch.where(there, codes, noise(total + 3, PAGE, h, d) & 15), torch.where(there, scales, noise(total + 3, PAGE, h, d // BLOCK))
        s["pages"] = _pack_pages(codes, scales, noise(total + 3, PAGE, h, d) & 15, noise(total + 3, PAGE, h, d // BLOCK) & 63)
        del k, codes, scales
        rows = sum(new)
        s.update(page_table=table, seq_len=torch.tensor(length, dtype=torch.int32, device=dev), q_start=_starts(new, dev), k_scale=0.5 + unit(h), rows=rows,
                 scale=1 / math.sqrt(d), q=(1.3 * normal(rows, case["hq"], d)).to(torch.bfloat16), lse=torch.empty(rows, case["hq"], device=dev))
        _weights(s, lambda sums, where, head: s["lse"].__setitem__(where, sums), lse_only=True)
        s["score0"] = unit(case["seqs"], columns * PAGE) * 3
        s["score"] = torch.empty_like(s["score0"])
        return s
    held = _held(case)
    lens = [n for n, _ in held]
    fresh = sum(-(-b // PAGE) for n, b in held if 0 <= b < n)
    used = sum(-(-n // PAGE) for n in lens)
    p = used + fresh + 3
    table, _ = _page_tables(lens, _columns(case), r.permutation(p))
    # a step that is tried: every page of a sequence is held once more, so that it can be taken back
    ref = np.zeros(p, np.int32)
    ref[table[table >= 0]] = 2
    saved = torch.from_numpy(np.concatenate([table.reshape(-1), np.array(lens, np.int32), ref])).to(dev)
    book, n_seq = saved.clone(), case["seqs"]
    a, b = n_seq * _columns(case), n_seq * _columns(case) + n_seq
    # attention weight: the first tokens draw much, few others some, most hardly any
    score = (2 * normal(n_seq, _columns(case) * PAGE)).exp() * 0.01
    score[:, :4] += 5
    s.update(saved=saved, book=book, page_table=book[:a].view(n_seq, -1), seq_len=book[a:b], ref=book[b:],
             pool=noise(case["layers"], p, case["hk"], PAGE * (case["d"] + case["d"] // 8)), score0=score, score=score.clone(),
             budget=torch.tensor([c for _, c in held], dtype=torch.int32, device=dev),
             kept=torch.empty(n_seq, case["budget"], dtype=torch.int32, device=dev))
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import expert_routing_moe_gb300 as moe
    case = s["case"]
    if case["op"] == "linear":
        if "handle" not in s:   # a program keeps the description of its weights, its cache or its pool
            s["handle"] = moe.Weight4(s["tiles"], case["n"], case["k"], s["row_scale"])
        if case["add"]:
            s["y"].copy_(s["y0"])
        moe.moe_linear_w4(s["x"], s["handle"], s["y"], bias=s["bias"], accumulate=case["add"])
        return {"y": s["y"]}
    if case["op"] == "verify":
        if "handle" not in s:
            s["handle"] = torch.zeros(moe.verify_workspace(s["rows"], case["seqs"], case["v"]), dtype=torch.uint8, device=s["logits"].device)
        moe.moe_verify_drafts(s["logits"], s["tokens"], s["uniform"], s["q_start"], s["accepted"], s["next"], s["n_new"], draft_logits=s["draft_logits"],
                              temperature=s["temperature"], workspace=s["handle"])
        return {"accepted": s["accepted"], "next": s["next"], "n_new": s["n_new"]}
    s["score"].copy_(s["score0"])
    if case["op"] == "weigh":
        if "handle" not in s:
            view = moe.Kv4Cache(s["pages"], s["page_table"], s["seq_len"], case["d"], s["k_scale"])
            n = moe.kv4_weigh_workspace(view, s["rows"], case["hq"])
            s["handle"] = view, torch.zeros(max(n, 256), dtype=torch.uint8, device=s["q"].device)
        view, ws = s["handle"]
        moe.moe_kv4_weigh(s["q"], view, s["q_start"], s["lse"], s["score"], s["scale"], max_new=case["new"], window=case["window"], last=case["last"], workspace=ws)
        return {"score": s["score"]}
    s["book"].copy_(s["saved"])   # back to the committed state
    if "handle" not in s:
        pool = moe.Kv4Pool(s["pool"], s["page_table"], s["seq_len"], s["ref"], case["d"])
        s["handle"] = pool, torch.zeros(moe.kv4_evict_workspace(pool), dtype=torch.uint8, device=s["pool"].device)
    pool, ws = s["handle"]
    moe.moe_kv4_evict(pool, s["score"], s["budget"], case["sinks"], case["recent"], ws, kept=s["kept"])
    return {"book": s["book"], "pool": s["pool"], "score": s["score"], "kept": s["kept"]}


def _run_plain(s):
    op = s["case"]["op"]
    if op == "linear":
        case = s["case"]
        y = s["x"].float() @ (_unpack_weights(s["tiles"], case["n"], case["k"]) * s["row_scale"][:, None]).t()
        if case["bias"]:
            y += s["bias"]
        if case["add"]:
            y += s["y0"]
        return {"y": y.to(DTYPES[case["out"]])}
    if op == "verify":
        return _verify(s)
    s["score"].copy_(s["score0"])
    if op == "weigh":
        def add(sums, where, head):
            s["score"] += sums
        _weights(s, add)
        return {"score": s["score"]}
    s["book"].copy_(s["saved"])
    return _evict(s)


def _weights(s, use, lse_only=False):
    """Attention's probabilities, a key head at a time: their sums over the rows that count go to `use`, or the rows' log-sum-exp."""
    case, length = s["case"], s["seq_len"].long()
    hq, hk, d = case["hq"], case["hk"], case["d"]
    group, n, most = hq // hk, length.numel(), case["new"]
    keys = _keys(s["pages"][s["page_table"].clamp(min=0).reshape(-1).long()], d).reshape(n, -1, hk, d)
    at = torch.arange(keys.shape[1], device=keys.device)
    keys = torch.where((at < length[:, None])[..., None, None], keys, torch.zeros_like(keys))
    start = s["q_start"].long()
    i = torch.arange(most, device=keys.device)
    count = start[1:] - start[:-1]
    if case["last"] and not lse_only:
        i = i[:min(most, case["last"])]
        skip = (count - case["last"]).clamp(min=0)
    else:
        skip = torch.zeros_like(count)
    i = i + skip[:, None]                                                   # [n][rows]
    good = i < count[:, None]
    row = (start[:-1, None] + i).clamp(max=s["rows"] - 1)
    pos = (length - count)[:, None] + i
    seen = (at <= pos[..., None]) & (at < length[:, None, None]) & good[..., None]
    if case["window"]:
        seen &= at > pos[..., None] - case["window"]
    for h in range(hk):
        q = s["q"][row, h * group:(h + 1) * group].float()                  # [n][rows][group][d]
        x = (q.flatten(1, 2) @ keys[:, :, h].transpose(1, 2)) * (s["scale"] * s["k_scale"][h])
        x = x.unflatten(1, (-1, group)).masked_fill_(~seen[:, :, None], -math.inf)
        if lse_only:
            use(torch.logsumexp(x, -1)[good], (slice(None), slice(h * group, (h + 1) * group)), h)
            continue
        z = s["lse"][row, h * group:(h + 1) * group][..., None]
        use(x.sub_(torch.where(torch.isfinite(z), z, torch.zeros_like(z))).exp_().sum((1, 2)), None, h)


def _weights_of_logits(logits, temp):
    """What a row's tokens weigh, relative to its strongest: fp32 numbers whose every operation is rounded in a known way, so
    that whole numbers made of them are the same for everybody.  2^t with t = n + f by the series of 2^f in Horner's form with
    fused products."""
    m = logits.amax(-1, keepdim=True)
    t = ((logits - m) * (torch.tensor(LOG2E, device=m.device) / temp)[:, None]).clamp(min=-60)
    n = t.round()
    f = (t - n).double()
    c = [float(np.float32(math.log(2) ** i / math.factorial(i))) for i in range(7)]
    p = torch.full_like(t, c[6])
    for i in range(5, -1, -1):
        p = (p.double() * f + c[i]).float()
    return p * ((n.int() + 127) << 23).view(torch.float32)


def _whole(w):
    """Numbers from 0 to 1 as multiples of 2^-42."""
    return (w.double() * 2.0 ** 42).round().long()


def _verify(s):
    case, temp, start = s["case"], s["temperature"], s["q_start"].long()
    v, rows, n_seq = case["v"], s["rows"], case["seqs"]
    dev = temp.device
    count = start[1:] - start[:-1]
    seq = torch.arange(n_seq, device=dev).repeat_interleave(count)
    greedy = (temp == 0)[seq]
    row_temp = torch.where(greedy, torch.ones_like(seq, dtype=torch.float32), temp[seq])
    token = torch.cat([s["tokens"][1:].long(), s["tokens"][:1].long()])[:, None]     # the draft that a row judges
    logits = s["logits"].float()
    w = _weights_of_logits(logits, row_temp)
    best = (logits == logits.amax(-1, keepdim=True)).int().argmax(-1)
    only = torch.zeros_like(w).scatter_(1, best[:, None], 1.0)
    w = torch.where(greedy[:, None], only, w)
    whole = _whole(w)
    total = whole.sum(-1)
    p = whole.gather(1, token).squeeze(1).double() / total.double()
    q = torch.ones_like(p)
    if case["by_model"]:
        wq = _weights_of_logits(s["draft_logits"].float(), row_temp)
        whole_q = _whole(wq)
        total_q = whole_q.sum(-1)
        q = torch.where(greedy, q, whole_q.gather(1, token).squeeze(1).double() / total_q.double())
    u = torch.cat([s["uniform"][1:], s["uniform"][:1]]).double()
    r = torch.arange(rows, device=dev)
    last = r == (start[1:] - 1)[seq]
    stop = last | ~(u * q < p)                      # a row after which nothing is accepted
    first = torch.full((n_seq,), rows, device=dev).scatter_reduce(0, seq, torch.where(stop, r, torch.full_like(r, rows)), "amin")
    live = count > 0
    first = torch.where(live, first, torch.zeros_like(first))
    accepted = torch.where(live, first - start[:-1], torch.zeros_like(first))
    # the token that follows: from the target where all was accepted, else from what the target has beyond the draft
    refused = live & ~last[first]
    mine = whole[first]
    if case["by_model"]:
        inv_p, inv_q = ((2.0 ** 42 / z.double()).float()[first, None] for z in (total, total_q))
        beyond = _whole((w[first] * inv_p - wq[first] * inv_q).clamp(min=0))
        beyond = torch.where(greedy[first, None], mine, beyond)
    else:
        beyond = mine.scatter(1, token[first], torch.zeros_like(mine[:, :1]))
    beyond = torch.where((refused & (beyond.sum(-1) > 0))[:, None], beyond, mine)
    sums = beyond.cumsum(-1)
    all_ = sums[:, -1]
    at = (s["uniform"][start[:-1].clamp(max=rows - 1)].double() * all_.double()).floor().long()
    at = torch.minimum(at.clamp(min=0), all_ - 1)
    following = (sums > at[:, None]).int().argmax(-1)
    i32 = torch.int32
    return {"accepted": accepted.to(i32), "next": torch.where(live, following, torch.full_like(following, -1)).to(i32),
            "n_new": torch.where(live, accepted - count + 1, torch.zeros_like(accepted)).to(i32)}


def _evict(s):
    """The best tokens by score, with the first and the last ones, in their order; whatever page a reference more holds is left and a free one written."""
    case, table, length, ref = s["case"], s["page_table"], s["seq_len"], s["ref"]
    score, d, sinks, recent = s["score"], case["d"], case["sinks"], case["recent"]
    n_seq, columns = table.shape
    dev = table.device
    was, budget = length.long(), s["budget"].long()
    cut = (budget >= 0) & (budget < was)
    now = torch.where(cut, budget, was)
    at = torch.arange(score.shape[1], device=dev)
    there = at < was[:, None]
    always = there & ((at < sinks) | (at >= (was - recent)[:, None]))
    order = torch.where(always, torch.full_like(score, math.inf), torch.where(there, score, torch.full_like(score, -math.inf)))
    rank = torch.empty_like(order, dtype=torch.long)
    rank.scatter_(1, order.argsort(dim=1, descending=True, stable=True), at.expand(n_seq, -1).contiguous())
    keep = there & (rank < now[:, None])
    old = torch.where(keep, at, torch.full_like(at, 1 << 30)).sort(1).values             # [n_seq][places]: the kept tokens' old places
    kept = torch.where(old < 1 << 30, old, torch.full_like(old, -1))
    first = torch.where(keep | ~there, torch.full_like(at, 1 << 30), at).amin(1) // PAGE  # the page of the first token that goes
    score.copy_(torch.where(cut[:, None] & there, torch.where(kept >= 0, score.gather(1, kept.clamp(min=0)), torch.zeros_like(score)), score))
    column = torch.arange(columns, device=dev)
    written = cut[:, None] & (column >= first[:, None]) & (column < ((now + PAGE - 1) // PAGE)[:, None])
    dropped = cut[:, None] & (column >= ((now + PAGE - 1) // PAGE)[:, None]) & (table >= 0)
    from_page = table.gather(1, (kept // PAGE).clamp(min=0))
    fresh = written & (ref[table.clamp(min=0).long()] > 1)
    free = torch.argsort((ref != 0).to(torch.uint8), stable=True)
    place = free[(fresh.reshape(-1).cumsum(0) - 1).clamp(min=0)].reshape(fresh.shape).int()
    gone = fresh | dropped
    ref.index_add_(0, table.clamp(min=0).reshape(-1).long(), -gone.reshape(-1).int())
    ref.index_add_(0, place.reshape(-1).long(), fresh.reshape(-1).int())
    table.copy_(torch.where(dropped, torch.full_like(table, -1), torch.where(fresh, place, table)))
    length.copy_(now.int())
    # the tokens of the pages that are written, from the pages as they were
    which, col = torch.nonzero(written, as_tuple=True)
    tok = (col[:, None] * PAGE + torch.arange(PAGE, device=dev))                          # [pages][64] places
    src = kept[which[:, None], tok]
    page, off, real = from_page[which[:, None], tok].long(), (src % PAGE), src >= 0
    to = table[which, col].long()
    for layer in range(case["layers"]):
        parts = _split_pages(s["pool"][layer], d)
        new = [torch.where(real[..., None, None], t[page, off], torch.zeros_like(t[:1, :1])) for t in parts]
        s["pool"][layer][to] = _pack_pages(*new)
    cols = s["kept"].shape[1]
    s["kept"].fill_(-1)
    width = min(cols, kept.shape[1])
    s["kept"][:, :width] = kept[:, :width].int()
    return {"book": s["book"], "pool": s["pool"], "score": s["score"], "kept": s["kept"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, written apart from the plain forms
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "verify":
        return None   # whole numbers
    s = prepare(case, seed)
    if case["op"] == "evict":     # of its floating outputs; the rest are whole numbers
        score = s["score0"].cpu().numpy().copy()
        for i, (n, b) in enumerate(_held(case)):
            if 0 <= b < n:
                middle = range(min(case["sinks"], n), max(min(case["sinks"], n), n - case["recent"]))
                best = sorted(middle, key=lambda j: (-score[i, j], j))[:b - (n - len(middle))]
                left = sorted(set(range(n)) - set(middle) | set(best))
                score[i, :n] = np.concatenate([score[i, left], np.zeros(n - b, np.float32)])
        return {"book": None, "pool": None, "score": torch.from_numpy(score).double(), "kept": None}
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        dev = s["x"].device
        value = torch.tensor([(-1.0 if c & 8 else 1.0) * E2M1[c & 7] for c in range(16)], dtype=torch.float64, device=dev)
        y = torch.empty(case["t"], n, dtype=torch.float64, device=dev)
        col = torch.arange(k, device=dev)
        x = s["x"].double()
        for r0 in range(0, n, 8192):
            r = torch.arange(r0, min(n, r0 + 8192), device=dev)[:, None]
            tile = s["tiles"].reshape(-1)
            base = ((r // TILE) * s["tiles"].shape[1] + col // TILE) * 9216
            c, i, q = col % TILE // 32, col % 32, r % TILE
            byte = base + q // 8 * 512 + c * 128 + ((q % 8) ^ (2 * c)) * 16 + i // 8 * 4 + i % 2 * 2
            half = tile[byte].int() + 256 * tile[byte + 1].int()
            at = torch.tensor(_BITS, device=dev).int()[i % 8 // 2]                              # [k][4]
            code = sum(((half >> at[:, b]) & 1) << (3 - b) for b in range(4))
            scale = tile[base + 8192 + q * 8 + col % TILE // BLOCK].contiguous().view(torch.float8_e4m3fn).double()
            y[:, r0:r0 + r.shape[0]] = x @ (value[code] * scale * s["row_scale"][r0:r0 + r.shape[0], None].double()).t()
        if case["bias"]:
            y = y + s["bias"].double()
        return {"y": y + s["y0"].double() if case["add"] else y}
    hq, hk, d = case["hq"], case["hk"], case["d"]
    start, length = s["q_start"].tolist(), s["seq_len"].tolist()
    out = s["score0"].double()
    for i, m in enumerate(length):
        n = start[i + 1] - start[i]
        if m == 0:
            continue
        pages = s["pages"][s["page_table"][i, :-(-m // PAGE)].long()]
        keys = _keys(pages, d).reshape(-1, hk, d)[:m].double()
        lo = n - min(n, case["last"]) if case["last"] else 0
        place = torch.arange(m, device=keys.device)
        for b in range(lo, n, 1024):
            pos = torch.arange(m - n + b, m - n + min(n, b + 1024), device=keys.device)[:, None]
            hidden = place > pos
            if case["window"]:
                hidden |= place <= pos - case["window"]
            for h in range(hq):
                c = h // (hq // hk)
                rows = slice(start[i] + b, start[i] + min(n, b + 1024))
                x = s["q"][rows, h].double() @ keys[:, c].t() * (s["scale"] * s["k_scale"][c].double()) - s["lse"][rows, h, None].double()
                out[i, :m] += torch.exp(x).masked_fill(hidden, 0.0).sum(0)
    return {"score": out}
