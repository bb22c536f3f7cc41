"""The operators of the attention half of a decoder layer, as cases to be timed and compared.

Three operators: the norm and rotation of queries and keys with the append to
a cache held in 4 bits ("rotate"), attention over that cache ("attend"), and
the pages of the cache ("beam": reorder and grow the beams of a search;
"compact": pack the pool's live pages).  `run` computes them in plain torch
where `own` is false and through expert_routing_moe_gb300 where it is true.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 64     # tokens of a page
BLOCK = 16    # numbers that share a scale
EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    # 32 query heads over 4 cached heads of 128 numbers unless a case says otherwise
    big = {"hq": 32, "hk": 4, "d": 128}
    small = {"hq": 14, "hk": 2, "d": 64}
    return [
        # one user's next token: latency alone
        {"name": "rotate-1", "op": "rotate", "seqs": 1, "new": 1, "ctx": 1500, **big, "axes": 1, "dtype": "bf16", "cached": True, "pairs": False},
        # a decode batch of a model that sees images
        {"name": "rotate-64", "op": "rotate", "seqs": 64, "new": 1, "ctx": 30000, **big, "axes": 3, "dtype": "bf16", "cached": True, "pairs": False},
        # a few odd prompts in fp32 without a cache, pairs side by side
        {"name": "rotate-f32-777", "op": "rotate", "seqs": 3, "new": 259, "ctx": 259, **small, "axes": 3, "dtype": "f32", "cached": False, "pairs": True},
        # a prefill batch: 8192 new tokens
        {"name": "rotate-8192", "op": "rotate", "seqs": 4, "new": 2048, "ctx": 5000, **big, "axes": 3, "dtype": "bf16", "cached": True, "pairs": False},
        # one user, short context: latency alone
        {"name": "attend-1", "op": "attend", "seqs": 1, "new": 1, "ctx": 333, **big, "window": 0, "idle": 0},
        # a decode batch of 32 ragged contexts
        {"name": "attend-32", "op": "attend", "seqs": 32, "new": 1, "ctx": 8192, **big, "window": 0, "idle": 2},
        # one user with a long document
        {"name": "attend-long", "op": "attend", "seqs": 1, "new": 1, "ctx": 131071, **big, "window": 0, "idle": 0},
        # a windowed layer of a small model, four drafted tokens a sequence
        {"name": "attend-window", "op": "attend", "seqs": 48, "new": 4, "ctx": 6000, **small, "window": 1000, "idle": 3},
        # prompt chunks behind a cached prefix
        {"name": "attend-chunk", "op": "attend", "seqs": 4, "new": 500, "ctx": 9001, **big, "window": 0, "idle": 0},
        # a whole prompt
        {"name": "attend-8192", "op": "attend", "seqs": 1, "new": 8192, "ctx": 8192, **big, "window": 0, "idle": 0},
        # one step of a beam search, the pages of 48 layers: reorder, then room for a token each
        {"name": "beam-8x8", "op": "beam", "groups": 8, "beams": 8, "ctx": 1000, "layers": 48, "hk": 4, "d": 128, "pages": 512},
        # half of a pool is free, in holes
        {"name": "compact-4096", "op": "compact", "seqs": 100, "ctx": 2600, "layers": 8, "hk": 4, "d": 128, "pages": 4096},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    heads = rng.choice([(32, 4, 128), (14, 2, 64), (16, 16, 64), (8, 1, 128), (24, 2, 128), (12, 4, 64)])
    shape = {"hq": heads[0], "hk": heads[1], "d": heads[2]}
    op = rng.choice(["rotate", "attend", "attend", "attend", "beam", "compact"])
    if op == "rotate":
        tokens = _spread(rng, 1, 8000)
        seqs = rng.randint(1, min(tokens, 64))
        new = max(1, tokens // seqs)
        cached = rng.random() < 0.75
        return {"op": op, "seqs": seqs, "new": new, "ctx": new + _spread(rng, 1, 30000), **shape, "axes": rng.choice([1, 3]),
                "dtype": "bf16" if rng.random() < 0.7 else "f32", "cached": cached, "pairs": rng.random() < 0.3}
    if op == "attend":
        kind = rng.choice(["step", "draft", "chunk"])
        seqs = _spread(rng, 1, 64) if kind != "chunk" else rng.randint(1, 4)
        new = 1 if kind == "step" else rng.randint(2, 7) if kind == "draft" else _spread(rng, 16, 2000)
        ctx = new + _spread(rng, 1, 16000 if kind == "chunk" else min(100000, 400000 // seqs))
        if kind == "chunk":
            seqs = max(1, min(seqs, 32_000_000 // (new * ctx)))
        return {"op": op, "seqs": seqs, "new": new, "ctx": ctx, **shape, "window": _spread(rng, 100, 4000) if rng.random() < 0.25 else 0,
                "idle": rng.randint(0, min(3, seqs - 1))}
    layers = rng.choice([4, 8, 24, 48])
    if op == "beam":
        groups, beams, ctx = rng.randint(1, 8), rng.randint(2, 8), _spread(rng, 20, 1500)
        return {"op": op, "groups": groups, "beams": beams, "ctx": ctx, "layers": layers, "hk": heads[1], "d": heads[2],
                "pages": groups * (-(-ctx // PAGE) + 3 * beams) + rng.randint(0, 100)}
    seqs, ctx = rng.randint(2, 100), _spread(rng, 40, 2600)
    return {"op": op, "seqs": seqs, "ctx": ctx, "layers": 8, "hk": heads[1], "d": heads[2], "pages": 2 + int(seqs * (ctx / PAGE + 1) * rng.uniform(1.0, 1.5))}


# ---------------------------------------------------------------------------
# The sizes that a case stands for: from the case alone, so that its work is known.
# ---------------------------------------------------------------------------
def _sizes(case):
    """(new tokens, cached tokens with them) of each sequence; idle ones have one row and nothing cached."""
    rng = random.Random(case["seqs"] * 1000003 + case["ctx"] * 31 + case["new"])
    new, length = [], []
    for i in range(case["seqs"]):
        n = case["new"] if i == 0 or case["new"] == 1 or case["op"] == "rotate" else rng.randint(max(1, case["new"] // 3), case["new"])
        m = case["ctx"] if i == 0 else max(n, _spread(rng, 1, case["ctx"]))
        if i > 0 and i <= case.get("idle", 0):
            n, m = 1, 0
        new.append(n)
        length.append(m)
    return new, length


def _pairs(case):
    """Visible (query, key) pairs, and cached tokens that some query of their sequence sees."""
    pairs = seen = 0
    for n, m in zip(*_sizes(case)):
        if m == 0:
            continue
        w = case["window"] or m
        first, last = m - n, m - 1                  # positions of the new tokens
        full = max(0, last - max(first, w - 1) + 1)  # those whose window is full
        pairs += full * w + sum(p + 1 for p in range(first, min(last, w - 2) + 1))
        seen += m - max(0, first - w + 1)
    return pairs, seen


def _page_bytes(case):
    return case["hk"] * PAGE * (case["d"] + case["d"] // 8)


def _parents(case):
    """Each beam's parent in its group, and one finished group (no parent)."""
    rng = random.Random(case["groups"] * 1009 + case["beams"] * 31 + case["ctx"])
    out = []
    for g in range(case["groups"]):
        for b in range(case["beams"]):
            out.append(-1 if g == 1 and case["groups"] > 2 else g * case["beams"] + rng.choice([b, rng.randrange(case["beams"])]))
    return out


def _beam_lengths(case):
    rng = random.Random(case["groups"] + 77 * case["ctx"])
    return [max(1, case["ctx"] - rng.randrange(PAGE)) for _ in range(case["groups"])]


def _held(case):
    rng = random.Random(case["seqs"] + 13 * case["ctx"])
    return [rng.randint(max(1, case["ctx"] // 4), case["ctx"]) for _ in range(case["seqs"])]


def work(case):
    if case["op"] == "rotate":
        tokens = case["seqs"] * case["new"]
        size = 2 if case["dtype"] == "bf16" else 4
        heads, rows = case["hq"] + 2 * case["hk"], tokens * case["d"]
        read = rows * size * (heads if case["cached"] else case["hq"] + case["hk"]) + tokens * (case["d"] * 4 + 4 * case["axes"])
        kv = case["hk"] * tokens * (case["d"] + case["d"] // 8)
        # the cached numbers are written once in 4 bits, and read and returned as values
        write = rows * size * case["hq"] + (2 * kv + rows * 2 * 2 * case["hk"] if case["cached"] else rows * size * case["hk"])
        return {"bytes": read + write, "flops": rows * heads * 10}
    if case["op"] == "attend":
        pairs, seen = _pairs(case)
        rows = sum(_sizes(case)[0])
        return {"bytes": seen * case["hk"] * (case["d"] + case["d"] // 8) + rows * case["hq"] * (4 * case["d"] + 4), "flops": 4 * case["d"] * case["hq"] * pairs}
    if case["op"] == "beam":
        parents, lengths, copies = _parents(case), _beam_lengths(case), 0
        for g, n in enumerate(lengths):
            kept = [p for p in parents[g * case["beams"]:(g + 1) * case["beams"]] if p >= 0]
            if n % PAGE:
                copies += sum(kept.count(p) - 1 for p in set(kept))
        book = 8 * (case["groups"] * case["beams"] * (_columns(case) + 1) + case["pages"])
        return {"bytes": 2 * copies * case["layers"] * _page_bytes(case) + book, "flops": 0}
    live = sum(-(-n // PAGE) for n in _held(case))
    moved = live * max(0, case["pages"] - live) / case["pages"]   # live pages beyond the first `live` ones, as they lie at random
    return {"bytes": 2 * moved * case["layers"] * _page_bytes(case) + 8 * (case["seqs"] * _columns(case) + case["pages"]), "flops": 0}


def _columns(case):
    """Columns of a page table: a page more than the longest sequence has."""
    return -(-case["ctx"] // PAGE) + 1


# ---------------------------------------------------------------------------
# The cache in 4 bits, in plain torch.  A page of one head: the keys' codes, the
# keys' scales, the values' codes, the values' scales.
#   keys     byte tok*(d/2) + i/2, the even i in the low half
#   scales   of token g + 8 i (g < 8), block b = t*(d/64) + r (t < 4): ((t*8 + g)*8 + i)*(d/64) + r
#   values   of tokens 2j and 2j + 1 (low and high half), number e = g*(d/8) + u: (((j/4)*8 + g)*4 + j%4)*(d/8) + u
#   scales   of token 2j + h, block b: ((b*4 + j%4)*8 + j/4)*2 + h
# ---------------------------------------------------------------------------
def _pack(kc, ks, vc, vs):
    """Codes [n][64][heads][d] and scale bytes [n][64][heads][d/16] as pages [n][heads][bytes]."""
    n, _, h, d = kc.shape
    kc, ks, vc, vs = (t.permute(0, 2, 1, 3) for t in (kc, ks, vc, vs))       # [n][h][64][.]
    k = kc.reshape(n, h, PAGE, d // 2, 2)
    k = k[..., 0] | (k[..., 1] << 4)
    s = ks.reshape(n, h, 8, 8, 4, d // 64).permute(0, 1, 4, 3, 2, 5)         # i g t r -> t g i r
    v = vc.reshape(n, h, PAGE // 2, 2, d)
    v = (v[:, :, :, 0] | (v[:, :, :, 1] << 4)).reshape(n, h, 8, 4, 8, d // 8).permute(0, 1, 2, 4, 3, 5)
    w = vs.reshape(n, h, 8, 4, 2, d // 16).permute(0, 1, 5, 3, 2, 4)         # j/4 j%4 h b -> b j%4 j/4 h
    return torch.cat([t.reshape(n, h, -1) for t in (k, s, v, w)], -1).contiguous()


def _unpack(pages, d):
    """The inverse of _pack, as values without the heads' own scales: keys and values [n][64][heads][d] in fp32."""
    n, h, _ = pages.shape
    a, b = PAGE * d // 2, PAGE * d // 16
    k, s, v, w = pages.split([a, b, a, b], -1)
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=pages.device)
    k = torch.stack([k & 15, k >> 4], -1).reshape(n, h, PAGE, d)
    s = s.reshape(n, h, 4, 8, 8, d // 64).permute(0, 1, 4, 3, 2, 5).reshape(n, h, PAGE, d // 16)
    v = v.reshape(n, h, 8, 8, 4, d // 8).permute(0, 1, 2, 4, 3, 5).reshape(n, h, PAGE // 2, 1, d)
    v = torch.cat([v & 15, v >> 4], 3).reshape(n, h, PAGE, d)
    w = w.reshape(n, h, d // 16, 4, 8, 2).permute(0, 1, 4, 3, 5, 2).reshape(n, h, PAGE, d // 16)
    out = []
    for codes, scales in ((k, s), (v, w)):
        scales = scales.contiguous().view(torch.float8_e4m3fn).float().repeat_interleave(BLOCK, -1)
        out.append((lut[codes.long()] * scales).permute(0, 2, 1, 3))
    return out


def _quantise(z):
    """Codes and scale bytes of the blocks of 16 along the last axis of z (fp32)."""
    b = z.unflatten(-1, (-1, BLOCK))
    s = (b.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    r = s.float()
    m = b * torch.where(r > 0, 1 / r, torch.zeros_like(r)).unsqueeze(-1)
    a = m.abs()
    # to the nearest of E2M1, ties to the even code
    c = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5).byte()
    return (c | ((m < 0).byte() << 3)).flatten(-2), s.view(torch.uint8)


def _value(codes, scales):
    lut = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=codes.device)
    return lut[codes.long()] * scales.view(torch.float8_e4m3fn).float().repeat_interleave(BLOCK, -1)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _table(n_pos, rot, dev):
    """(cos, sin) of every position and frequency, from 64-bit angles: far ones keep their places."""
    f = 1e6 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
    angle = torch.arange(n_pos, device=dev, dtype=torch.float64)[:, None] * f
    return torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()


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
    noise = lambda *s: torch.randint(0, 256, s, generator=g, device=dev, dtype=torch.uint8)  # noqa: E731
    s = {"case": dict(case)}
    if case["op"] in ("rotate", "attend"):
        new, length = _sizes(case)
        h, d, columns = case["hk"], case["d"], _columns(case)
        total = sum(-(-n // PAGE) for n in length)
        order = r.permutation(total + 3)
        table, _ = _page_tables(length, columns, order)
        s.update(q_start=_starts(new, dev), seq_len=torch.tensor(length, dtype=torch.int32, device=dev), page_table=torch.from_numpy(table).to(dev),
                 k_scale=(0.5 + torch.rand(h, generator=g, device=dev)), v_scale=(0.5 + torch.rand(h, generator=g, device=dev)), rows=sum(new))
    if case["op"] == "rotate":
        dt, t, d = DTYPES[case["dtype"]], sum(new), case["d"]
        heads = case["hq"] + 2 * case["hk"]
        # activations: heads of different sizes, and a few numbers far out
        x = normal(t, heads, d) * (0.3 + 2 * torch.rand(heads, 1, generator=g, device=dev))
        x *= 1 + 9 * (torch.rand(t, heads, d, generator=g, device=dev) < 0.003)
        pos = torch.cat([torch.arange(m - n, m, device=dev, dtype=torch.int32) for n, m in zip(new, length)])
        rot = d
        if case["axes"] == 3:
            # half of the tokens are an image 37 wide: their time stands still, their rows and columns count
            image = (torch.arange(t, device=dev) // 100) % 2 == 1
            at = torch.arange(t, device=dev, dtype=torch.int32) % 100
            base = pos - at
            pos = torch.stack([torch.where(image, base, pos), torch.where(image, base + at // 37, pos), torch.where(image, base + at % 37, pos)]).clamp(min=0)
            axis = [0] * (rot // 8) + [1] * (3 * rot // 16) + [2] * (3 * rot // 16) if not case["pairs"] else [i % 3 for i in range(rot // 2)]
        else:
            pos, axis = pos[None], [0] * (rot // 2)
        s.update(qkv=x.reshape(t, heads * d).to(dt), positions=pos.to(torch.int32).contiguous(), axis=torch.tensor(axis, dtype=torch.uint8, device=dev), table=_table(case["ctx"] + 200, rot, dev),
                 q_weight=1 + 0.2 * normal(d), k_weight=1 + 0.2 * normal(d), q_out=torch.empty(t, case["hq"], d, dtype=dt, device=dev))
        if case["cached"]:
            s.update(pages=noise(total + 3, case["hk"], PAGE * (d + d // 8)), k_val=torch.empty(t, case["hk"], d, dtype=torch.bfloat16, device=dev),
                     v_val=torch.empty(t, case["hk"], d, dtype=torch.bfloat16, device=dev))
        else:
            s.update(k_out=torch.empty(t, case["hk"], d, dtype=dt, device=dev))
        return s
    if case["op"] == "attend":
        # keys with a few strong channels and a first token that draws attention, as normed keys have them
        k = normal(total + 3, PAGE, h, d) * (0.6 + 1.4 * torch.rand(d, generator=g, device=dev))
        v = normal(total + 3, PAGE, h, d)
        pages = _pack(*_quantise(k), *_quantise(v))
        # what no token has written yet is whatever the memory held
        written = torch.zeros(total + 3, PAGE, dtype=torch.bool, device=dev)
        at = torch.arange(columns * PAGE, device=dev).reshape(columns, PAGE)
        for i, m in enumerate(length):
            k_pages = -(-m // PAGE)
            written[s["page_table"][i, :k_pages].long()] = at[:k_pages] < m
        junk = _pack(noise(total + 3, PAGE, h, d) & 15, noise(total + 3, PAGE, h, d // 16), noise(total + 3, PAGE, h, d) & 15, noise(total + 3, PAGE, h, d // 16))
        s["pages"] = _merge(pages, junk, written, d)
        s.update(q=(1.3 * normal(s["rows"], case["hq"], d)).to(torch.bfloat16), out=torch.empty(s["rows"], case["hq"], d, dtype=torch.bfloat16, device=dev),
                 lse=torch.empty(s["rows"], case["hq"], device=dev), scale=1 / math.sqrt(d))
        return s
    p = case["pages"]
    if case["op"] == "beam":
        n_seq = case["groups"] * case["beams"]
        lengths = _beam_lengths(case)
        order = r.permutation(p)
        table, at = np.full((n_seq, _columns(case)), -1, np.int32), 0
        ref, lens = np.zeros(p, np.int32), np.zeros(n_seq, np.int32)
        for i in range(n_seq):
            m = lengths[i // case["beams"]]
            full, part = m // PAGE, -(-m // PAGE) - m // PAGE
            if i % case["beams"] == 0:   # a group shares the full pages of its prompt
                shared = order[at:at + full]
                at += full
            table[i, :full] = shared
            table[i, full:full + part] = order[at:at + part]
            at += part
            lens[i] = m
        for i in range(n_seq):
            ref[table[i][table[i] >= 0]] += 1
        s.update(parent=torch.tensor(_parents(case), dtype=torch.int32, device=dev))
        s["n_new"] = (s["parent"] >= 0).int()
    else:
        lens = np.array(_held(case), np.int32)
        table, at = _page_tables(lens, _columns(case), r.permutation(p))
        ref = np.zeros(p, np.int32)
        ref[table[table >= 0]] = 1
        s.update(n_live=torch.empty(1, dtype=torch.int32, device=dev))
    n_seq = len(lens)
    saved = torch.from_numpy(np.concatenate([table.reshape(-1), lens, ref])).to(dev)
    book = saved.clone()
    a, b = n_seq * _columns(case), n_seq * _columns(case) + n_seq
    s.update(saved=saved, book=book, page_table=book[:a].view(n_seq, -1), seq_len=book[a:b], ref=book[b:],
             pool=noise(case["layers"], p, case["hk"], PAGE * (case["d"] + case["d"] // 8)))
    return s


def _merge(pages, junk, written, d):
    """`pages` where a token was written, `junk` elsewhere, number by number."""
    ones, n, h = torch.full((1,), 15, dtype=torch.uint8, device=pages.device), pages.shape[0], pages.shape[1]
    m = written[:, :, None, None].byte()
    four = (m * ones).expand(n, PAGE, h, d).contiguous()
    full = (m * 255).expand(n, PAGE, h, d // 16).contiguous()
    mask = _pack(four, full, four, full)
    return (pages & mask) | (junk & ~mask)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import expert_routing_moe_gb300 as moe
    case = s["case"]
    if case["op"] == "rotate":
        if "handle" not in s:   # a program keeps the description of its cache and of its positions
            view = moe.Kv4Cache(s["pages"], s["page_table"], s["seq_len"], case["d"], s["k_scale"], s["v_scale"]) if case["cached"] else None
            s["handle"] = view, moe.Rope(s["table"], s["positions"], s["axis"], pairs=case["pairs"])
        view, rope = s["handle"]
        if case["cached"]:
            moe.moe_qk_norm_rope(s["qkv"], case["hq"], case["hk"], s["q_out"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, rope=rope, cache=view,
                                 q_start=s["q_start"])
            moe.moe_kv4_read(view, s["q_start"], s["k_val"], s["v_val"])
            return {"q": s["q_out"], "k": s["k_val"], "v": s["v_val"]}
        moe.moe_qk_norm_rope(s["qkv"], case["hq"], case["hk"], s["q_out"], s["k_out"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, rope=rope)
        return {"q": s["q_out"], "k": s["k_out"]}
    if case["op"] == "attend":
        if "handle" not in s:
            view = moe.Kv4Cache(s["pages"], s["page_table"], s["seq_len"], case["d"], s["k_scale"], s["v_scale"])
            n = moe.attention_kv4_workspace(s["rows"], case["hq"], case["hk"], case["d"])
            s["handle"] = view, torch.zeros(n, dtype=torch.uint8, device=s["q"].device)
        view, ws = s["handle"]
        moe.moe_attention_kv4(s["q"], view, s["q_start"], s["out"], s["scale"], max_new=case["new"], window=case["window"], lse=s["lse"], workspace=ws)
        return {"out": s["out"], "lse": s["lse"]}
    s["book"].copy_(s["saved"])   # back to the committed state, as a program that tries a step does
    if "handle" not in s:
        pool = moe.Kv4Pool(s["pool"], s["page_table"], s["seq_len"], s["ref"], case["d"])
        s["handle"] = pool, torch.zeros(moe.kv4_pool_workspace(pool), dtype=torch.uint8, device=s["pool"].device)
    pool, ws = s["handle"]
    if case["op"] == "beam":
        moe.moe_kv4_assign(pool, s["parent"])
        moe.moe_kv4_reserve(pool, s["n_new"], ws)
        return {"book": s["book"], "pool": s["pool"]}
    moe.moe_kv4_compact(pool, s["n_live"], ws)
    return {"book": s["book"], "pool": s["pool"], "live": s["n_live"]}


def _run_plain(s):
    op = s["case"]["op"]
    if op == "rotate":
        return _rotate(s)
    if op == "attend":
        return _attend(s)
    s["book"].copy_(s["saved"])
    return _beam(s) if op == "beam" else _compact(s)


def _rotate(s):
    case = s["case"]
    hq, hk, d, dt = case["hq"], case["hk"], case["d"], s["qkv"].dtype
    x = s["qkv"].reshape(-1, hq + 2 * hk, d).float()
    x, v = x[:, :hq + hk], x[:, hq + hk:]
    w = torch.cat([s["q_weight"].expand(hq, d), s["k_weight"].expand(hk, d)])
    # the sum of the squares in 64 bits: the keys' codes stand next to borders
    mean = x.double().square().sum(-1, keepdim=True).float() / d
    y = x * (1 / (mean + EPS).sqrt()) * w
    cs = s["table"][s["positions"][s["axis"].long()].long(), torch.arange(d // 2, device=x.device)[:, None]]   # [d/2][t][2]
    cos, sin = (cs[..., i].t()[:, None] for i in (0, 1))
    a, b = (y[..., 0::2], y[..., 1::2]) if case["pairs"] else y.chunk(2, -1)
    p, q = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([p, q], -1).flatten(-2) if case["pairs"] else torch.cat([p, q], -1)
    out, k = y[:, :hq].to(dt), y[:, hq:]
    if not case["cached"]:
        return {"q": out, "k": k.to(dt)}
    ks, vs = s["k_scale"][:, None], s["v_scale"][:, None]
    return {"q": out, "k": (_value(*_quantise(k * (1 / ks))) * ks).bfloat16(), "v": (_value(*_quantise(v * (1 / vs))) * vs).bfloat16()}


def _attend(s):
    case, table, length = s["case"], s["page_table"], s["seq_len"].long()
    hq, hk, d = case["hq"], case["hk"], case["d"]
    n, most = table.shape[0], case["new"]
    k, v = (t.reshape(n, -1, hk, d) for t in _unpack(s["pages"][table.clamp(min=0).reshape(-1).long()], d))
    at = torch.arange(k.shape[1], device=k.device)
    there = (at < length[:, None])[..., None, None]
    k = torch.where(there, k, torch.zeros_like(k)) * s["k_scale"][:, None]
    v = torch.where(there, v, torch.zeros_like(v)) * s["v_scale"][:, None]
    start = s["q_start"].long()
    i = torch.arange(most, device=k.device)
    count = start[1:] - start[:-1]
    row = (start[:-1, None] + i).clamp(max=s["rows"] - 1)
    q = s["q"][row].float().reshape(n, most, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, d)    # rows: head, then token
    pos = (length - count)[:, None] + i
    seen = (at <= pos[..., None]) & (at < length[:, None, None])
    if case["window"]:
        seen &= at > pos[..., None] - case["window"]
    x = (q @ k.permute(0, 2, 3, 1)) * s["scale"]
    x = x.unflatten(2, (hq // hk, most)).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = (x - torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v.permute(0, 2, 1, 3)).unflatten(2, (hq // hk, most)) / torch.where(total > 0, total, torch.ones_like(total))
    lse = (top + total.log()).squeeze(-1)
    lse = torch.where(total.squeeze(-1) > 0, lse, torch.full_like(lse, -math.inf))
    good = i < count[:, None]
    return {"out": o.permute(0, 3, 1, 2, 4).reshape(n, most, hq, d)[good].bfloat16(), "lse": lse.permute(0, 3, 1, 2).reshape(n, most, hq)[good]}


def _beam(s):
    """Tables and lengths of the parents, references counted anew; then room for n_new tokens, and shared last pages copied."""
    table, length, ref, parent = s["page_table"], s["seq_len"], s["ref"], s["parent"].long()
    old, was = table.clone(), length.clone()
    alive = parent >= 0
    table.copy_(torch.where(alive[:, None], old[parent.clamp(min=0)], torch.full_like(old, -1)))
    length.copy_(torch.where(alive, was[parent.clamp(min=0)], torch.zeros_like(was)))
    count = torch.zeros(ref.numel() + 1, dtype=torch.int64, device=ref.device)
    one = torch.ones(table.numel(), dtype=torch.int64, device=ref.device)
    change = count.scatter_add(0, table.reshape(-1).long() % count.numel(), one) - count.scatter_add(0, old.reshape(-1).long() % count.numel(), one)
    ref += change[:-1].int()
    # the last page of a sequence that grows is copied if it is partly full and shared, but for the last one of those that share it when nobody else does
    n = torch.arange(table.shape[0], device=ref.device)
    grows = s["n_new"] > 0
    held = (length + PAGE - 1) // PAGE
    last = table[n, (held - 1).clamp(min=0).long()].long()
    part = grows & (length % PAGE != 0)
    same = part[:, None] & part & (last[:, None] == last)                  # [s][s']
    keeps = (same.sum(1) == ref[last.clamp(min=0)]) & (torch.where(same, n, torch.full_like(n, -1)).amax(1) == n)
    copies = part & (ref[last.clamp(min=0)] > 1) & ~keeps
    after = length + s["n_new"]
    need = (after + PAGE - 1) // PAGE
    column = torch.arange(table.shape[1], device=ref.device)
    fresh = (column >= held[:, None]) & (column < need[:, None]) & grows[:, None]
    want = torch.cat([copies[:, None], fresh], 1)
    free = torch.argsort((ref != 0).to(torch.uint8), stable=True)
    place = free[(want.reshape(-1).cumsum(0) - 1).clamp(min=0)].reshape(want.shape).int()
    ref.index_add_(0, last.clamp(min=0), -copies.int())
    ref.index_add_(0, place.reshape(-1).long(), want.reshape(-1).int())
    table.copy_(torch.where(fresh, place[:, 1:], table))
    at = (held - 1).clamp(min=0).long()[:, None]
    table.scatter_(1, at, torch.where(copies[:, None], place[:, :1], table.gather(1, at)))
    length.copy_(after)
    s["pool"][:, place[:, 0][copies].long()] = s["pool"][:, last[copies]]
    return {"book": s["book"], "pool": s["pool"]}


def _compact(s):
    """The live pages beyond the first `live` ones move, in order, to the free pages below."""
    table, ref = s["page_table"], s["ref"]
    live = ref != 0
    n = live.sum()
    at = torch.arange(ref.numel(), device=ref.device)
    source, target = torch.nonzero(live & (at >= n)).squeeze(1), torch.nonzero(~live & (at < n)).squeeze(1)
    to = at.clone()
    to[source] = target
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    ref[target] = ref[source]
    ref[source] = 0
    s["pool"][:, target] = s["pool"][:, source]
    return {"book": s["book"], "pool": s["pool"], "live": n.int().reshape(1)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, written apart from the plain forms
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] in ("beam", "compact"):
        return None   # whole numbers
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(s)
    hq, hk, d = case["hq"], case["hk"], case["d"]
    start, length = s["q_start"].tolist(), s["seq_len"].tolist()
    out = torch.zeros(s["rows"], hq, d, dtype=torch.float64, device=s["q"].device)
    lse = torch.full((s["rows"], hq), -math.inf, dtype=torch.float64, device=s["q"].device)
    for i, m in enumerate(length):
        n = start[i + 1] - start[i]
        if m == 0:
            continue
        k, v = (t.reshape(-1, hk, d)[:m].double() for t in _unpack(s["pages"][s["page_table"][i, :-(-m // PAGE)].long()], d))
        pos = torch.arange(m - n, m, device=k.device)[:, None]
        key = torch.arange(m, device=k.device)
        hidden = (key > pos) | ((key <= pos - case["window"]) if case["window"] else torch.zeros_like(key, dtype=torch.bool))
        for h in range(hq):
            c = h // (hq // hk)
            x = s["q"][start[i]:start[i + 1], h].double() @ (k[:, c] * s["k_scale"][c].double()).t() * s["scale"]
            x = x.masked_fill(hidden, -math.inf)
            z = torch.logsumexp(x, -1, keepdim=True)
            lse[start[i]:start[i + 1], h] = z.squeeze(-1)
            out[start[i]:start[i + 1], h] = torch.exp(x - z) @ (v[:, c] * s["v_scale"][c].double())
    return {"out": out, "lse": lse}


def _exact_rotate(s):
    case = s["case"]
    hq, hk, d = case["hq"], case["hk"], case["d"]
    x = s["qkv"].double().reshape(-1, hq + 2 * hk, d)
    half = torch.arange(d // 2, device=x.device)
    first, second = (2 * half, 2 * half + 1) if case["pairs"] else (half, half + d // 2)
    cos, sin = s["table"][s["positions"].long().t()[:, s["axis"].long()], half].double().unsqueeze(1).unbind(-1)   # [t][1][d/2]
    y = x[:, :hq + hk]
    y = y / torch.sqrt((y ** 2).mean(-1, keepdim=True) + EPS)
    y = torch.cat([y[:, :hq] * s["q_weight"].double(), y[:, hq:] * s["k_weight"].double()], 1)
    a, b = y[..., first], y[..., second]
    y[..., first], y[..., second] = a * cos - b * sin, a * sin + b * cos
    if not case["cached"]:
        return {"q": y[:, :hq], "k": y[:, hq:]}
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)

    def cached(y, scale):
        z = y / scale.double()[:, None]
        b = z.reshape(z.shape[0], hk, d // BLOCK, BLOCK)
        top = (b.abs().amax(-1, keepdim=True) / 6).clamp(max=448)
        e = torch.floor(torch.log2(top.clamp(min=2.0 ** -20))).clamp(min=-6)    # e4m3: three bits behind the first, subnormals below 2^-6
        sc = torch.round(top / 2 ** (e - 3)) * 2 ** (e - 3)
        m = torch.where(sc > 0, b / sc.clamp(min=1e-30), torch.zeros_like(b))
        far = (m.abs().unsqueeze(-1) - grid).abs()
        near = far.amin(-1, keepdim=True) == far
        low = torch.where(near, torch.arange(8, device=x.device), torch.full((8,), 99, device=x.device)).amin(-1)
        code = torch.where((near.sum(-1) == 2) & (low % 2 == 1), low + 1, low)   # a tie goes to the even one
        return (grid[code] * m.sign() * sc).reshape(z.shape) * scale.double()[:, None]

    return {"q": y[:, :hq], "k": cached(y[:, hq:], s["k_scale"]), "v": cached(x[:, hq + hk:], s["v_scale"])}
