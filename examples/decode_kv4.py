"""A small mixture-of-experts decoder served from a 4-bit cache: prompts, decode
steps replayed from one CUDA graph, a prompt forked into beams, and the pool
packed.  Random weights; prints tokens/s and the cache's size.

With --drafts n the decode goes on with n drafted tokens a sequence and step: a
4-bit head's logits accept or refuse them, and the refused ones leave the cache.  With
--budget b the layers weigh their cached tokens, and the caches are then cut
to the b tokens that drew most.  --four-bit: the projections in 4 bits too.

    python examples/decode_kv4.py [--layers 4] [--batch 32] [--prompt 500] [--steps 64] [--drafts 4] [--budget 256] [--four-bit]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import __graft_entry__ as entry  # noqa: E402
import expert_routing_moe_gb300 as moe  # noqa: E402


class Layer:
    """x += attention(norm(x)); x += experts(norm(x)), the residual x in fp32."""

    def __init__(self, H, n_q, n_kv, D, N, I, k, max_tokens, table, gen, dev, four_bit, weighs):
        bf = torch.bfloat16
        w = lambda *s: (torch.randn(*s, generator=gen, device=dev) * s[-1] ** -0.5)  # noqa: E731
        ones = torch.ones(D, device=dev)
        form = moe.Weight4.pack if four_bit else lambda t: t
        self.attention = moe.AttentionLayer(form(w((n_q + 2 * n_kv) * D, H).to(bf)), form(w(H, n_q * D).to(bf)), n_q, n_kv, max_tokens, ones, ones,
                                            table=table, weighs=weighs)
        self.experts = moe.MoELayer(w(N, H), w(N, I, H).to(bf), w(N, I, H).to(bf), w(N, H, I).to(bf), k=k, max_tokens=max_tokens)

    @staticmethod
    def norm(x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def forward(self, x, cache, q_start, max_new, positions=None, score=None, fresh=True):
        x += self.attention.forward(self.norm(x), cache, q_start, max_new, positions, score, 32, fresh)
        self.experts.forward(self.norm(x), accumulate_into=x)


def speculate(a, S, H, pages, run, positions, gen, dev):
    """Steps of a.drafts drafted tokens a sequence, from one graph."""
    n, V = a.drafts + 1, a.vocabulary
    i32 = dict(dtype=torch.int32, device=dev)
    words = torch.randn(V, H, generator=gen, device=dev)
    head = moe.Weight4.pack((words * H ** -0.5).bfloat16())
    tokens, uniform, q_start = torch.zeros(S, n, **i32), torch.zeros(S * n, device=dev), torch.arange(0, S * n + 1, n, **i32)
    accepted, token, n_new = (torch.zeros(S, **i32) for _ in range(3))
    logits, taken = torch.zeros(S * n, V, device=dev), torch.zeros(1, dtype=torch.int64, device=dev)
    workspace = torch.zeros(moe.verify_workspace(S * n, S, V), dtype=torch.uint8, device=dev)
    status, room, behind = torch.zeros(2, **i32), torch.full((S,), n, **i32), torch.arange(n, **i32)

    def step():
        uniform.uniform_()
        pages.reserve(room)
        x = words[tokens.view(-1).long()]
        run(x, q_start, n, (positions[:, None] + behind).view(1, -1))
        moe.moe_linear_w4(Layer.norm(x), head, logits, st=status)
        moe.moe_verify_drafts(logits, tokens.view(-1), uniform, q_start, accepted, token, n_new, workspace=workspace, st=status)
        pages.reserve(n_new)             # the refused drafts' tokens leave the cache
        positions.add_(room + n_new)
        taken.add_((accepted + 1).sum())
        # a stand-in for a drafting model: what the target thought of the place behind
        tokens.copy_(torch.cat([token[:, None], logits.view(S, n, V)[:, :n - 1].argmax(-1)], 1))

    step()
    taken.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    t0 = time.perf_counter()
    for _ in range(a.steps - 1):
        graph.replay()
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0]
    print("with drafts: %.0f tokens/s, %.2f a step and sequence" % (int(taken) / (time.perf_counter() - t0), int(taken) / S / max(a.steps - 1, 1)))


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--batch", type=int, default=32)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=128)
    ap.add_argument("--intermediate", type=int, default=768)
    ap.add_argument("--vocabulary", type=int, default=32000)
    ap.add_argument("--drafts", type=int, default=0)
    ap.add_argument("--budget", type=int, default=0)
    ap.add_argument("--four-bit", action="store_true")
    a = ap.parse_args()
    entry.build()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    gen = torch.Generator(device=dev).manual_seed(0)
    H, n_q, n_kv, D, k = a.hidden, 32, 4, 128, 8
    S, longest = a.batch, a.prompt + a.steps * (2 + a.drafts if a.drafts else 1) + 64
    chunk = max(S * (1 + a.drafts), a.prompt)
    table = moe.rope_table(longest, D, device=dev)
    pages = moe.KvPages(a.layers, S * (-(-longest // 64) + 1), n_kv, D, S, longest, dev, evicts=a.budget > 0)
    caches = [pages.layer(i) for i in range(a.layers)]
    layers = [Layer(H, n_q, n_kv, D, a.experts, a.intermediate, k, chunk, table, gen, dev, a.four_bit, caches[0] if a.budget else None)
              for _ in range(a.layers)]
    i32 = dict(dtype=torch.int32, device=dev)

    def run(x, q_start, max_new, positions=None):
        for i, (layer, cache) in enumerate(zip(layers, caches)):
            layer.forward(x, cache, q_start, max_new, positions, pages.score, i == 0)

    # prompts, one sequence at a time
    t0 = time.perf_counter()
    for s in range(S):
        add = torch.zeros(S, **i32)
        add[s] = a.prompt
        pages.reserve(add)
        q_start = torch.zeros(S + 1, **i32)
        q_start[s + 1:] = a.prompt
        run(torch.randn(a.prompt, H, generator=gen, device=dev), q_start, a.prompt)
    torch.cuda.synchronize()
    print("prompts: %.0f tokens/s" % (S * a.prompt / (time.perf_counter() - t0)))

    # decode steps: one graph, which follows the tables and lengths that it finds
    one, q_start = torch.ones(S, **i32), torch.arange(S + 1, **i32)
    x = torch.randn(S, H, generator=gen, device=dev)
    x0 = x.clone()

    def step():
        pages.reserve(one)
        x.copy_(x0)
        run(x, q_start, 1)

    saved = pages.snapshot()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    pages.restore(saved)                 # the step that warmed up is undone
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    print("decode: %.0f tokens/s (%.1f us a layer)" % (S * a.steps / dt, dt / a.steps / a.layers * 1e6))

    positions = pages.seq_len.clone()    # of the next tokens: an evicted token's place is taken, its position is not
    if a.budget:
        pages.evict(torch.full((S,), a.budget, **i32), 4, min(64, a.budget // 2))
        print("evicted: %d tokens a sequence were %d" % (int(pages.seq_len[0]), int(positions[0])))
    if a.drafts:
        speculate(a, S, H, pages, run, positions, gen, dev)

    # the first sequence forks into four beams, which then go their own ways; the last half ends
    parent = torch.arange(S, **i32)
    parent[1:min(4, S)] = 0
    parent[S - S // 2 if S >= 8 else S:] = -1
    pages.assign(parent)
    add = (parent >= 0).int()
    pages.reserve(add)
    live = int(pages.compact())
    code, detail = pages.device_status()
    assert code == 0, moe.status_string(code, True)
    for layer in layers:
        for part in (layer.attention, layer.experts):
            code, detail = part.device_status()
            assert code == 0, (moe.status_string(code, True), detail)
    tokens = int(pages.seq_len.sum())
    print("after forking and packing: %d tokens in %d pages, %.1f MB a layer (bf16 would take %.1f)"
          % (tokens, live, live * moe.kv4_page_bytes(n_kv, D) / 1e6, live * 64 * n_kv * D * 4 / 1e6))
    assert torch.isfinite(x).all()


if __name__ == "__main__":
    main()
