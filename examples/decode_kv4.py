"""A small mixture-of-experts decoder served from a 4-bit cache: prompts, decode
steps replayed from one CUDA graph, a prompt forked into beams, and the pool
packed.  Random weights; prints tokens/s and the cache's size.

    python examples/decode_kv4.py [--layers 4] [--batch 32] [--prompt 500] [--steps 64]
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

    def __init__(self, H, n_q, n_kv, D, N, I, k, max_tokens, table, gen, dev):
        bf = torch.bfloat16
        w = lambda *s: (torch.randn(*s, generator=gen, device=dev) * s[-1] ** -0.5)  # noqa: E731
        ones = torch.ones(D, device=dev)
        self.attention = moe.AttentionLayer(w((n_q + 2 * n_kv) * D, H).to(bf), w(H, n_q * D).to(bf), n_q, n_kv, max_tokens, ones, ones,
                                            table=table)
        self.experts = moe.MoELayer(w(N, H), w(N, I, H).to(bf), w(N, I, H).to(bf), w(N, H, I).to(bf), k=k, max_tokens=max_tokens)

    @staticmethod
    def norm(x):
        return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def forward(self, x, cache, q_start, max_new):
        x += self.attention.forward(self.norm(x), cache, q_start, max_new)
        self.experts.forward(self.norm(x), accumulate_into=x)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--batch", type=int, default=32)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=128)
    ap.add_argument("--intermediate", type=int, default=768)
    a = ap.parse_args()
    entry.build()
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    gen = torch.Generator(device=dev).manual_seed(0)
    H, n_q, n_kv, D, k = a.hidden, 32, 4, 128, 8
    S, longest = a.batch, a.prompt + a.steps + 64
    chunk = max(S, a.prompt)
    table = moe.rope_table(longest, D, device=dev)
    layers = [Layer(H, n_q, n_kv, D, a.experts, a.intermediate, k, chunk, table, gen, dev) for _ in range(a.layers)]
    pages = moe.KvPages(a.layers, S * (-(-longest // 64) + 1), n_kv, D, S, longest, dev)
    caches = [pages.layer(i) for i in range(a.layers)]
    i32 = dict(dtype=torch.int32, device=dev)

    def run(x, q_start, max_new):
        for layer, cache in zip(layers, caches):
            layer.forward(x, cache, q_start, max_new)

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
