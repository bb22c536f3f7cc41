"""The products with weights in 4 bits, the scores of cached tokens, the verification
of drafts and the eviction together, as a server runs them."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import _kv4
import _verify
import _w4
import expert_routing_moe_gb300 as moe
from _gpu import DEV, dev, host
from test_gpu_kv4_evict import Host

pytestmark = pytest.mark.gpu
H, NQ, NKV, D, V, LAYERS = 256, 8, 2, 64, 1001, 2


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _weights(rng, N, K):
    """(Weight4, the same weights in bf16): codes times scales have six significant bits, so both are exact."""
    codes = rng.integers(0, 16, (N, K)).astype(np.uint8)
    scales = rng.integers(0x14, 0x1c, (N, -(-K // 16))).astype(np.uint8)     # 2^-5 to 2^-4
    w = _w4.values(codes, scales, np.ones(N))
    return moe.Weight4(dev(_w4.pack_codes(codes, scales)), N, K), torch.tensor(w, device=DEV).bfloat16()


def _layer(rng, max_tokens, four, weighs=None, window=0):
    ones = torch.ones(D, device=DEV)
    w_qkv, w_o = _weights(rng, (NQ + 2 * NKV) * D, H), _weights(rng, H, NQ * D)
    at = 0 if four else 1
    return moe.AttentionLayer(w_qkv[at], w_o[at], NQ, NKV, max_tokens, ones, ones, table=moe.rope_table(4000, D, device=DEV), window=window, weighs=weighs)


@pytest.mark.parametrize("n", [1, 5, 40, 130])
def test_projections_in_4_bits(n):
    """The same weights in both forms: the layer's outputs are as close as those of bf16 products whose sums
    are ordered differently."""
    x = torch.randn(n, H, device=DEV).bfloat16()
    outs = []
    for four in (True, False):
        layer = _layer(np.random.default_rng(3), n, four)
        pages = moe.KvPages(1, 5, NKV, D, 1, 256, DEV)
        cache = pages.layer(0)
        pages.reserve(_i32([n]))
        y = layer.forward(x, cache, _i32([0, n]), n)
        assert pages.device_status() == (0, 0) and layer.device_status() == (0, 0)
        outs.append(y.float())
    # a bf16 step of q, k or v, and for few numbers a code of the cache
    assert (outs[0] - outs[1]).norm() / outs[1].norm() < 0.02


@pytest.mark.parametrize("rows,last,window", [(1, 0, 0), (5, 2, 0), (150, 0, 0), (150, 40, 70)])
def test_a_layer_weighs_what_it_attends_to(rows, last, window):
    """forward's score is that of moe_kv4_weigh after the attention, bit for bit; a second layer adds to it."""
    before = 70
    pages = moe.KvPages(LAYERS, 8, NKV, D, 1, 256, DEV, evicts=True)
    caches = [pages.layer(i) for i in range(LAYERS)]
    layers = [_layer(np.random.default_rng(i), 150, True, caches[0], window) for i in range(LAYERS)]
    x = torch.randn(150, H, device=DEV).bfloat16()
    q_start = _i32([0, before])
    pages.reserve(_i32([before]))
    for i in range(LAYERS):
        layers[i].forward(x[:before], caches[i], q_start, before, score=pages.score, fresh=i == 0)
    assert float(pages.score[0, :before].min()) > 0 and not pages.score[0, before:].any()
    # every row's weights sum to 1 for each head (fp32 sums of 0.5 million numbers below 1)
    assert abs(float(pages.score.double().sum()) - LAYERS * NQ * before) < 1e-3 * LAYERS * NQ * before
    pages.score[0, before:] = 7                        # of tokens that were there before
    mine = pages.score.clone()
    q_start = _i32([0, rows])
    pages.reserve(_i32([rows]))
    for i in range(LAYERS):
        layers[i].forward(x[:rows], caches[i], q_start, rows, score=pages.score, last=last, fresh=i == 0)
    for i in range(LAYERS):
        q = layers[i].qkv[:rows, :NQ * D].unflatten(1, (NQ, D))
        out, lse = torch.empty(rows, NQ, D, dtype=torch.bfloat16, device=DEV), torch.empty(rows, NQ, device=DEV)
        moe.moe_attention_kv4(q, caches[i], q_start, out, D ** -0.5, rows, window, lse)
        moe.moe_kv4_weigh(q, caches[i], q_start, lse, mine, D ** -0.5, rows, window, last, i == 0)
    assert torch.equal(mine, pages.score)
    assert pages.device_status() == (0, 0) and all(layer.device_status() == (0, 0) for layer in layers)


class Held:
    """What _kv4.attention reads, from the GPU's cache."""

    def __init__(self, cache, lengths):
        at = np.r_[0, np.cumsum(lengths)]
        k, v = (torch.empty(int(at[-1]), NKV, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        moe.moe_kv4_read(cache, _i32(at.tolist()), k, v)
        k, v = host(k.double()), host(v.double())
        self.n_kv, self.lengths = NKV, list(lengths)
        self.k, self.v = ([x[a:b] for a, b in zip(at, at[1:])] for x in (k, v))


class Server:
    def __init__(self, prompts, drafts, budget):
        rng = np.random.default_rng(11)
        self.S, self.drafts = len(prompts), drafts
        self.rows = self.S * (drafts + 1)
        self.pages = moe.KvPages(LAYERS, 24, NKV, D, self.S, 512, DEV, evicts=True)
        self.caches = [self.pages.layer(i) for i in range(LAYERS)]
        self.layers = [_layer(rng, max(max(prompts), self.rows), True, self.caches[0]) for _ in range(LAYERS)]
        self.head = _weights(rng, V, H)[0]
        self.table = torch.randn(V, H, device=DEV)
        self.pos = torch.zeros(self.S, dtype=torch.int32, device=DEV)
        self.budget = _i32(budget)
        for s, n in enumerate(prompts):
            add = np.zeros(self.S, np.int32)
            add[s] = n
            self.pages.reserve(dev(add))
            q_start = dev(np.r_[0, np.cumsum(add)].astype(np.int32))
            x = torch.randn(n, H, device=DEV)
            for i, layer in enumerate(self.layers):
                x += layer.forward(x.bfloat16(), self.caches[i], q_start, n, score=self.pages.score, last=32, fresh=i == 0)
            self.pos += dev(add)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.q_start = torch.arange(0, self.rows + 1, drafts + 1, **i32)
        self.tokens, self.uniform = torch.zeros(self.rows, **i32), torch.zeros(self.rows, device=DEV)
        self.temperature = torch.tensor([0.0, 0.8, 1.2], device=DEV)[torch.arange(self.S, device=DEV) % 3]
        self.accepted, self.next, self.n_new = (torch.zeros(self.S, **i32) for _ in range(3))
        self.room = torch.full((self.S,), drafts + 1, **i32)
        self.logits = torch.zeros(self.rows, V, device=DEV)
        self.kept = torch.zeros(self.S, 512, **i32)
        self.x = torch.zeros(self.rows, H, device=DEV)
        self.ws = torch.zeros(moe.verify_workspace(self.rows, self.S, V), dtype=torch.uint8, device=DEV)
        self.status = torch.zeros(2, **i32)

    def ahead(self):
        """The drafts' rows through the layers and the head."""
        self.pages.reserve(self.room)
        place = (self.pos[:, None] + torch.arange(self.drafts + 1, dtype=torch.int32, device=DEV)).reshape(1, -1)
        self.x.copy_(self.table[self.tokens.long()])
        for i, layer in enumerate(self.layers):
            self.x.add_(layer.forward(self.x.bfloat16(), self.caches[i], self.q_start, self.drafts + 1, place, self.pages.score, fresh=i == 0))
        moe.moe_linear_w4(self.x.bfloat16(), self.head, self.logits, st=self.status)

    def accept(self):
        """Drafts that the model takes stay, the others' tokens leave the cache."""
        moe.moe_verify_drafts(self.logits, self.tokens, self.uniform, self.q_start, self.accepted, self.next, self.n_new,
                              temperature=self.temperature, workspace=self.ws, st=self.status)
        self.pages.reserve(self.n_new)
        self.pos += self.room + self.n_new

    def cut(self):
        self.pages.evict(self.budget, 4, 20, self.kept)

    def step(self):
        self.ahead()
        self.accept()
        self.cut()

    def draw(self, rng):
        """Some drafts that a greedy sequence takes, among others."""
        self.tokens.copy_(dev(rng.integers(0, V, self.rows).astype(np.int32)))
        self.uniform.copy_(dev(rng.random(self.rows).astype(np.float32)))

    def state(self):
        p = self.pages
        return [t.clone() for t in (p.book, p.pages, p.score, self.pos)]

    def back(self, state):
        p = self.pages
        for t, v in zip((p.book, p.pages, p.score, self.pos), state):
            t.copy_(v)

    def clean(self):
        return (self.pages.device_status() == (0, 0) and not self.status.any() and all(layer.device_status() == (0, 0) for layer in self.layers))


def test_steps_with_drafts_and_eviction():
    """Three sequences, two steps; each stage against its definition on what the stage before it left."""
    server = Server([190, 70, 300], 3, [128, -1, 200])
    rng = np.random.default_rng(5)
    lengths = np.array([190, 70, 300])
    for turn in range(2):
        server.draw(rng)
        state = server.state()
        server.ahead()
        # the target's own choice is drafted, so that greedy sequences take some
        if turn == 1:
            best = server.logits.argmax(1).int()
            server.back(state)
            server.tokens.view(3, 4)[:, 1:] = best.view(3, 4)[:, :3]
            server.ahead()
        # attention over what the cache holds, of the last layer
        q = server.layers[-1].qkv[:server.rows, :NQ * D].unflatten(1, (NQ, D))
        held = Held(server.caches[-1], lengths + 4)
        out, _, tol, _ = _kv4.attention(held, host(q.double()), [0, 4, 8, 12], D ** -0.5)
        assert (np.abs(host(server.layers[-1].att[:server.rows].double()) - out) <= tol).all()
        # the head: exact products, sums of 256 in fp32, 2^-24 a step relative to their magnitudes
        x, w = host(server.x.bfloat16().double()), _w4_of(server.head)
        assert (np.abs(host(server.logits.double()) - x @ w.T) <= 256 * 2.0 ** -24 * (np.abs(x) @ np.abs(w).T)).all()
        server.accept()
        want = _verify.verify(host(server.logits), host(server.tokens), host(server.uniform), host(server.q_start), None, host(server.temperature))
        for mine, theirs in zip((server.accepted, server.next, server.n_new), want):
            assert np.array_equal(host(mine), theirs)
        lengths = lengths + 4 + want[2]
        assert server.pages.seq_len.tolist() == lengths.tolist()
        # the tokens that stay, and what they hold
        k = [Held(c, lengths) for c in server.caches]
        rules = Host.__new__(Host)
        rules.layers, rules.n_kv, rules.D, rules.columns = LAYERS, NKV, D, server.pages.page_table.shape[1]
        rules.len, rules.table, rules.ref = host(server.pages.seq_len).copy(), host(server.pages.page_table).copy(), host(server.pages.ref).copy()
        rules.data, rules.score = host(server.pages.pages).copy(), host(server.pages.score).copy()
        server.cut()
        assert rules.evict(host(server.budget), 4, 20, 512) == (0, 0)
        assert np.array_equal(host(server.kept), rules.kept)
        for mine, theirs in ((server.pages.seq_len, rules.len), (server.pages.page_table, rules.table), (server.pages.ref, rules.ref), (server.pages.score, rules.score),
                             (server.pages.pages, rules.data)):
            assert np.array_equal(host(mine), theirs)
        lengths = np.where((host(server.budget) >= 0) & (lengths > host(server.budget)), host(server.budget), lengths)
        for i, c in enumerate(server.caches):
            after = Held(c, lengths)
            for s in range(3):
                kept = rules.kept[s, :lengths[s]]
                assert np.array_equal(after.k[s], k[i].k[s][kept]) and np.array_equal(after.v[s], k[i].v[s][kept])
    assert lengths[0] == 128 and lengths[2] == 200 and server.clean()


def _w4_of(w):
    """A Weight4's weights in 64 bits, through products with unit vectors."""
    eye = torch.eye(w.K, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(w.K, w.N, device=DEV)
    moe.moe_linear_w4(eye, w, y)
    return host(y.double()).T


def test_a_captured_step_is_the_eager_one():
    server = Server([190, 70, 300], 3, [128, -1, 200])
    server.draw(np.random.default_rng(6))
    start = server.state()
    outs = (server.logits, server.accepted, server.next, server.n_new, server.kept)
    server.step()
    eager = server.state() + [t.clone() for t in outs]
    side = torch.cuda.Stream()
    server.back(start)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        server.step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(eager, server.state() + list(outs)))
    server.back(start)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        server.step()
    for _ in range(2):
        server.back(start)
        for t in outs:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(eager, server.state() + list(outs)))
    # other tokens and another budget through the same graph, against an eager step
    server.draw(np.random.default_rng(7))
    server.budget.copy_(_i32([100, 60, -1]))
    server.back(start)
    graph.replay()
    replayed = server.state() + [t.clone() for t in outs]
    server.back(start)
    server.step()
    assert all(torch.equal(a, b) for a, b in zip(replayed, server.state() + list(outs)))
    assert server.pages.seq_len.tolist()[:2] == [100, 60] and server.clean()


def test_a_trial_with_eviction_is_undone():
    """restore() brings tokens and scores back, and the pages that the trial read are as they were."""
    server = Server([190, 70, 300], 3, [128, -1, 200])
    server.draw(np.random.default_rng(8))
    lengths = [190, 70, 300]
    before = [Held(c, lengths) for c in server.caches]
    score, pos = server.pages.score.clone(), server.pos.clone()
    saved = server.pages.snapshot()
    server.step()
    assert server.pages.seq_len.tolist()[0] == 128 and not torch.equal(score, server.pages.score)
    server.pages.restore(saved)
    server.pos.copy_(pos)
    assert torch.equal(score, server.pages.score) and server.pages.seq_len.tolist() == lengths
    for a, c in zip(before, server.caches):
        b = Held(c, lengths)
        assert all(np.array_equal(x, y) for x, y in zip(a.k + a.v, b.k + b.v))
    saved = server.pages.snapshot()
    server.step()
    server.pages.release(saved)
    assert server.pages.seq_len.tolist()[0] == 128 and not server.pages.trials and not server.pages.trial_scores
    assert server.clean()


def test_scores_follow_forks():
    pages = moe.KvPages(1, 12, NKV, D, 3, 128, DEV, evicts=True)
    pages.reserve(_i32([100, 30, 0]))
    pages.score.copy_(torch.arange(3 * 128, device=DEV).view(3, 128))
    want = pages.score.clone()
    pages.assign(_i32([1, 0, 0]))
    assert torch.equal(pages.score, want[[1, 0, 0]]) and pages.seq_len.tolist() == [30, 100, 100]
    pages.assign(_i32([3, 0, 0]))                      # refused
    assert torch.equal(pages.score, want[[1, 0, 0]]) and pages.device_status()[0] != 0


def test_what_was_not_asked_for_is_refused():
    pages = moe.KvPages(1, 4, NKV, D, 1, 128, DEV)
    with pytest.raises(moe.MoeError):
        pages.evict(_i32([10]))
    layer = _layer(np.random.default_rng(0), 4, True)
    pages.reserve(_i32([4]))
    with pytest.raises(moe.MoeError):
        layer.forward(torch.zeros(4, H, dtype=torch.bfloat16, device=DEV), pages.layer(0), _i32([0, 4]), 4, score=torch.zeros(1, 128, device=DEV))


def test_the_example_drafts_and_evicts():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "decode_kv4.py"), "--layers", "2", "--batch", "8", "--prompt", "170", "--steps", "4", "--hidden", "256",
                        "--experts", "16", "--intermediate", "128", "--vocabulary", "1001", "--drafts", "3", "--budget", "100", "--four-bit"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "evicted: 100 tokens a sequence were 174" in r.stdout and "with drafts" in r.stdout and "after forking and packing" in r.stdout
