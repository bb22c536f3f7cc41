"""The attention half of a decoder layer for serving: a resident layer (device
weights, preallocated buffers, the C-ABI calls of one pass in order: norms +
rotary positions + append to the 4-bit cache -> attention over it) and the
pages of all layers' caches.  The two projections are plain library products
where their weights are bf16, and moe_linear_w4 where they are a Weight4;
everything between them is the library's own kernels.  Buffers are sized once,
so a pass allocates nothing and can be captured in a CUDA graph."""
from __future__ import annotations

import contextlib
from typing import Optional, Union

import torch

from . import _abi as abi


def rope_table(n_pos: int, rot: int, base: float = 1e6, device="cuda", inv_freq: Optional[torch.Tensor] = None) -> torch.Tensor:
    """(cos, sin) of every position and pair, [n_pos][rot/2][2] fp32, from
    64-bit angles (a far position times a frequency near 1 keeps only a few
    digits of its angle in 32).  inv_freq [rot/2] replaces base^(-2i/rot)."""
    if inv_freq is None:
        inv_freq = base ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float64) / rot)
    angle = torch.arange(n_pos, device=device, dtype=torch.float64)[:, None] * inv_freq.to(device=device, dtype=torch.float64)
    return torch.stack([angle.cos(), angle.sin()], -1).float().contiguous()


def rope_axes(sections, interleaved: bool = False, device="cuda") -> torch.Tensor:
    """The axis of each pair, [sum(sections)] uint8: sections[a] pairs turn with
    axis a (time, height, width, ...), in one run each, or taken in turn while
    an axis has pairs left (interleaved)."""
    if not interleaved:
        order = [a for a, n in enumerate(sections) for _ in range(n)]
    else:
        left, order = list(sections), []
        while any(left):
            for a in range(len(left)):
                if left[a]:
                    left[a] -= 1
                    order.append(a)
    return torch.tensor(order, dtype=torch.uint8, device=device)


class KvPages:
    """The 4-bit caches of n_layers layers in pages of 64 tokens, for up to
    max_seqs sequences of up to max_len tokens.  page_table, seq_len and ref
    are views of one int32 tensor, `book`.

    A step that is only tried (drafts, a beam that may be dropped) begins with
    snapshot() and ends with restore(), which undoes all of its reserves and
    assigns, or with release(), which keeps them.  In between the snapshot
    holds a reference on every page that a sequence has: none of them is handed
    out, and a sequence that grows into a partly filled one gets a copy, so the
    pool needs a free page for each of those.  Trials may be nested; the last
    begun ends first.  Pages cannot be packed during one.

    evicts: also has the workspace of evict(), and `score` [max_seqs][places of
    max_len] fp32, zero, which AttentionLayer.forward adds to.  Scores follow
    their tokens in evict() and assign(), and restore() brings them back too.
    A token that comes in a pass without a score has what was last in its place."""

    def __init__(self, n_layers: int, n_pages: int, n_kv: int, head_dim: int, max_seqs: int, max_len: int, device="cuda", evicts: bool = False):
        cols = -(-max_len // abi.MOE_KV4_PAGE)
        a, b = max_seqs * cols, max_seqs * cols + max_seqs
        self.book = torch.zeros(b + n_pages, dtype=torch.int32, device=device)
        self.book[:a] = -1
        self.page_table, self.seq_len, self.ref = self.book[:a].view(max_seqs, cols), self.book[a:b], self.book[b:]
        bytes_ = abi.MOE_KV4_PAGE * (head_dim + head_dim // 8)
        self.pages = torch.zeros(n_layers, n_pages, n_kv, bytes_, dtype=torch.uint8, device=device)
        self.pool = abi.Kv4Pool(self.pages, self.page_table, self.seq_len, self.ref, head_dim)
        self.workspace = torch.zeros(max(abi.kv4_pool_workspace(self.pool), 256), dtype=torch.uint8, device=device)
        self.status = torch.zeros(2, dtype=torch.int32, device=device)
        self.n_live = torch.zeros(1, dtype=torch.int32, device=device)
        self.trials = []                     # the snapshots that live, first to last
        self.trial_scores = []
        self.score = self.evict_workspace = None
        if evicts:
            self.score = torch.zeros(max_seqs, cols * abi.MOE_KV4_PAGE, dtype=torch.float32, device=device)
            self.evict_workspace = torch.zeros(max(abi.kv4_evict_workspace(self.pool), 256), dtype=torch.uint8, device=device)

    def layer(self, i: int, k_scale=None, v_scale=None) -> abi.Kv4Cache:
        return self.pool.layer(i, k_scale, v_scale)

    def reserve(self, n_new: torch.Tensor, stream=None):
        """Room for n_new [max_seqs] int32 more tokens (negative: fewer)."""
        abi.moe_kv4_reserve(self.pool, n_new, self.workspace, self.status, stream)

    def assign(self, parent: torch.Tensor, stream=None):
        """Sequence s becomes what parent[s] was, its score among it; -1 frees it.  A parent
        outside [-1, max_seqs) is reported and its sequence kept (moe_kv4_assign)."""
        abi.moe_kv4_assign(self.pool, parent, self.status, stream)
        if self.score is not None:
            with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
                n = self.score.shape[0]
                own = torch.arange(n, device=parent.device)
                # (a parent that is refused leaves its own sequence as it was, and the others move)
                self.score.copy_(self.score[torch.where((parent >= 0) & (parent < n), parent.long(), own)])

    def compact(self, stream=None) -> torch.Tensor:
        """Moves the pages in use to the lowest numbers; their count [1] int32."""
        if self.trials:
            raise abi.MoeError("pages are not packed while a snapshot lives: restore or release it first")
        abi.moe_kv4_compact(self.pool, self.n_live, self.workspace, self.status, stream)
        return self.n_live

    def evict(self, budget: torch.Tensor, sinks: int = 4, recent: int = 64, kept: Optional[torch.Tensor] = None, stream=None):
        """Every sequence with more than budget[s] tokens ([max_seqs] int32, negative: all
        stay) keeps that many: its first `sinks`, its last `recent` and the
        others by self.score, which moves with them (moe_kv4_evict).  Keys stay
        turned to the positions that their tokens had, so what comes behind them
        has positions of its own (forward's `positions`), not its places."""
        if self.evict_workspace is None:
            raise abi.MoeError("pages made without evicts=True have no scores")
        abi.moe_kv4_evict(self.pool, self.score, budget, sinks, recent, self.evict_workspace, kept, self.status, stream)

    def _hold(self, saved: torch.Tensor, count: int):
        """`count` more references on every page for each entry of the saved table that names it."""
        n = self.ref.numel()
        pages = saved[:self.page_table.numel()].long()
        pages = torch.where((pages >= 0) & (pages < n), pages, n)     # one number more for entries without a page
        held = torch.zeros(n + 1, dtype=torch.int32, device=saved.device)
        held.index_add_(0, pages, torch.full_like(saved[:pages.numel()], count))
        self.ref += held[:n]

    def snapshot(self) -> torch.Tensor:
        """Begins a step that is only tried, on the current stream."""
        saved = self.book.clone()
        self._hold(saved, 1)
        self.trials.append(saved)
        self.trial_scores.append(None if self.score is None else self.score.clone())
        return saved

    def _end(self, saved: torch.Tensor):
        if not self.trials or self.trials[-1] is not saved:
            raise abi.MoeError("a snapshot is restored or released once, the last one first")
        self.trials.pop()
        return self.trial_scores.pop()

    def restore(self, saved: torch.Tensor):
        """Ends the trial that began with `saved`: every sequence has its tokens of then."""
        score = self._end(saved)
        self.book.copy_(saved)
        if score is not None:
            self.score.copy_(score)

    def release(self, saved: torch.Tensor):
        """Ends the trial that began with `saved` and keeps what it did."""
        self._end(saved)
        self._hold(saved, -1)

    def device_status(self):
        code, detail = (int(v) for v in self.status.tolist())
        return code, detail


def _rows_of(w: Union[torch.Tensor, abi.Weight4]) -> int:
    return w.N if isinstance(w, abi.Weight4) else w.shape[0]


class AttentionLayer:
    """w_qkv [(n_q + 2 n_kv) D][H], w_o [H][n_q D] bf16 or Weight4; q_norm, k_norm [D] fp32 or
    None; rope: table and axes of moe_qk_norm_rope (rope_table, rope_axes).

    weighs: a cache of the tables that forward's `score` belongs to, or None."""

    def __init__(self, w_qkv: Union[torch.Tensor, abi.Weight4], w_o: Union[torch.Tensor, abi.Weight4], n_q: int, n_kv: int, max_tokens: int,
                 q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 table: Optional[torch.Tensor] = None, axis: Optional[torch.Tensor] = None, pairs: bool = False,
                 scale: Optional[float] = None, window: int = 0, weighs: Optional[abi.Kv4Cache] = None):
        self.w_qkv, self.w_o, self.n_q, self.n_kv, self.max_T = w_qkv, w_o, n_q, n_kv, max_tokens
        self.D = _rows_of(w_qkv) // (n_q + 2 * n_kv)
        self.q_norm, self.k_norm, self.eps = q_norm, k_norm, eps
        self.table, self.axis, self.pairs = table, axis, pairs
        self.scale = self.D ** -0.5 if scale is None else scale
        self.window = window
        dev, bf = w_qkv.tensors[0].device if isinstance(w_qkv, abi.Weight4) else w_qkv.device, torch.bfloat16
        self.qkv = torch.empty(max_tokens, _rows_of(w_qkv), dtype=bf, device=dev)
        self.att = torch.empty(max_tokens, n_q, self.D, dtype=bf, device=dev)
        self.y = torch.empty(max_tokens, _rows_of(w_o), dtype=bf, device=dev)
        n = abi.attention_kv4_workspace(max_tokens, n_q, n_kv, self.D)
        self.workspace = torch.zeros(max(n, 256), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(2, dtype=torch.int32, device=dev)
        self.lse = self.weigh_workspace = None
        if weighs is not None:
            n = abi.kv4_weigh_workspace(weighs, max_tokens, n_q)
            self.lse = torch.empty(max_tokens, n_q, dtype=torch.float32, device=dev)
            self.weigh_workspace = torch.zeros(max(n, 256), dtype=torch.uint8, device=dev)

    def _product(self, x: torch.Tensor, w: Union[torch.Tensor, abi.Weight4], y: torch.Tensor):
        if isinstance(w, abi.Weight4):
            abi.moe_linear_w4(x, w, y, st=self.status)
        else:
            torch.mm(x, w.t(), out=y)

    def forward(self, x: torch.Tensor, cache: abi.Kv4Cache, q_start: torch.Tensor, max_new: int,
                positions: Optional[torch.Tensor] = None, score: Optional[torch.Tensor] = None, last: int = 0,
                fresh: bool = True) -> torch.Tensor:
        """x [T][H] bf16: rows q_start[s] .. q_start[s+1]-1 are the last tokens of
        sequence s of the cache, which has room for them (KvPages.reserve).
        positions [axes][T] int32, or None: their places.  Returns a view of the
        layer's output buffer, [T][H] bf16 (without the residual).  Runs on the
        current stream.

        score [S][places] fp32 (KvPages.score), or None: the weight that every token
        draws from the rows (their last `last` where that is not 0) is added to
        it; with fresh the rows' own tokens begin at 0 (moe_kv4_weigh).  Of
        layers that share a score one has fresh, the first."""
        T = x.shape[0]
        if T > self.max_T:
            raise abi.MoeError("batch %d exceeds the layer's max_tokens %d" % (T, self.max_T))
        if score is not None and self.lse is None:
            raise abi.MoeError("a layer made without weighs has no buffers for a score")
        qkv, att, y = self.qkv[:T], self.att[:T], self.y[:T]
        lse = None if score is None else self.lse[:T]
        self._product(x, self.w_qkv, qkv)
        q = qkv[:, :self.n_q * self.D].unflatten(1, (self.n_q, self.D))
        rope = None if self.table is None else abi.Rope(self.table, positions, self.axis, self.pairs)
        abi.moe_qk_norm_rope(qkv, self.n_q, self.n_kv, q, None, self.q_norm, self.k_norm, self.eps, rope, cache, q_start,
                             self.status)
        abi.moe_attention_kv4(q, cache, q_start, att, self.scale, max_new, self.window, lse, self.workspace, self.status)
        if score is not None:
            abi.moe_kv4_weigh(q, cache, q_start, lse, score, self.scale, max_new, self.window, last, fresh, self.weigh_workspace, self.status)
        self._product(att.flatten(1), self.w_o, y)
        return y

    def device_status(self):
        code, detail = (int(v) for v in self.status.tolist())
        return code, detail
