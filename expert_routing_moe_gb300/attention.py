"""The attention half of a decoder layer for serving: a resident layer (device
weights, preallocated buffers, the C-ABI calls of one pass in order: norms +
rotary positions + append to the 4-bit cache -> attention over it) and the
pages of all layers' caches.  The two projections are plain library products;
everything between them is the library's own kernels.  Buffers are sized once,
so a pass allocates nothing and can be captured in a CUDA graph."""
from __future__ import annotations

from typing import Optional

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
    begun ends first.  Pages cannot be packed during one."""

    def __init__(self, n_layers: int, n_pages: int, n_kv: int, head_dim: int, max_seqs: int, max_len: int, device="cuda"):
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

    def layer(self, i: int, k_scale=None, v_scale=None) -> abi.Kv4Cache:
        return self.pool.layer(i, k_scale, v_scale)

    def reserve(self, n_new: torch.Tensor, stream=None):
        """Room for n_new [max_seqs] int32 more tokens (negative: fewer)."""
        abi.moe_kv4_reserve(self.pool, n_new, self.workspace, self.status, stream)

    def assign(self, parent: torch.Tensor, stream=None):
        """Sequence s becomes what parent[s] was; -1 frees it."""
        abi.moe_kv4_assign(self.pool, parent, self.status, stream)

    def compact(self, stream=None) -> torch.Tensor:
        """Moves the pages in use to the lowest numbers; their count [1] int32."""
        if self.trials:
            raise abi.MoeError("pages are not packed while a snapshot lives: restore or release it first")
        abi.moe_kv4_compact(self.pool, self.n_live, self.workspace, self.status, stream)
        return self.n_live

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
        return saved

    def _end(self, saved: torch.Tensor):
        if not self.trials or self.trials[-1] is not saved:
            raise abi.MoeError("a snapshot is restored or released once, the last one first")
        self.trials.pop()

    def restore(self, saved: torch.Tensor):
        """Ends the trial that began with `saved`: every sequence has its tokens of then."""
        self._end(saved)
        self.book.copy_(saved)

    def release(self, saved: torch.Tensor):
        """Ends the trial that began with `saved` and keeps what it did."""
        self._end(saved)
        self._hold(saved, -1)

    def device_status(self):
        code, detail = (int(v) for v in self.status.tolist())
        return code, detail


class AttentionLayer:
    """w_qkv [(n_q + 2 n_kv) D][H], w_o [H][n_q D] bf16; q_norm, k_norm [D] fp32 or
    None; rope: table and axes of moe_qk_norm_rope (rope_table, rope_axes)."""

    def __init__(self, w_qkv: torch.Tensor, w_o: torch.Tensor, n_q: int, n_kv: int, max_tokens: int,
                 q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 table: Optional[torch.Tensor] = None, axis: Optional[torch.Tensor] = None, pairs: bool = False,
                 scale: Optional[float] = None, window: int = 0):
        self.w_qkv, self.w_o, self.n_q, self.n_kv, self.max_T = w_qkv, w_o, n_q, n_kv, max_tokens
        self.D = w_qkv.shape[0] // (n_q + 2 * n_kv)
        self.q_norm, self.k_norm, self.eps = q_norm, k_norm, eps
        self.table, self.axis, self.pairs = table, axis, pairs
        self.scale = self.D ** -0.5 if scale is None else scale
        self.window = window
        dev, bf = w_qkv.device, torch.bfloat16
        self.qkv = torch.empty(max_tokens, w_qkv.shape[0], dtype=bf, device=dev)
        self.att = torch.empty(max_tokens, n_q, self.D, dtype=bf, device=dev)
        self.y = torch.empty(max_tokens, w_o.shape[0], dtype=bf, device=dev)
        n = abi.attention_kv4_workspace(max_tokens, n_q, n_kv, self.D)
        self.workspace = torch.zeros(max(n, 256), dtype=torch.uint8, device=dev)
        self.status = torch.zeros(2, dtype=torch.int32, device=dev)

    def forward(self, x: torch.Tensor, cache: abi.Kv4Cache, q_start: torch.Tensor, max_new: int,
                positions: Optional[torch.Tensor] = None) -> torch.Tensor:
        """x [T][H] bf16: rows q_start[s] .. q_start[s+1]-1 are the last tokens of
        sequence s of the cache, which has room for them (KvPages.reserve).
        positions [axes][T] int32, or None: their places.  Returns a view of the
        layer's output buffer, [T][H] bf16 (without the residual).  Runs on the
        current stream."""
        T = x.shape[0]
        if T > self.max_T:
            raise abi.MoeError("batch %d exceeds the layer's max_tokens %d" % (T, self.max_T))
        qkv, att, y = self.qkv[:T], self.att[:T], self.y[:T]
        torch.mm(x, self.w_qkv.t(), out=qkv)
        q = qkv[:, :self.n_q * self.D].unflatten(1, (self.n_q, self.D))
        rope = None if self.table is None else abi.Rope(self.table, positions, self.axis, self.pairs)
        abi.moe_qk_norm_rope(qkv, self.n_q, self.n_kv, q, None, self.q_norm, self.k_norm, self.eps, rope, cache, q_start,
                             self.status)
        abi.moe_attention_kv4(q, cache, q_start, att, self.scale, max_new, self.window, None, self.workspace, self.status)
        torch.mm(att.flatten(1), self.w_o.t(), out=y)
        return y

    def device_status(self):
        code, detail = (int(v) for v in self.status.tolist())
        return code, detail
