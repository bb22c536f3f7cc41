"""ctypes binding of the C ABI in include/moe_gb300.h.

Argument marshalling only: each function takes PyTorch CUDA tensors, passes
their device pointers, sizes and the current CUDA stream to the library, and
raises on a non-zero status.  Every step of the layer runs in the library's
CUDA kernels.  If the library has not been built the first call raises; there
is no other implementation to fall back to.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from dataclasses import dataclass
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_gb300.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "moe_gb300.h")

MOE_OK = 0
MOE_DTYPE_F32, MOE_DTYPE_BF16 = 0, 1
MOE_ROUTE_FROM_LOGITS, MOE_ROUTE_RENORM_TOPK = 1, 2
MOE_FFN_FUSE_COMBINE, MOE_FFN_ZERO_Y = 1, 2
MOE_OP_DISPATCH, MOE_OP_FFN, MOE_OP_CALIBRATE, MOE_OP_TOKEN_WEIGHTS, MOE_OP_ROUTE_DISPATCH = 1, 2, 3, 4, 5
ROUTE_DISPATCH_MAX_T, ROUTE_DISPATCH_MAX_SLOTS = 256, 2048
DECODE_LAYER_MAX_T = 64
MOE_SLOT_KEPT, MOE_SLOT_REROUTED, MOE_SLOT_DROPPED = 0, 1, 2
MOE_DEV_OK, MOE_DEV_NONFINITE, MOE_DEV_TIMEOUT, MOE_DEV_BAD_INDEX, MOE_DEV_NO_PAGES = 0, 1, 2, 3, 4
MOE_KV4_PAGE, MOE_KV4_BLOCK = 64, 16

_lock = threading.Lock()
_lib = None
_fast = None   # the module _fastcall, once the library is loaded


class MoeError(RuntimeError):
    pass


class _SereParams(ctypes.Structure):
    _fields_ = [("k_primary", ctypes.c_int), ("rho", ctypes.c_float), ("sim", ctypes.c_void_p),
                ("protect", ctypes.c_void_p), ("union_bitmap", ctypes.c_void_p), ("stats", ctypes.c_void_p)]


class _Kv4CacheParams(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("S", ctypes.c_int32), ("n_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class _RopeParams(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("axis", ctypes.c_void_p),
                ("n_pos", ctypes.c_int32), ("rot", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("pairs", ctypes.c_int32)]


class _Kv4PoolParams(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("layer_stride", ctypes.c_longlong), ("page_bytes", ctypes.c_longlong),
                ("page_table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p), ("ref", ctypes.c_void_p),
                ("n_layers", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("S", ctypes.c_int32)]


class _W4Params(ctypes.Structure):
    _fields_ = [("tiles", ctypes.c_void_p), ("row_scale", ctypes.c_void_p), ("N", ctypes.c_int32), ("K", ctypes.c_int32)]


EXPORTS = ["moe_route", "moe_route_dispatch", "moe_decode_layer", "moe_reroute_sere", "moe_dispatch_capacity", "moe_ffn_grouped", "moe_combine",
           "moe_residual_to_bf16", "moe_token_weights", "moe_similarity_calibrate", "moe_workspace_size", "moe_status_string",
           "moe_qk_norm_rope", "moe_attention_kv4", "moe_attention_kv4_workspace", "moe_kv4_read", "moe_kv4_reserve",
           "moe_kv4_assign", "moe_kv4_compact", "moe_kv4_page_bytes", "moe_kv4_pool_workspace", "moe_kv4_weigh",
           "moe_kv4_weigh_workspace", "moe_kv4_evict", "moe_kv4_evict_workspace", "moe_w4_bytes", "moe_w4_pack", "moe_linear_w4",
           "moe_verify_drafts", "moe_verify_workspace"]


def load(path: str = LIB_PATH):
    """Load the shared library (no GPU needed to load it)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise MoeError("libmoe_gb300.so is not built; run __graft_entry__.build() "
                               "(or python expert_routing_moe_gb300/build.py)")
            L = ctypes.CDLL(path)
            i, u32, f, p, sz = ctypes.c_int, ctypes.c_uint32, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
            L.moe_route.argtypes = [p, i, p, i, i, i, i, i, u32, p, p, p, p, p, p]
            L.moe_route.restype = i
            L.moe_route_dispatch.argtypes = [p, i, p, i, i, i, i, u32, p, p, p, p, p, p, p, p, p, p, sz, p, p]
            L.moe_route_dispatch.restype = i
            L.moe_decode_layer.argtypes = [p, p, p, p, p, i, i, i, i, i, u32, u32, p, p, p, p, p, p, p, p, p, p,
                                           p, sz, p, sz, p, p]
            L.moe_decode_layer.restype = i
            L.moe_reroute_sere.argtypes = [p, p, i, i, i, i, p, p, p]
            L.moe_reroute_sere.restype = i
            L.moe_dispatch_capacity.argtypes = [p, p, i, i, i, i, i, p, f, p, p, p, p, p, p, p, p, p, p, p, p, p,
                                                p, sz, p, p]
            L.moe_dispatch_capacity.restype = i
            L.moe_dispatch_capacity_static.argtypes = [p, p, i, i, i, i, i, p, f, p, p, p, p, p, p, p, p, p, p,
                                                       p, p, p, p, p]
            L.moe_dispatch_capacity_static.restype = i
            L.moe_ffn_grouped.argtypes = [p, i, p, p, p, i, i, i, i, i, p, p, p, p, u32, p, p, sz, p, p]
            L.moe_ffn_grouped.restype = i
            L.moe_combine.argtypes = [p, p, p, i, i, i, p, p]
            L.moe_combine.restype = i
            L.moe_residual_to_bf16.argtypes = [p, p, ctypes.c_longlong, p]
            L.moe_residual_to_bf16.restype = i
            L.moe_token_weights.argtypes = [p, i, i, i, p, f, f, p, p, p, p, sz, p, p]
            L.moe_token_weights.restype = i
            L.moe_similarity_calibrate.argtypes = [p, i, p, p, p, i, i, i, p, p, sz, p, p]
            L.moe_similarity_calibrate.restype = i
            L.moe_workspace_size.argtypes = [i, i, i, i, i, i, i, i, i]
            L.moe_workspace_size.restype = sz
            L.moe_status_string.argtypes = [i, i]
            L.moe_status_string.restype = ctypes.c_char_p
            ll = ctypes.c_longlong
            L.moe_kv4_page_bytes.argtypes = [i, i]
            L.moe_kv4_page_bytes.restype = sz
            L.moe_qk_norm_rope.argtypes = [p, i, ll, i, i, i, i, p, p, f, p, p, ll, p, ll, p, p, p, p]
            L.moe_qk_norm_rope.restype = i
            L.moe_kv4_read.argtypes = [p, p, i, p, p, p, p]
            L.moe_kv4_read.restype = i
            L.moe_attention_kv4.argtypes = [p, ll, i, i, p, p, i, f, i, p, ll, p, p, sz, p, p]
            L.moe_attention_kv4.restype = i
            L.moe_attention_kv4_workspace.argtypes = [i, i, i, i]
            L.moe_attention_kv4_workspace.restype = sz
            L.moe_kv4_reserve.argtypes = [p, p, p, sz, p, p]
            L.moe_kv4_reserve.restype = i
            L.moe_kv4_assign.argtypes = [p, p, p, p]
            L.moe_kv4_assign.restype = i
            L.moe_kv4_compact.argtypes = [p, p, p, sz, p, p]
            L.moe_kv4_compact.restype = i
            L.moe_kv4_pool_workspace.argtypes = [i, i]
            L.moe_kv4_pool_workspace.restype = sz
            L.moe_kv4_weigh.argtypes = [p, ll, i, i, p, p, i, p, f, i, i, p, ll, i, p, sz, p, p]
            L.moe_kv4_weigh.restype = i
            L.moe_kv4_weigh_workspace.argtypes = [i, i, i, i, i, i]
            L.moe_kv4_weigh_workspace.restype = sz
            L.moe_kv4_evict.argtypes = [p, i, p, ll, p, i, i, p, ll, p, sz, p, p]
            L.moe_kv4_evict.restype = i
            L.moe_kv4_evict_workspace.argtypes = [i, i, i]
            L.moe_kv4_evict_workspace.restype = sz
            L.moe_w4_bytes.argtypes = [i, i]
            L.moe_w4_bytes.restype = sz
            L.moe_w4_pack.argtypes = [p, i, ll, p, p, p]
            L.moe_w4_pack.restype = i
            L.moe_linear_w4.argtypes = [p, ll, i, p, p, p, i, ll, i, p, p]
            L.moe_linear_w4.restype = i
            L.moe_verify_drafts.argtypes = [p, i, ll, i, i, p, p, p, i, p, ll, p, p, p, p, p, sz, p, p]
            L.moe_verify_drafts.restype = i
            L.moe_verify_workspace.argtypes = [i, i, i]
            L.moe_verify_workspace.restype = sz
            _load_fastcall(L)
            _lib = L
    return _lib


def _load_fastcall(L):
    """The C module that makes the calls of a decoder's step; built beside
    the library, so it is there when the library is."""
    global _fast
    from . import _fastcall
    addr = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    # (a torch built without CUDA has no raw stream to read: every tensor is refused before it is asked for)
    _fastcall.setup(torch.bfloat16, torch.float32, torch.int32, torch.uint8, getattr(torch._C, "_cuda_getCurrentRawStream", None),
                    *(addr(f) for f in (L.moe_qk_norm_rope, L.moe_kv4_read, L.moe_attention_kv4, L.moe_kv4_reserve,
                                        L.moe_kv4_assign, L.moe_kv4_compact, L.moe_kv4_weigh, L.moe_kv4_evict, L.moe_linear_w4,
                                        L.moe_verify_drafts)))
    _fast = _fastcall


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise MoeError("expected a CUDA tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(rc: int, what: str):
    if rc != MOE_OK:
        msg = load().moe_status_string(rc, 0).decode()
        raise MoeError("%s: %s (%d)" % (what, msg, rc))


def status_string(code: int, device: bool) -> str:
    return load().moe_status_string(int(code), 1 if device else 0).decode()


@dataclass
class SereParams:
    """SERE reroute parameters: K' primaries, threshold rho, similarity [N][N]
    fp32, optional protect [N] uint8, optional outputs union_bitmap
    [ceil(N/32)] int32 and stats [8] int32 (all CUDA tensors)."""
    k_primary: int
    rho: float
    sim: torch.Tensor
    protect: Optional[torch.Tensor] = None
    union_bitmap: Optional[torch.Tensor] = None
    stats: Optional[torch.Tensor] = None

    def _c(self) -> _SereParams:
        return _SereParams(self.k_primary, self.rho, _ptr(self.sim), _ptr(self.protect), _ptr(self.union_bitmap),
                           _ptr(self.stats))


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MOE_DTYPE_BF16
    if t.dtype == torch.float32:
        return MOE_DTYPE_F32
    raise MoeError("unsupported dtype %s" % t.dtype)


def workspace_size(op: int, T: int, H: int, I: int, N: int, k: int, R: int, capped: bool, dtype: int) -> int:
    return int(load().moe_workspace_size(op, T, H, I, N, k, R, 1 if capped else 0, dtype))


def moe_route(x, w_router, logits, ids, gates, k: int, flags: int = 0, sere: Optional[SereParams] = None,
              st=None, stream=None):
    """Router GEMM (unless MOE_ROUTE_FROM_LOGITS), softmax gate and top-R
    ranking, optionally with the SERE reroute fused in.  ids/gates are [T][R]."""
    T, N = logits.shape
    R = ids.shape[1]
    H = 0 if x is None else x.shape[1]
    xd = MOE_DTYPE_F32 if x is None else _dtype_code(x)
    sp = None if sere is None else ctypes.byref(sere._c())
    rc = load().moe_route(_ptr(x), xd, _ptr(w_router), T, H, N, R, k, flags, _ptr(logits), _ptr(ids), _ptr(gates),
                          sp, _ptr(st), _stream(stream))
    _check(rc, "moe_route")


def moe_route_dispatch(x, w_router, logits, ids, gates, counts, offsets, row_token, row_gate, active, workspace,
                       flags: int = 0, sere: Optional[SereParams] = None, st=None, stream=None):
    """Decode batches (T <= 256): moe_route with R = k (optionally with SERE)
    and the uncapped dispatch in one launch.  ids/gates are [T][k]; workspace
    is workspace_size(MOE_OP_ROUTE_DISPATCH, ...) bytes, zero-filled before
    its first use (each call leaves it zeroed)."""
    T, N = logits.shape
    k = ids.shape[1]
    H = x.shape[1]
    sp = None if sere is None else ctypes.byref(sere._c())
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().moe_route_dispatch(_ptr(x), _dtype_code(x), _ptr(w_router), T, H, N, k, flags, _ptr(logits),
                                   _ptr(ids), _ptr(gates), sp, _ptr(counts), _ptr(offsets), _ptr(row_token),
                                   _ptr(row_gate), _ptr(active), _ptr(workspace), ws_bytes, _ptr(st),
                                   _stream(stream))
    _check(rc, "moe_route_dispatch")


def moe_decode_layer(x, w_router, w_gate, w_up, w_down, logits, ids, gates, counts, offsets, row_token, row_gate,
                     active, y, route_ws, ffn_ws, route_flags: int = 0, zero_y: bool = True,
                     sere: Optional[SereParams] = None, st=None, stream=None):
    """One decode layer (T <= 64, bf16): routing + dispatch in one launch and
    the FFN with the combine fused in, the FFN starting on the experts known
    to be active as soon as ranking ends.  y [T][H] fp32 is zeroed first when
    zero_y, else accumulated into."""
    T, H = x.shape
    N, I = w_gate.shape[0], w_gate.shape[1]
    k = ids.shape[1]
    sp = None if sere is None else ctypes.byref(sere._c())
    nb = lambda t: t.numel() * t.element_size()
    rc = load().moe_decode_layer(_ptr(x), _ptr(w_router), _ptr(w_gate), _ptr(w_up), _ptr(w_down), T, H, I, N, k,
                                 route_flags, MOE_FFN_ZERO_Y if zero_y else 0, sp, _ptr(logits), _ptr(ids),
                                 _ptr(gates), _ptr(counts), _ptr(offsets), _ptr(row_token), _ptr(row_gate),
                                 _ptr(active), _ptr(y), _ptr(route_ws), nb(route_ws), _ptr(ffn_ws), nb(ffn_ws),
                                 _ptr(st), _stream(stream))
    _check(rc, "moe_decode_layer")


def moe_reroute_sere(ids, gates, N: int, k: int, sere: SereParams, st=None, stream=None):
    T, ld = ids.shape
    rc = load().moe_reroute_sere(_ptr(ids), _ptr(gates), ld, T, N, k, ctypes.byref(sere._c()), _ptr(st),
                                 _stream(stream))
    _check(rc, "moe_reroute_sere")


def moe_dispatch_capacity(ids, gates, N: int, k: int, R: int, counts, offsets, row_token, row_gate, active,
                          workspace, token_w=None, capacity_factor: float = 0.0, out_ids=None, out_gates=None,
                          slot_row=None, slot_status=None, load_q=None, cap_q=None, st=None, stream=None,
                          modality_bias=None, r_v=None):
    T, ld = ids.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().moe_dispatch_capacity(_ptr(ids), _ptr(gates), ld, T, N, k, R, _ptr(token_w),
                                      float(capacity_factor), _ptr(modality_bias), _ptr(r_v), _ptr(counts),
                                      _ptr(offsets), _ptr(row_token),
                                      _ptr(row_gate), _ptr(active), _ptr(out_ids), _ptr(out_gates),
                                      _ptr(slot_row), _ptr(slot_status), _ptr(load_q), _ptr(cap_q),
                                      _ptr(workspace), ws_bytes, _ptr(st), _stream(stream))
    _check(rc, "moe_dispatch_capacity")


def moe_dispatch_capacity_static(ids, gates, N: int, k: int, R: int, counts, offsets, row_token, row_gate, active,
                                 token_w=None, capacity_factor: float = 0.0, out_ids=None, out_gates=None,
                                 slot_row=None, slot_status=None, load_q=None, cap_q=None, st=None, stream=None,
                                 modality_bias=None, r_v=None):
    """moe_dispatch_capacity without a workspace: the library's own fixed
    device scratch is used (T <= 2048; calls on one device must not overlap)."""
    T, ld = ids.shape
    rc = load().moe_dispatch_capacity_static(_ptr(ids), _ptr(gates), ld, T, N, k, R, _ptr(token_w),
                                             float(capacity_factor), _ptr(modality_bias), _ptr(r_v), _ptr(counts),
                                             _ptr(offsets), _ptr(row_token),
                                             _ptr(row_gate), _ptr(active), _ptr(out_ids), _ptr(out_gates),
                                             _ptr(slot_row), _ptr(slot_status), _ptr(load_q), _ptr(cap_q), _ptr(st),
                                             _stream(stream))
    _check(rc, "moe_dispatch_capacity_static")


def moe_ffn_grouped(x, w_gate, w_up, w_down, k: int, offsets, row_token, row_gate, active, out, workspace,
                    flags: int = MOE_FFN_FUSE_COMBINE | MOE_FFN_ZERO_Y, st=None, stream=None):
    T, H = x.shape
    N, I = w_gate.shape[0], w_gate.shape[1]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().moe_ffn_grouped(_ptr(x), _dtype_code(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), T, H, I, N, k,
                                _ptr(offsets), _ptr(row_token), _ptr(row_gate), _ptr(active), flags, _ptr(out),
                                _ptr(workspace), ws_bytes, _ptr(st), _stream(stream))
    _check(rc, "moe_ffn_grouped")


def moe_combine(rows_out, slot_row, slot_gate, y, stream=None):
    T, k = slot_row.shape
    H = y.shape[1]
    rc = load().moe_combine(_ptr(rows_out), _ptr(slot_row), _ptr(slot_gate), T, H, k, _ptr(y), _stream(stream))
    _check(rc, "moe_combine")


def moe_residual_to_bf16(x, y, stream=None):
    """y = bf16(x), round to nearest even: x fp32 and y bf16 CUDA tensors of
    the same number of elements (a multiple of 8)."""
    if x.numel() != y.numel():
        raise MoeError("moe_residual_to_bf16: %d elements in, %d out" % (x.numel(), y.numel()))
    rc = load().moe_residual_to_bf16(_ptr(x), _ptr(y), x.numel(), _stream(stream))
    _check(rc, "moe_residual_to_bf16")


def moe_token_weights(x, is_visual, entropy, token_w, r_v=None, delta: float = 1.0, eps: float = 1e-6, st=None,
                      stream=None, workspace=None):
    """MACS entropy-weighted token load: entropy [T], token_w [T] and R_v [1]
    (fp32 CUDA tensors) from the token features x [T][H] and is_visual [T]
    uint8.  workspace: workspace_size(MOE_OP_TOKEN_WEIGHTS, T, ...) bytes; when
    omitted a buffer is allocated for this call (not graph-capturable)."""
    T, H = x.shape
    if workspace is None:
        workspace = torch.empty(max(workspace_size(MOE_OP_TOKEN_WEIGHTS, T, 1, 1, 1, 1, 1, False, 0), 256),
                                dtype=torch.uint8, device=x.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().moe_token_weights(_ptr(x), _dtype_code(x), T, H, _ptr(is_visual), float(delta), float(eps),
                                  _ptr(entropy), _ptr(token_w), _ptr(r_v), _ptr(workspace), ws_bytes, _ptr(st),
                                  _stream(stream))
    _check(rc, "moe_token_weights")


def moe_similarity_calibrate(x, w_gate, w_up, w_down, sim, workspace, st=None, stream=None):
    """SERE similarity matrix [N][N] fp32 from the experts' outputs on the
    calibration tokens x [n][H] bf16 (workspace: workspace_size(MOE_OP_CALIBRATE, n, H, I, N, 1, 1, False,
    MOE_DTYPE_BF16) bytes)."""
    n, H = x.shape
    N, I = w_gate.shape[0], w_gate.shape[1]
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().moe_similarity_calibrate(_ptr(x), n, _ptr(w_gate), _ptr(w_up), _ptr(w_down), H, I, N, _ptr(sim),
                                         _ptr(workspace), ws_bytes, _ptr(st), _stream(stream))
    _check(rc, "moe_similarity_calibrate")


# ---------------------------------------------------------------------------
# The attention half of a layer: norms, rotary positions, the 4-bit cache
# ---------------------------------------------------------------------------
def _addr(t: Optional[torch.Tensor], dtype=None, what: str = "") -> Optional[int]:
    """A CUDA tensor's address; checks its dtype and that it is dense."""
    if t is None:
        return None
    if t.is_cuda and (dtype is None or t.dtype is dtype) and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise MoeError("%s: expected a CUDA tensor" % what)
    if dtype is not None and t.dtype is not dtype:
        raise MoeError("%s: expected %s, got %s" % (what, dtype, t.dtype))
    raise MoeError("%s: expected a dense tensor" % what)


def _status(st: Optional[torch.Tensor]) -> Optional[int]:
    """A device status's address: two int32 numbers."""
    if st is not None and st.numel() < 2:
        raise MoeError("status: expected 2 numbers, got %d" % st.numel())
    return _addr(st, torch.int32, "status")


def _rows(t: torch.Tensor, T: int, width: int, dtype, what: str):
    """(address, leading dimension) of T rows of `width` numbers whose trailing
    dimensions are dense; only the first may have a stride of its own."""
    if not t.is_cuda:
        raise MoeError("%s: expected a CUDA tensor" % what)
    if t.dtype is not dtype:
        raise MoeError("%s: expected %s, got %s" % (what, dtype, t.dtype))
    shape, stride = t.shape, t.stride()
    n = 1
    for k in range(len(shape) - 1, 0, -1):
        if stride[k] != n and shape[k] != 1:
            raise MoeError("%s: only the rows may be strided" % what)
        n *= shape[k]
    if len(shape) < 2 or n != width or shape[0] != T:
        raise MoeError("%s: expected %d rows of %d numbers, got %s" % (what, T, width, list(shape)))
    return t.data_ptr(), (stride[0] if T > 1 else max(stride[0], width))


class Kv4Cache:
    """One layer's 4-bit paged cache, as the kernels see it (moe_kv4_cache):
    pages [n_pages][n_kv][64 * (D + D/8)] uint8, page_table [S][max_pages] and
    seq_len [S] int32, head_dim D, optional k_scale and v_scale [n_kv] fp32.
    Holds the tensors; keep it for as long as the cache is used."""

    def __init__(self, pages, page_table, seq_len, head_dim: int, k_scale=None, v_scale=None):
        if pages.dim() != 3 or pages.shape[2] != MOE_KV4_PAGE * (head_dim + head_dim // 8):
            raise MoeError("pages: expected [n_pages][n_kv][%d], got %s"
                           % (MOE_KV4_PAGE * (head_dim + head_dim // 8), list(pages.shape)))
        if page_table.dim() != 2 or seq_len.dim() != 1 or page_table.shape[0] != seq_len.shape[0]:
            raise MoeError("page_table is [S][max_pages] and seq_len [S]")
        self.n_pages, self.n_kv = pages.shape[0], pages.shape[1]
        for t, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is not None and t.numel() != self.n_kv:
                raise MoeError("%s: expected %d numbers" % (what, self.n_kv))
        self.head_dim, self.S, self.max_pages = head_dim, seq_len.shape[0], page_table.shape[1]
        self.tensors = (pages, page_table, seq_len, k_scale, v_scale)
        i32, f32 = torch.int32, torch.float32
        self._c = _Kv4CacheParams(_addr(pages, torch.uint8, "pages"), _addr(page_table, i32, "page_table"),
                                  _addr(seq_len, i32, "seq_len"), _addr(k_scale, f32, "k_scale"),
                                  _addr(v_scale, f32, "v_scale"), self.n_pages, page_table.shape[1], self.S,
                                  self.n_kv, head_dim)
        self._ref = ctypes.addressof(self._c)


class Rope:
    """Rotary positions (moe_rope_params): table [n_pos][rot/2][2] fp32 of
    (cos, sin), positions [axes][T] int32 (None: the place in the sequence),
    axis [rot/2] uint8 (None: axis 0 for every pair), pairs: neighbours are
    rotated together instead of the two halves."""

    def __init__(self, table, positions=None, axis=None, pairs: bool = False):
        if table.dim() != 3 or table.shape[2] != 2:
            raise MoeError("table: expected [n_pos][rot/2][2], got %s" % list(table.shape))
        if positions is not None and positions.dim() != 2:
            raise MoeError("positions: expected [axes][T]")
        if axis is not None and axis.numel() != table.shape[1]:
            raise MoeError("axis: expected %d numbers" % table.shape[1])
        self.tensors = (table, positions, axis)
        self.T = None if positions is None else positions.shape[1]
        self._c = _RopeParams(_addr(table, torch.float32, "table"), _addr(positions, torch.int32, "positions"),
                              _addr(axis, torch.uint8, "axis"), table.shape[0], 2 * table.shape[1],
                              1 if positions is None else positions.shape[0], 1 if pairs else 0)
        self._ref = ctypes.addressof(self._c)


class Kv4Pool:
    """The pages of a cache of several layers (moe_kv4_pool): pages
    [n_layers][n_pages][n_kv][64 * (D + D/8)] uint8, page_table
    [S][max_pages], seq_len [S] and ref [n_pages] int32.  Holds the tensors."""

    def __init__(self, pages, page_table, seq_len, ref, head_dim: int):
        if pages.dim() != 4 or pages.shape[3] != MOE_KV4_PAGE * (head_dim + head_dim // 8):
            raise MoeError("pages: expected [n_layers][n_pages][n_kv][%d], got %s"
                           % (MOE_KV4_PAGE * (head_dim + head_dim // 8), list(pages.shape)))
        if page_table.dim() != 2 or page_table.shape[0] != seq_len.numel() or ref.numel() != pages.shape[1]:
            raise MoeError("page_table is [S][max_pages], seq_len [S] and ref [n_pages]")
        self.tensors = (pages, page_table, seq_len, ref)
        self.head_dim, self.n_layers, self.n_pages, self.S = head_dim, pages.shape[0], pages.shape[1], seq_len.numel()
        self.max_pages = page_table.shape[1]
        i32 = torch.int32
        page_bytes = pages.shape[2] * pages.shape[3]
        self._c = _Kv4PoolParams(_addr(pages, torch.uint8, "pages"), self.n_pages * page_bytes, page_bytes,
                                 _addr(page_table, i32, "page_table"), _addr(seq_len, i32, "seq_len"),
                                 _addr(ref, i32, "ref"), self.n_layers, self.n_pages, page_table.shape[1], self.S)
        self._ref = ctypes.addressof(self._c)

    def layer(self, i: int, k_scale=None, v_scale=None) -> Kv4Cache:
        """Layer i's cache."""
        pages, page_table, seq_len, _ = self.tensors
        return Kv4Cache(pages[i], page_table, seq_len, self.head_dim, k_scale, v_scale)


def kv4_page_bytes(n_kv: int, head_dim: int) -> int:
    return int(load().moe_kv4_page_bytes(n_kv, head_dim))


def attention_kv4_workspace(T: int, n_q: int, n_kv: int, head_dim: int) -> int:
    return int(load().moe_attention_kv4_workspace(T, n_q, n_kv, head_dim))


def kv4_pool_workspace(pool: Kv4Pool) -> int:
    return int(load().moe_kv4_pool_workspace(pool.S, pool.n_pages))


def _raw_stream(stream, t: torch.Tensor) -> int:
    """The given stream, or the current one of the tensor's device (read
    without building a Stream object, which takes longer than a launch)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device()) if stream is None else stream.cuda_stream


def _check_starts(q_start, S: int):
    if q_start.numel() != S + 1:
        raise MoeError("q_start: expected %d numbers, got %d" % (S + 1, q_start.numel()))
    return _addr(q_start, torch.int32, "q_start")


def moe_qk_norm_rope(qkv, n_q: int, n_kv: int, q_out, k_out=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                     rope: Optional[Rope] = None, cache: Optional[Kv4Cache] = None, q_start=None, st=None,
                     stream=None):
    """Norms of q and k for each head (q_weight, k_weight [D] fp32; None = no
    norm), rotary positions and the append of k and v to `cache` (with q_start
    [S+1] int32), in one launch.  qkv [T][(n_q + 2 n_kv) D] bf16 or fp32, q_out
    [T][n_q][D] and k_out [T][n_kv][D] of the same dtype; rows may be strided,
    and q_out may be qkv's own query part."""
    if _fast is None:
        load()
    rc = _fast.qk_norm_rope(qkv, n_q, n_kv, q_out, k_out, q_weight, k_weight, eps, rope, cache, q_start, st) if stream is None else None
    if rc == MOE_OK:
        return
    if rc is not None:
        _check(rc, "moe_qk_norm_rope")
    T, width = qkv.shape[0], 1
    for d in qkv.shape[1:]:
        width *= d
    if n_q + 2 * n_kv < 1 or width % (n_q + 2 * n_kv):
        raise MoeError("qkv: rows of %d numbers are not %d heads" % (width, n_q + 2 * n_kv))
    D = width // (n_q + 2 * n_kv)
    dt = qkv.dtype
    x, ld = _rows(qkv, T, width, dt, "qkv")
    q, ld_q = (None, 0) if n_q == 0 else _rows(q_out, T, n_q * D, dt, "q_out")
    k, ld_k = (None, 0) if k_out is None else _rows(k_out, T, n_kv * D, dt, "k_out")
    if q_weight is not None and q_weight.numel() != D or k_weight is not None and k_weight.numel() != D:
        raise MoeError("q_weight, k_weight: expected %d numbers" % D)
    if rope is not None and rope.T is not None and rope.T != T:
        raise MoeError("positions: expected %d tokens, got %d" % (T, rope.T))
    if cache is not None and q_start is None:
        raise MoeError("a cache needs q_start")
    f32 = torch.float32
    rc = load().moe_qk_norm_rope(x, _dtype_code(qkv), ld, T, n_q, n_kv, D, _addr(q_weight, f32, "q_weight"),
                                 _addr(k_weight, f32, "k_weight"), eps, None if rope is None else rope._ref, q, ld_q, k,
                                 ld_k, None if cache is None else cache._ref,
                                 None if cache is None else _check_starts(q_start, cache.S),
                                 _status(st), _raw_stream(stream, qkv))
    _check(rc, "moe_qk_norm_rope")


def moe_kv4_read(cache: Kv4Cache, q_start, k_out=None, v_out=None, st=None, stream=None):
    """The last q_start[s+1] - q_start[s] tokens of every sequence as values:
    k_out, v_out [T][n_kv][D] bf16."""
    if _fast is None:
        load()
    rc = _fast.kv4_read(cache, q_start, k_out, v_out, st) if stream is None else None
    if rc == MOE_OK:
        return
    if rc is not None:
        _check(rc, "moe_kv4_read")
    T = 0
    for t, what in ((k_out, "k_out"), (v_out, "v_out")):
        if t is not None:
            if t.dim() != 3 or t.shape[1] != cache.n_kv or t.shape[2] != cache.head_dim or (T and t.shape[0] != T):
                raise MoeError("%s: expected [T][%d][%d], got %s" % (what, cache.n_kv, cache.head_dim, list(t.shape)))
            T = t.shape[0]
    bf = torch.bfloat16
    rc = load().moe_kv4_read(cache._ref, _check_starts(q_start, cache.S), T, _addr(k_out, bf, "k_out"),
                             _addr(v_out, bf, "v_out"), _status(st), _raw_stream(stream, q_start))
    _check(rc, "moe_kv4_read")


def moe_attention_kv4(q, cache: Kv4Cache, q_start, out, scale: float, max_new: int, window: int = 0, lse=None,
                      workspace=None, st=None, stream=None):
    """Attention over the cache: rows q_start[s] .. q_start[s+1]-1 of q
    [T][n_q][D] bf16 are the last tokens of sequence s; out like q, lse
    [T][n_q] fp32.  max_new bounds the rows of a sequence.  workspace:
    attention_kv4_workspace(...) bytes, zero-filled before its first use; when
    omitted a buffer is allocated for this call (not graph-capturable)."""
    if _fast is None:
        load()
    rc = _fast.attention(q, cache, q_start, out, scale, max_new, window, lse, workspace, st) if stream is None else None
    if rc == MOE_OK:
        return
    if rc is not None:
        _check(rc, "moe_attention_kv4")
    D = cache.head_dim
    if q.dim() != 3 or q.shape[2] != D:
        raise MoeError("q: expected [T][n_q][%d], got %s" % (D, list(q.shape)))
    T, n_q = q.shape[0], q.shape[1]
    qp, ld_q = _rows(q, T, n_q * D, torch.bfloat16, "q")
    op, ld_o = _rows(out, T, n_q * D, torch.bfloat16, "out")
    if lse is not None and lse.numel() != T * n_q:
        raise MoeError("lse: expected [%d][%d]" % (T, n_q))
    if workspace is None:
        n = attention_kv4_workspace(T, n_q, cache.n_kv, D)
        # cleared, used and given back in the order of the call's own stream
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            workspace = torch.zeros(max(n, 256), dtype=torch.uint8, device=q.device)
    rc = load().moe_attention_kv4(qp, ld_q, T, n_q, cache._ref, _check_starts(q_start, cache.S), max_new, scale, window,
                                  op, ld_o, _addr(lse, torch.float32, "lse"), _addr(workspace, None, "workspace"),
                                  workspace.numel() * workspace.element_size(), _status(st),
                                  _raw_stream(stream, q))
    _check(rc, "moe_attention_kv4")


def _pool_vector(t, pool: Kv4Pool, what: str) -> int:
    if t.numel() != pool.S:
        raise MoeError("%s: expected %d numbers, got %d" % (what, pool.S, t.numel()))
    return _addr(t, torch.int32, what)


def moe_kv4_reserve(pool: Kv4Pool, n_new, workspace, st=None, stream=None):
    """Room for n_new [S] int32 more tokens of every sequence (negative: fewer),
    shared last pages copied first.  workspace: kv4_pool_workspace(pool) bytes."""
    if _fast is None:
        load()
    rc = _fast.reserve(pool, n_new, workspace, st) if stream is None else None
    if rc == MOE_OK:
        return
    if rc is not None:
        _check(rc, "moe_kv4_reserve")
    rc = load().moe_kv4_reserve(pool._ref, _pool_vector(n_new, pool, "n_new"), _addr(workspace, None, "workspace"),
                                workspace.numel() * workspace.element_size(), _status(st),
                                _raw_stream(stream, n_new))
    _check(rc, "moe_kv4_reserve")


def moe_kv4_assign(pool: Kv4Pool, parent, st=None, stream=None):
    """Every sequence becomes what parent[s] was (parent [S] int32, -1 = empty):
    forking, reordering and freeing."""
    if _fast is None:
        load()
    rc = _fast.assign(pool, parent, None, st) if stream is None else None
    if rc == MOE_OK:
        return
    if rc is not None:
        _check(rc, "moe_kv4_assign")
    rc = load().moe_kv4_assign(pool._ref, _pool_vector(parent, pool, "parent"), _status(st),
                               _raw_stream(stream, parent))
    _check(rc, "moe_kv4_assign")


def moe_kv4_compact(pool: Kv4Pool, n_live, workspace, st=None, stream=None):
    """Moves the pool's pages in use to its lowest page numbers; n_live [1]
    int32 out (or None): their count."""
    if _fast is None:
        load()
    rc = _fast.compact(pool, n_live, workspace, st) if stream is None else None
    if rc == MOE_OK:
        return
    if rc is not None:
        _check(rc, "moe_kv4_compact")
    rc = load().moe_kv4_compact(pool._ref, _addr(n_live, torch.int32, "n_live"), _addr(workspace, None, "workspace"),
                                workspace.numel() * workspace.element_size(), _status(st),
                                _raw_stream(stream, workspace))
    _check(rc, "moe_kv4_compact")


# ---------------------------------------------------------------------------
# Eviction from the cache by the attention that its tokens draw
# ---------------------------------------------------------------------------
def kv4_weigh_workspace(cache: Kv4Cache, T: int, n_q: int) -> int:
    return int(load().moe_kv4_weigh_workspace(cache.S, T, n_q, cache.n_kv, cache.head_dim, cache.max_pages))


def kv4_evict_workspace(pool: Kv4Pool) -> int:
    return int(load().moe_kv4_evict_workspace(pool.S, pool.max_pages, pool.n_pages))


def _scores(score, S: int, max_pages: int):
    """(address, leading dimension) of one fp32 score for every place of the tables."""
    if score.dim() != 2 or score.shape[0] != S or score.shape[1] < max_pages * MOE_KV4_PAGE:
        raise MoeError("score: expected [%d][%d or more], got %s" % (S, max_pages * MOE_KV4_PAGE, list(score.shape)))
    return _rows(score, S, score.shape[1], torch.float32, "score")


def _bytes(workspace: Optional[torch.Tensor]) -> int:
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def moe_kv4_weigh(q, cache: Kv4Cache, q_start, lse, score, scale: float, max_new: int, window: int = 0, last: int = 0,
                  fresh: bool = False, workspace=None, st=None, stream=None):
    """Adds the attention weight that every cached token draws from the rows
    (those of moe_attention_kv4, with its lse [T][n_q] fp32) to score [S][max_pages * 64
    or more] fp32: only of each sequence's last `last` rows where that is not 0.  fresh: the
    entries of the rows' own tokens are set instead.  workspace:
    kv4_weigh_workspace(...) bytes; when omitted a buffer is allocated for this call (not
    graph-capturable)."""
    if _fast is None:
        load()
    rc = _fast.weigh(q, cache, q_start, lse, score, scale, max_new, window, last, fresh, workspace, st) if stream is None else None
    if rc == MOE_OK:
        return
    if rc is not None:
        _check(rc, "moe_kv4_weigh")
    D = cache.head_dim
    if q.dim() != 3 or q.shape[2] != D:
        raise MoeError("q: expected [T][n_q][%d], got %s" % (D, list(q.shape)))
    T, n_q = q.shape[0], q.shape[1]
    qp, ld_q = _rows(q, T, n_q * D, torch.bfloat16, "q")
    if lse.numel() != T * n_q:
        raise MoeError("lse: expected [%d][%d]" % (T, n_q))
    sp, ld_s = _scores(score, cache.S, cache.max_pages)
    if workspace is None:
        n = kv4_weigh_workspace(cache, T, n_q)
        if n:
            with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
                workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    rc = load().moe_kv4_weigh(qp, ld_q, T, n_q, cache._ref, _check_starts(q_start, cache.S), max_new, _addr(lse, torch.float32, "lse"),
                              scale, window, last, sp, ld_s, 1 if fresh else 0, _addr(workspace, None, "workspace"), _bytes(workspace),
                              _status(st), _raw_stream(stream, q))
    _check(rc, "moe_kv4_weigh")


def moe_kv4_evict(pool: Kv4Pool, score, budget, sinks: int, recent: int, workspace, kept=None, st=None, stream=None):
    """Every sequence with more than budget[s] tokens (budget [S] int32, negative: all stay)
    keeps its first `sinks`, its last `recent` and the best others by score [S][max_pages *
    64 or more] fp32, moved to its front in every layer with their scores; the pages behind are
    released.  kept [S][any] int32 out (or None): the place that each token had, -1 behind.
    workspace: kv4_evict_workspace(pool) bytes."""
    if _fast is None:
        load()
    rc = _fast.evict(pool, score, budget, sinks, recent, workspace, kept, st) if stream is None else None
    if rc == MOE_OK:
        return
    if rc is not None:
        _check(rc, "moe_kv4_evict")
    sp, ld_s = _scores(score, pool.S, pool.max_pages)
    kp, ld_k = None, 0
    if kept is not None:
        if kept.dim() != 2 or kept.shape[0] != pool.S:
            raise MoeError("kept: expected [%d][any], got %s" % (pool.S, list(kept.shape)))
        kp, ld_k = _addr(kept, torch.int32, "kept"), kept.shape[1]
    rc = load().moe_kv4_evict(pool._ref, pool.head_dim, sp, ld_s, _pool_vector(budget, pool, "budget"), sinks, recent, kp, ld_k,
                              _addr(workspace, None, "workspace"), _bytes(workspace), _status(st), _raw_stream(stream, budget))
    _check(rc, "moe_kv4_evict")


# ---------------------------------------------------------------------------
# Products with weights in 4 bits
# ---------------------------------------------------------------------------
def w4_bytes(N: int, K: int) -> int:
    """Bytes of the tiles of [N][K] weights in 4 bits."""
    return int(load().moe_w4_bytes(N, K))


class Weight4:
    """Weights [N][K] in 4 bits (moe_w4): tiles uint8 in the layout of the header, of
    w4_bytes(N, K) in all, and row_scale [N] fp32 (None: 1).  Holds the tensors."""

    def __init__(self, tiles, N: int, K: int, row_scale=None):
        want = -(-N // 128) * -(-K // 128) * 9216
        if N < 1 or K < 1 or tiles.numel() != want:
            raise MoeError("tiles: expected %d bytes for [%d][%d], got %d" % (want, N, K, tiles.numel()))
        if row_scale is not None and row_scale.numel() != N:
            raise MoeError("row_scale: expected %d numbers, got %d" % (N, row_scale.numel()))
        self.tensors, self.N, self.K = (tiles, row_scale), N, K
        self._c = _W4Params(_addr(tiles, torch.uint8, "tiles"), _addr(row_scale, torch.float32, "row_scale"), N, K)
        self._ref = ctypes.addressof(self._c)

    @classmethod
    def empty(cls, N: int, K: int, device="cuda") -> "Weight4":
        """Room for weights that moe_w4_pack writes."""
        tiles = torch.empty(-(-N // 128), -(-K // 128), 9216, dtype=torch.uint8, device=device)
        return cls(tiles, N, K, torch.empty(N, dtype=torch.float32, device=device))

    @classmethod
    def pack(cls, w, st=None, stream=None) -> "Weight4":
        """w [N][K] bf16 or fp32, rounded to 4 bits."""
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            out = cls.empty(w.shape[0], w.shape[1], w.device)
        moe_w4_pack(w, out, st, stream)
        return out


def moe_w4_pack(w, out: Weight4, st=None, stream=None):
    """Rounds w [N][K] bf16 or fp32 (rows may be strided) to 4 bits, with a scale for
    each row and each 16 columns, into `out`."""
    code = _dtype_code(w)
    wp, ld = _rows(w, out.N, out.K, w.dtype, "w")
    rc = load().moe_w4_pack(wp, code, ld, out._ref, _status(st), _raw_stream(stream, w))
    _check(rc, "moe_w4_pack")


def moe_linear_w4(x, w: Weight4, y, bias=None, accumulate: bool = False, st=None, stream=None):
    """y [T][N] = x [T][K] w^T + bias: x bf16, y bf16 or fp32, bias [N] fp32 or None; rows
    may be strided.  accumulate: added to y (fp32)."""
    if _fast is None:
        load()
    rc = _fast.linear(x, w, y, bias, accumulate, st) if stream is None else None
    if rc == MOE_OK:
        return
    if rc is not None:
        _check(rc, "moe_linear_w4")
    T = x.shape[0]
    xp, ld_x = _rows(x, T, w.K, torch.bfloat16, "x")
    code = _dtype_code(y)
    yp, ld_y = _rows(y, T, w.N, y.dtype, "y")
    if bias is not None and bias.numel() != w.N:
        raise MoeError("bias: expected %d numbers, got %d" % (w.N, bias.numel()))
    if accumulate and code != MOE_DTYPE_F32:
        raise MoeError("y: only fp32 is added to")
    rc = load().moe_linear_w4(xp, ld_x, T, w._ref, _addr(bias, torch.float32, "bias"), yp, code, ld_y, 1 if accumulate else 0,
                              _status(st), _raw_stream(stream, x))
    _check(rc, "moe_linear_w4")


# ---------------------------------------------------------------------------
# Verification of drafted tokens
# ---------------------------------------------------------------------------
def verify_workspace(T: int, S: int, V: int) -> int:
    return int(load().moe_verify_workspace(T, S, V))


def moe_verify_drafts(logits, tokens, uniform, q_start, accepted, next_token, n_new=None, draft_logits=None, temperature=None,
                      workspace=None, st=None, stream=None):
    """How many drafted tokens the target accepts, and the token that follows.  Rows
    q_start[s] .. q_start[s+1]-1 are a sequence's newest token and its drafts: logits
    [T][V] bf16 or fp32 of the target, draft_logits like them (None: drafts without a
    distribution), tokens [T] int32, uniform [T] fp32 from [0, 1), temperature [S] fp32
    (None: 1; 0: greedy).  Out, [S] int32: accepted drafts, the token that follows, and n_new =
    accepted - drafts, which moe_kv4_reserve takes to cut the refused ones.  workspace:
    verify_workspace(...) bytes; when omitted a buffer is allocated for this call."""
    if _fast is None:
        load()
    rc = _fast.verify(logits, tokens, uniform, q_start, accepted, next_token, n_new, draft_logits, temperature, workspace, st) if stream is None else None
    if rc == MOE_OK:
        return
    if rc is not None:
        _check(rc, "moe_verify_drafts")
    if logits.dim() != 2:
        raise MoeError("logits: expected [T][V], got %s" % list(logits.shape))
    T, V = logits.shape
    code = _dtype_code(logits)
    lp, ld = _rows(logits, T, V, logits.dtype, "logits")
    dp, ld_d = (None, 0) if draft_logits is None else _rows(draft_logits, T, V, logits.dtype, "draft_logits")
    S = accepted.numel()
    i32, f32 = torch.int32, torch.float32
    for t, n, what in ((tokens, T, "tokens"), (uniform, T, "uniform"), (next_token, S, "next_token"), (n_new, S, "n_new"),
                       (temperature, S, "temperature")):
        if t is not None and t.numel() != n:
            raise MoeError("%s: expected %d numbers, got %d" % (what, n, t.numel()))
    if workspace is None:
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            workspace = torch.empty(max(verify_workspace(T, S, V), 256), dtype=torch.uint8, device=logits.device)
    rc = load().moe_verify_drafts(lp, code, ld, T, V, _addr(tokens, i32, "tokens"), _addr(uniform, f32, "uniform"),
                                  _check_starts(q_start, S), S, dp, ld_d, _addr(temperature, f32, "temperature"),
                                  _addr(accepted, i32, "accepted"), _addr(next_token, i32, "next_token"), _addr(n_new, i32, "n_new"),
                                  _addr(workspace, None, "workspace"), _bytes(workspace), _status(st), _raw_stream(stream, logits))
    _check(rc, "moe_verify_drafts")
