"""Python binding of the hs C ABI (include/hs.h): argument marshalling only.

Every step of the resolution runs in the CUDA kernels of ``libhs.so``; this module only converts torch tensors,
streams and integers into the plain pointers and sizes of the C entry points, and raises :class:`HsError` on a
negative return code. PyTorch is used for device memory and streams. There is no CPU fallback: if the library
has not been built, loading it raises.

The method is the per-layer selection resolution of "HiSparse: Scaling Sparse-Attention Decoding with
Hierarchical KV Cache Management" (Abstract); the policy and the memory layout are documented in hs.h.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading

from . import build as _build_mod

__all__ = [
    "HsError", "hs_pool_desc", "hs_meta_layout", "load", "hs_meta_bytes", "hs_get_meta_layout", "hs_pool_create",
    "hs_pool_reset", "hs_step_begin", "hs_resolve", "hs_prefetch", "hs_get_error", "hs_get_counters",
    "hs_pool_destroy", "hs_host_alloc", "hs_host_free", "hs_error_string", "HS_DEVERR_RANGE", "HS_DEVERR_DUP",
    "HS_DEVERR_STATE", "HostBuffer", "PoolBuffers", "hs_probe_link", "hs_gather", "hs_gather_history",
    "hs_resolve_shared", "hs_resolve_tiered", "hs_mla_decode", "hs_mla_decode_history", "HS_DEVERR_TIMEOUT",
    "MLA_HEADS", "MLA_D_QK", "MLA_D_V", "hs_probe_launch", "hs_debug_attention", "hs_step_begin_fused", "hs_probe_link_static", "HS_ERR_TOO_LARGE",
    "hs_resolve_ids", "hs_prefetch_ids", "hs_append", "hs_append_desc", "append_desc", "hs_paged_rows", "paged_rows",
    "hs_gather_values", "hs_gather_values_history", "hs_mla_decode_int4", "hs_mla_decode_int4_history",
    "hs_mla_prefix", "hs_mla_prefix_workspace", "hs_mla_prefix_workspace_bound", "HS_TYPE_BF16", "HS_TYPE_F16", "HS_TYPE_F32",
]

HS_OK = 0
HS_ERR_INVALID_ARG = -1
HS_ERR_CUDA = -2
HS_ERR_NOT_MAPPED = -3
HS_ERR_NO_MEMORY = -4
HS_ERR_UNSUPPORTED = -5
HS_ERR_TOO_LARGE = -6
HS_DEVERR_RANGE = 1
HS_DEVERR_DUP = 2
HS_DEVERR_STATE = 4
HS_DEVERR_TIMEOUT = 8
HS_TYPE_BF16, HS_TYPE_F16, HS_TYPE_F32 = 0, 1, 2
MLA_HEADS, MLA_D_QK, MLA_D_V = 128, 576, 512  # shape of the sparse MLA decode consumer

# the row formats of hs_append: bf16, fp8, 4 bits
KV_ROW_BYTES = (MLA_D_QK * 2, MLA_D_V + 4 * 4 + (MLA_D_QK - MLA_D_V) * 2, MLA_D_V // 2 + MLA_D_V // 16 + (MLA_D_QK - MLA_D_V) * 2)

LIB_PATH = _build_mod.LIB_PATH
_lib = None
_pool_row_bytes = {}  # of each open pool, by its handle
_lock = threading.Lock()


class HsError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {hs_error_string(code)} ({code})")
        self.code = code


class hs_pool_desc(ctypes.Structure):
    _fields_ = [
        ("layers", ctypes.c_int32), ("max_batch", ctypes.c_int32), ("ctx", ctypes.c_int32),
        ("slots", ctypes.c_int32), ("topk_max", ctypes.c_int32), ("row_bytes", ctypes.c_int32),
        ("host_pool", ctypes.c_void_p), ("host_layer_stride", ctypes.c_int64), ("host_req_stride", ctypes.c_int64),
        ("hot_buf", ctypes.c_void_p), ("meta", ctypes.c_void_p), ("noio_src", ctypes.c_void_p),
    ]


class hs_meta_layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("step", "error", "counters", "tok2slot", "slot_tok", "slot_stamp", "total")]


class hs_paged_rows(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_void_p), ("count", ctypes.c_int64), ("pages", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("page_rows", ctypes.c_int32), ("lists", ctypes.c_int32)]


class hs_append_desc(ctypes.Structure):
    _fields_ = [
        ("type", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("kv", ctypes.c_void_p),
        ("kv_stride", ctypes.c_int64), ("norm_weight", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
        ("req_ids", ctypes.c_void_p), ("positions", ctypes.c_void_p), ("q_rope", ctypes.c_void_p),
        ("q_rope_token_stride", ctypes.c_int64), ("q_rope_head_stride", ctypes.c_int64), ("q", ctypes.c_void_p),
        ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64), ("q_heads", ctypes.c_int32),
        ("norm_eps", ctypes.c_float),
    ]


def load():
    """Open libhs.so (built by ``build.build()``); raises if it is missing -- there is no other path."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run hierarchical_sparse_attention_hs_gb300.build.build()")
        lib = ctypes.CDLL(LIB_PATH)
        P, vp, i32, sz = ctypes.POINTER, ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
        sig = {
            "hs_meta_bytes": (sz, [P(hs_pool_desc)]),
            "hs_get_meta_layout": (ctypes.c_int, [P(hs_pool_desc), P(hs_meta_layout)]),
            "hs_pool_create": (ctypes.c_int, [P(hs_pool_desc), vp, P(vp)]),
            "hs_pool_reset": (ctypes.c_int, [vp, vp]),
            "hs_step_begin": (ctypes.c_int, [vp, vp]),
            "hs_step_begin_fused": (ctypes.c_int, [vp]),
            "hs_resolve": (ctypes.c_int, [vp, i32, i32, vp, i32, vp, vp]),
            "hs_prefetch": (ctypes.c_int, [vp, i32, i32, vp, i32, vp]),
            "hs_resolve_ids": (ctypes.c_int, [vp, i32, i32, vp, vp, i32, vp, vp]),
            "hs_prefetch_ids": (ctypes.c_int, [vp, i32, i32, vp, vp, i32, vp]),
            "hs_gather": (ctypes.c_int, [vp, i32, i32, vp, i32, vp, vp]),
            "hs_resolve_shared": (ctypes.c_int, [vp, i32, i32, i32, vp, i32, vp, vp]),
            "hs_resolve_tiered": (ctypes.c_int, [vp, i32, i32, vp, i32, vp, ctypes.c_int64, vp, vp]),
            "hs_gather_history": (ctypes.c_int, [vp, i32, i32, vp, i32, vp, vp]),
            "hs_mla_decode": (ctypes.c_int, [vp, i32, i32, vp, vp, i32, vp, ctypes.c_int64, ctypes.c_float, vp, vp,
                                             vp]),
            "hs_mla_decode_history": (ctypes.c_int, [vp, i32, i32, vp, vp, i32, ctypes.c_float, vp, vp, vp]),
            "hs_get_error": (ctypes.c_int, [vp, P(i32), i32]),
            "hs_get_counters": (ctypes.c_int, [vp, i32, P(ctypes.c_uint64)]),
            "hs_pool_destroy": (ctypes.c_int, [vp]),
            "hs_host_alloc": (ctypes.c_int, [sz, P(vp)]),
            "hs_host_free": (ctypes.c_int, [vp]),
            "hs_error_string": (ctypes.c_char_p, [ctypes.c_int]),
            "hs_probe_link": (ctypes.c_int, [vp, vp, sz, i32, vp, P(ctypes.c_double), P(ctypes.c_double)]),
            "hs_probe_launch": (ctypes.c_int, [vp, i32, i32, i32, i32, vp]),
            "hs_probe_link_static": (ctypes.c_int, [vp, sz, i32, vp, P(ctypes.c_double), P(ctypes.c_double)]),
            "hs_debug_attention": (ctypes.c_int, [ctypes.c_uint32, i32, P(i32)]),
            "hs_append": (ctypes.c_int, [vp, i32, i32, P(hs_append_desc), P(hs_paged_rows), i32, vp]),
            "hs_gather_values": (ctypes.c_int, [vp, i32, i32, vp, i32, vp, ctypes.c_int64, vp, i32, vp]),
            "hs_gather_values_history": (ctypes.c_int, [vp, i32, i32, vp, i32, vp, i32, vp]),
            "hs_mla_decode_int4": (ctypes.c_int, [vp, i32, i32, vp, vp, i32, vp, ctypes.c_int64, ctypes.c_float, vp, i32, vp,
                                                  vp]),
            "hs_mla_decode_int4_history": (ctypes.c_int, [vp, i32, i32, vp, vp, i32, ctypes.c_float, vp, i32, vp, vp]),
            "hs_mla_prefix": (ctypes.c_int, [vp, i32, vp, P(hs_paged_rows), i32, vp, ctypes.c_float, vp, vp, vp, i32, vp,
                                             vp, sz, vp]),
            "hs_mla_prefix_workspace": (sz, [vp, i32, i32]),
            "hs_mla_prefix_workspace_bound": (ctypes.c_int, [vp, i32, i32, P(sz)]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _addr(x) -> int | None:
    return x if x is None or isinstance(x, int) else x.data_ptr()


_current = None  # torch's current stream of a device and its current device, once torch is loaded


def _load_current():
    global _current
    import torch

    torch.cuda.current_device()  # starts CUDA; from then on the bare call under it is enough
    # the handle alone: making a Stream object of it takes longer than a small kernel
    _current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    return _current


def _stream(s) -> int | None:
    if s is None:
        handle, device = _current or _load_current()
        return handle(device())
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(rc: int, what: str) -> None:
    if rc != HS_OK:
        raise HsError(rc, what)


def hs_probe_link(host_ptr: int, dev, nbytes: int, iters: int = 5, stream=None) -> tuple:
    """(zero-copy SM read GB/s, cudaMemcpyAsync H2D GB/s) over `nbytes` of mapped host memory."""
    zc, cp = ctypes.c_double(), ctypes.c_double()
    _check(load().hs_probe_link(host_ptr, _addr(dev), nbytes, iters, _stream(stream), ctypes.byref(zc),
                                ctypes.byref(cp)), "hs_probe_link")
    return zc.value, cp.value


def hs_probe_link_static(host_ptr: int, nbytes: int, iters: int = 5, stream=None) -> tuple:
    """(zero-copy SM read GB/s, cudaMemcpyAsync H2D GB/s) with the library's own fixed device scratch (at most
    16 MiB); for callers that have no device allocator."""
    zc, cp = ctypes.c_double(), ctypes.c_double()
    _check(load().hs_probe_link_static(host_ptr, nbytes, iters, _stream(stream), ctypes.byref(zc), ctypes.byref(cp)),
           "hs_probe_link_static")
    return zc.value, cp.value


def hs_probe_launch(pool: int, layer: int, nlayers: int, batch: int, k: int, stream=None) -> None:
    _check(load().hs_probe_launch(pool, layer, nlayers, batch, k, _stream(stream)), "hs_probe_launch")


def hs_debug_attention(wait_limit: int = 0, stall: bool = False) -> int:
    """Test hook: set the attention kernel's wait limit (0 = default) and stall switch; returns the largest batch
    whose keys are split over two CTA pairs on the current device."""
    n = ctypes.c_int32()
    _check(load().hs_debug_attention(wait_limit, int(bool(stall)), ctypes.byref(n)), "hs_debug_attention")
    return int(n.value)


def hs_error_string(code: int) -> str:
    return load().hs_error_string(code).decode()


def hs_meta_bytes(desc: hs_pool_desc) -> int:
    return int(load().hs_meta_bytes(ctypes.byref(desc)))


def hs_get_meta_layout(desc: hs_pool_desc) -> dict:
    lay = hs_meta_layout()
    _check(load().hs_get_meta_layout(ctypes.byref(desc), ctypes.byref(lay)), "hs_get_meta_layout")
    return {n: int(getattr(lay, n)) for n, _ in hs_meta_layout._fields_}


def hs_pool_create(desc: hs_pool_desc, stream=None) -> int:
    h = ctypes.c_void_p()
    _check(load().hs_pool_create(ctypes.byref(desc), _stream(stream), ctypes.byref(h)), "hs_pool_create")
    _pool_row_bytes[h.value] = desc.row_bytes
    return h.value


def hs_pool_reset(pool: int, stream=None) -> None:
    _check(load().hs_pool_reset(pool, _stream(stream)), "hs_pool_reset")


def hs_step_begin(pool: int, stream=None) -> None:
    _check(load().hs_step_begin(pool, _stream(stream)), "hs_step_begin")


def hs_step_begin_fused(pool: int) -> None:
    _check(load().hs_step_begin_fused(pool), "hs_step_begin_fused")


def hs_resolve(pool: int, layer: int, batch: int, topk_idx, k: int, out_slots, stream=None) -> None:
    _check(load().hs_resolve(pool, layer, batch, _addr(topk_idx), k, _addr(out_slots), _stream(stream)),
           "hs_resolve")


def hs_prefetch(pool: int, layer: int, batch: int, topk_idx, k: int, stream=None) -> None:
    _check(load().hs_prefetch(pool, layer, batch, _addr(topk_idx), k, _stream(stream)), "hs_prefetch")


def hs_resolve_ids(pool: int, layer: int, batch: int, req_ids, topk_idx, k: int, out_slots, stream=None) -> None:
    _check(load().hs_resolve_ids(pool, layer, batch, _addr(req_ids), _addr(topk_idx), k, _addr(out_slots),
                                 _stream(stream)), "hs_resolve_ids")


def hs_prefetch_ids(pool: int, layer: int, batch: int, req_ids, topk_idx, k: int, stream=None) -> None:
    _check(load().hs_prefetch_ids(pool, layer, batch, _addr(req_ids), _addr(topk_idx), k, _stream(stream)),
           "hs_prefetch_ids")


def hs_resolve_shared(pool: int, layer0: int, nlayers: int, batch: int, topk_idx, k: int, out_slots,
                      stream=None) -> None:
    _check(load().hs_resolve_shared(pool, layer0, nlayers, batch, _addr(topk_idx), k, _addr(out_slots),
                                    _stream(stream)), "hs_resolve_shared")


def hs_resolve_tiered(pool: int, layer: int, batch: int, topk_idx, k: int, resident_row, resident_stride: int,
                      out_slots, stream=None) -> None:
    _check(load().hs_resolve_tiered(pool, layer, batch, _addr(topk_idx), k, _addr(resident_row), resident_stride,
                                    _addr(out_slots), _stream(stream)), "hs_resolve_tiered")


def hs_gather(pool: int, layer: int, batch: int, out_slots, k: int, dst, stream=None) -> None:
    _check(load().hs_gather(pool, layer, batch, _addr(out_slots), k, _addr(dst), _stream(stream)), "hs_gather")


def hs_mla_decode(pool: int, layer: int, batch: int, q, out_slots, k: int, resident_rows, resident_count: int,
                  sm_scale: float, out, lse, stream=None) -> None:
    _check(load().hs_mla_decode(pool, layer, batch, _addr(q), _addr(out_slots), k, _addr(resident_rows),
                                resident_count, sm_scale, _addr(out), _addr(lse), _stream(stream)), "hs_mla_decode")


def hs_mla_decode_history(pool: int, layer: int, batch: int, q, topk_idx, k: int, sm_scale: float, out, lse,
                          stream=None) -> None:
    _check(load().hs_mla_decode_history(pool, layer, batch, _addr(q), _addr(topk_idx), k, sm_scale, _addr(out),
                                        _addr(lse), _stream(stream)), "hs_mla_decode_history")


def hs_gather_history(pool: int, layer: int, batch: int, topk_idx, k: int, dst, stream=None) -> None:
    _check(load().hs_gather_history(pool, layer, batch, _addr(topk_idx), k, _addr(dst), _stream(stream)),
           "hs_gather_history")


def paged_rows(rows, pages, page_rows: int) -> hs_paged_rows:
    """The struct of an ordinary paged pool: `rows` a tensor [count][...] of contiguous rows, each 1152 or 656 or 416
    bytes (the pool's row_bytes), `pages` int32 [lists][entries] (or [entries], one list, request 0's). It keeps both tensors alive;
    build it once and pass it to every call."""
    import torch

    if not rows.is_contiguous() or not pages.is_contiguous():
        raise ValueError("paged_rows takes contiguous tensors")
    row_bytes = rows.element_size() * math.prod(rows.shape[1:])
    if row_bytes not in KV_ROW_BYTES:
        raise ValueError(f"rows is [count][...] with rows of 1152 or 656 or 416 bytes: {tuple(rows.shape)} of {rows.dtype} has "
                         f"{row_bytes}")
    if pages.dtype != torch.int32:
        raise ValueError(f"pages is int32, not {pages.dtype}")
    if pages.dim() not in (1, 2) or pages.numel() == 0:
        raise ValueError(f"pages is [lists][entries] or [entries], not {tuple(pages.shape)}")
    lists = 1 if pages.dim() == 1 else pages.shape[0]
    p = hs_paged_rows(rows.data_ptr(), rows.shape[0], pages.data_ptr(), pages.shape[-1], page_rows, lists)
    p._keep, p._row_bytes = (rows, pages), row_bytes
    return p


def _check_row_bytes(pool: int, paged) -> None:
    have, want = getattr(paged, "_row_bytes", None), _pool_row_bytes.get(pool)
    if have and want and have != want:
        raise ValueError(f"the paged rows have {have} bytes, the pool's {want}")


def append_desc(kv, inv_freq, positions, req_ids=None, norm_weight=None, norm_eps: float = 0.0,
                interleaved: bool = True, q_rope=None, q=None) -> hs_append_desc:
    """The struct of one append, from torch tensors: kv [n][576], inv_freq fp32 [32], positions and req_ids int32 [n],
    norm_weight fp32 [512], q_rope [n][heads][64] of kv's type, q bf16 [n][heads][576]; the last dimension of each is
    contiguous. It keeps the tensors alive; build it once and refill them between calls."""
    import torch

    types = {torch.bfloat16: HS_TYPE_BF16, torch.float16: HS_TYPE_F16, torch.float32: HS_TYPE_F32}
    if kv.dtype not in types or (q_rope is not None and q_rope.dtype != kv.dtype):
        raise ValueError("kv and q_rope are bf16, fp16 or fp32, both the same")
    for t, want in ((inv_freq, torch.float32), (positions, torch.int32), (req_ids, torch.int32),
                    (norm_weight, torch.float32), (q, torch.bfloat16)):
        if t is not None and t.dtype != want:
            raise ValueError(f"append_desc takes {want} there, not {t.dtype}")
    if any(t is not None and t.stride(-1) != 1 for t in (kv, inv_freq, positions, req_ids, norm_weight, q_rope, q)):
        raise ValueError("the last dimension of every tensor is contiguous")
    if (q_rope is None) != (q is None):
        raise ValueError("q_rope and q go together")
    n, width, rope = positions.shape[0], MLA_D_QK, MLA_D_QK - MLA_D_V
    heads = 0 if q is None else q.shape[1]
    for name, t, shape in (("kv", kv, (n, width)), ("inv_freq", inv_freq, (rope // 2,)), ("req_ids", req_ids, (n,)),
                           ("norm_weight", norm_weight, (MLA_D_V,)), ("q_rope", q_rope, (n, heads, rope)),
                           ("q", q, (n, heads, width))):
        if t is not None and tuple(t.shape) != shape:
            raise ValueError(f"{name} is {tuple(t.shape)}, not {shape}")
    d = hs_append_desc(types[kv.dtype], int(interleaved), kv.data_ptr(), kv.stride(0), _addr(norm_weight),
                       inv_freq.data_ptr(), _addr(req_ids), positions.data_ptr(), _addr(q_rope), 0, 0, _addr(q), 0, 0, 0,
                       norm_eps)
    if q is not None:
        d.q_rope_token_stride, d.q_rope_head_stride, d.q_heads = q_rope.stride(0), q_rope.stride(1), q_rope.shape[1]
        d.q_token_stride, d.q_head_stride = q.stride(0), q.stride(1)
    d._keep, d._tokens = (kv, inv_freq, positions, req_ids, norm_weight, q_rope, q), n
    return d


def hs_append(pool: int, layer: int, ntok: int, desc: hs_append_desc, paged: hs_paged_rows | None = None,
              to_history: bool = True, stream=None) -> None:
    if ntok > getattr(desc, "_tokens", ntok):
        raise ValueError(f"{ntok} tokens, but the descriptor's tensors hold {desc._tokens}")
    if paged is not None:
        _check_row_bytes(pool, paged)
    _check(load().hs_append(pool, layer, ntok, desc, paged, int(to_history), _stream(stream)), "hs_append")


_dtypes = None  # torch's bf16, fp32, int32 and fp16, once torch is loaded


def _load_dtypes():
    global _dtypes
    import torch

    _dtypes = torch.bfloat16, torch.float32, torch.int32, torch.float16
    return _dtypes


def _fits(t, dtype, nbytes: int) -> bool:
    """Whether a tensor has this type and as many bytes, in order. (Of an address nothing is known; None is the library's.)"""
    return t is None or isinstance(t, int) or (t.dtype is dtype and t.nbytes >= nbytes and t.is_contiguous())


def hs_mla_prefix(pool: int, batch: int, q, prefix: hs_paged_rows, max_length: int, prefix_length, sm_scale: float,
                  own_out, own_lse, out, out_type: int, lse, workspace, stream=None) -> None:
    _check_row_bytes(pool, prefix)
    bf16, f32, i32, _ = _dtypes or _load_dtypes()
    rows = batch * MLA_HEADS
    out_dtype = f32 if out_type == HS_TYPE_F32 else bf16
    if not (_fits(q, bf16, rows * MLA_D_QK * 2) and _fits(out, out_dtype, rows * MLA_D_V * out_dtype.itemsize) and
            _fits(lse, f32, rows * 4) and
            (own_out is None or _fits(own_out, f32, rows * MLA_D_V * 4) and _fits(own_lse, f32, rows * 4)) and
            (prefix_length is None or _fits(prefix_length, i32, 4))):
        raise ValueError(f"hs_mla_prefix of {batch} takes contiguous tensors: q bf16 [{batch}][128][576], out {out_dtype} "
                         f"[{batch}][128][512], lse fp32 [{batch}][128], own_out and own_lse fp32 as out and lse, "
                         f"prefix_length int32")
    _check(load().hs_mla_prefix(pool, batch, _addr(q), prefix, max_length, _addr(prefix_length), sm_scale,
                                _addr(own_out), _addr(own_lse), _addr(out), out_type, _addr(lse), _addr(workspace),
                                0 if workspace is None else workspace.nbytes, _stream(stream)), "hs_mla_prefix")


def hs_mla_prefix_workspace(pool: int, batch: int, max_length: int) -> int:
    return int(load().hs_mla_prefix_workspace(pool, batch, max_length))


def hs_mla_prefix_workspace_bound(pool: int, batch: int, max_length: int) -> int:
    n = ctypes.c_size_t()
    _check(load().hs_mla_prefix_workspace_bound(pool, batch, max_length, ctypes.byref(n)), "hs_mla_prefix_workspace_bound")
    return int(n.value)


_value_types = None  # of each HS_TYPE_*: torch's type, and the bytes of 576 values


def _load_value_types():
    global _value_types
    bf16, f32, _, f16 = _dtypes or _load_dtypes()
    _value_types = {HS_TYPE_BF16: (bf16, 2 * MLA_D_QK), HS_TYPE_F16: (f16, 2 * MLA_D_QK), HS_TYPE_F32: (f32, 4 * MLA_D_QK)}
    return _value_types


def _tensor(t, dtype, nbytes: int):
    """The address of a tensor that _fits, or False."""
    if t is None or isinstance(t, int):
        return t
    return t.dtype is dtype and t.nbytes >= nbytes and t.is_contiguous() and t.data_ptr()


def _refuse_host(what: str, entries, *tensors) -> None:
    """For a call with a tensor in host memory, which only a list may be, and only page-locked."""
    host = [t is not None and not isinstance(t, int) and not t.is_cuda for t in (entries, *tensors)]
    if any(host[1:]):
        raise ValueError(f"{what} takes tensors in device memory")
    if host[0] and not entries.is_pinned():
        raise ValueError(f"{what} takes a list in device memory or in page-locked host memory")


def _entries(what: str, batch: int, entries, k: int):
    at = _tensor(entries, (_dtypes or _load_dtypes())[2], batch * k * 4)
    if at is False:
        raise ValueError(f"{what} takes a contiguous int32 list [{batch}][{k}]")
    return at


def _has_rows(t, row_bytes: int) -> bool:
    """Whether the last dimensions of a tensor, as few as hold a row, hold whole rows of these bytes. (One dimension is plain
    memory, and of a pool that was not made here the rows are not known.)"""
    if t.dim() < 2 or t.numel() == 0 or not row_bytes:
        return True
    n = t.element_size()
    for d in reversed(t.shape[1:]):
        n *= d
        if n >= row_bytes:
            break
    return n >= row_bytes and n % row_bytes == 0


def _resident(what: str, pool: int, rows, count: int):
    if rows is None or isinstance(rows, int):
        return rows
    row_bytes, nbytes = _pool_row_bytes.get(pool, 0), rows.nbytes
    want = count * row_bytes
    if nbytes < want or not rows.is_contiguous() or nbytes != want and not _has_rows(rows, row_bytes):
        raise ValueError(f"{what} takes contiguous resident rows, {count} of {row_bytes} bytes, not {tuple(rows.shape)} of "
                         f"{rows.dtype}")
    return rows.data_ptr()


def _values(what: str, batch: int, k: int, dst, dst_type: int):
    # (of a type that there is not the library says so)
    t = (_value_types or _load_value_types()).get(dst_type)
    if t is None:
        return _addr(dst)
    at = _tensor(dst, t[0], batch * k * t[1])
    if at is False:
        raise ValueError(f"{what} writes a contiguous {t[0]} [{batch}][{k}][{MLA_D_QK}]")
    return at


# In the calls below an address that is not what was passed is a tensor's.


def hs_gather_values(pool: int, layer: int, batch: int, out_slots, k: int, resident_rows, resident_count: int, dst,
                     dst_type: int, stream=None) -> None:
    entries = _entries("hs_gather_values", batch, out_slots, k)
    rows = _resident("hs_gather_values", pool, resident_rows, resident_count)
    values = _values("hs_gather_values", batch, k, dst, dst_type)
    lib = _lib or load()
    if (entries is not out_slots and not out_slots.is_cuda or rows is not resident_rows and not resident_rows.is_cuda or
            values is not dst and not dst.is_cuda):
        _refuse_host("hs_gather_values", out_slots, resident_rows, dst)
    _check(lib.hs_gather_values(pool, layer, batch, entries, k, rows, resident_count, values, dst_type, _stream(stream)),
           "hs_gather_values")


def hs_gather_values_history(pool: int, layer: int, batch: int, topk_idx, k: int, dst, dst_type: int, stream=None) -> None:
    entries = _entries("hs_gather_values_history", batch, topk_idx, k)
    values = _values("hs_gather_values_history", batch, k, dst, dst_type)
    lib = _lib or load()
    if entries is not topk_idx and not topk_idx.is_cuda or values is not dst and not dst.is_cuda:
        _refuse_host("hs_gather_values_history", topk_idx, dst)
    _check(lib.hs_gather_values_history(pool, layer, batch, entries, k, values, dst_type, _stream(stream)),
           "hs_gather_values_history")


def _heads(what: str, batch: int, q, out, out_type: int, lse):
    bf16, f32, _, _ = _dtypes or _load_dtypes()
    rows = batch * MLA_HEADS
    dtype, size = (f32, 4) if out_type == HS_TYPE_F32 else (bf16, 2)
    at = _tensor(q, bf16, rows * (2 * MLA_D_QK)), _tensor(out, dtype, rows * (size * MLA_D_V)), _tensor(lse, f32, rows * 4)
    if at[0] is False or at[1] is False or at[2] is False:
        raise ValueError(f"{what} of {batch} takes contiguous tensors: q bf16 [{batch}][128][576], out {dtype} "
                         f"[{batch}][128][512], lse fp32 [{batch}][128]")
    return at


def hs_mla_decode_int4(pool: int, layer: int, batch: int, q, out_slots, k: int, resident_rows, resident_count: int,
                       sm_scale: float, out, out_type: int, lse, stream=None) -> None:
    entries = _entries("hs_mla_decode_int4", batch, out_slots, k)
    rows = _resident("hs_mla_decode_int4", pool, resident_rows, resident_count)
    at = _heads("hs_mla_decode_int4", batch, q, out, out_type, lse)
    lib = _lib or load()
    if (entries is not out_slots and not out_slots.is_cuda or rows is not resident_rows and not resident_rows.is_cuda or
            at[0] is not q and not q.is_cuda or at[1] is not out and not out.is_cuda or at[2] is not lse and not lse.is_cuda):
        _refuse_host("hs_mla_decode_int4", out_slots, resident_rows, q, out, lse)
    _check(lib.hs_mla_decode_int4(pool, layer, batch, at[0], entries, k, rows, resident_count, sm_scale, at[1], out_type, at[2],
                                  _stream(stream)), "hs_mla_decode_int4")


def hs_mla_decode_int4_history(pool: int, layer: int, batch: int, q, topk_idx, k: int, sm_scale: float, out, out_type: int,
                               lse, stream=None) -> None:
    entries = _entries("hs_mla_decode_int4_history", batch, topk_idx, k)
    at = _heads("hs_mla_decode_int4_history", batch, q, out, out_type, lse)
    lib = _lib or load()
    if (entries is not topk_idx and not topk_idx.is_cuda or at[0] is not q and not q.is_cuda or
            at[1] is not out and not out.is_cuda or at[2] is not lse and not lse.is_cuda):
        _refuse_host("hs_mla_decode_int4_history", topk_idx, q, out, lse)
    _check(lib.hs_mla_decode_int4_history(pool, layer, batch, at[0], entries, k, sm_scale, at[1], out_type, at[2],
                                          _stream(stream)), "hs_mla_decode_int4_history")


def hs_get_error(pool: int, clear: bool = False) -> int:
    v = ctypes.c_int32()
    _check(load().hs_get_error(pool, ctypes.byref(v), int(clear)), "hs_get_error")
    return int(v.value)


def hs_get_counters(pool: int, layer: int) -> list:
    arr = (ctypes.c_uint64 * 4)()
    _check(load().hs_get_counters(pool, layer, arr), "hs_get_counters")
    return [int(x) for x in arr]


def hs_pool_destroy(pool: int) -> None:
    _check(load().hs_pool_destroy(pool), "hs_pool_destroy")
    _pool_row_bytes.pop(pool, None)


def hs_host_alloc(nbytes: int) -> int:
    p = ctypes.c_void_p()
    _check(load().hs_host_alloc(nbytes, ctypes.byref(p)), "hs_host_alloc")
    return p.value


def hs_host_free(ptr: int) -> None:
    _check(load().hs_host_free(ptr), "hs_host_free")


class HostBuffer:
    """Page-locked, device-mapped host memory from hs_host_alloc, freed on close()."""

    def __init__(self, nbytes: int):
        self.nbytes = nbytes
        self.ptr = hs_host_alloc(nbytes)

    def numpy(self):
        import numpy as np

        return np.ctypeslib.as_array((ctypes.c_uint8 * self.nbytes).from_address(self.ptr))

    def close(self):
        if self.ptr:
            hs_host_free(self.ptr)
            self.ptr = 0

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class PoolBuffers:
    """Caller-side memory for one pool, allocated with torch (device) and hs_host_alloc (host), plus the handle.

    ``host_layers`` host-pool layers are allocated; with fewer than ``layers`` the pool's layer stride is 0 only
    when host_layers == 1 (all layers read one pool). ``layer_shift_rows`` S > 0 (with host_layers == 1) makes the
    layer stride S rows instead: the pool grows by (layers - 1) * S rows and layer l reads token t of request b from
    flat row b * ctx + t + l * S, so layers that select the same tokens read different rows. ``noio`` keeps a
    device copy of the host pool and selects the no-IO source. Views of the metadata arrays are exposed as torch
    tensors for inspection.
    """

    def __init__(self, layers, max_batch, ctx, slots, topk_max, row_bytes, host_layers=None, noio=False,
                 host: HostBuffer | None = None, stream=None, layer_shift_rows: int = 0):
        import torch

        self.layers, self.max_batch, self.ctx, self.slots = layers, max_batch, ctx, slots
        self.topk_max, self.row_bytes = topk_max, row_bytes
        self.host_layers = layers if host_layers is None else host_layers
        if self.host_layers not in (1, layers):
            raise ValueError("host_layers must be 1 (shared pool) or equal to layers")
        if layer_shift_rows < 0 or (layer_shift_rows and self.host_layers != 1):
            raise ValueError("layer_shift_rows applies to a shared host pool only")
        self.layer_shift_rows = layer_shift_rows if layers > 1 else 0
        per_layer = max_batch * ctx * row_bytes
        self.extra_rows = (layers - 1) * self.layer_shift_rows
        host_bytes = self.host_layers * per_layer + self.extra_rows * row_bytes
        self.host = host if host is not None else HostBuffer(host_bytes)
        self.hot = torch.zeros(layers * max_batch * slots * row_bytes, dtype=torch.uint8, device="cuda")
        self.noio_src = None
        if noio:
            self.noio_src = torch.empty(host_bytes, dtype=torch.uint8, device="cuda")
        layer_stride = per_layer if self.host_layers == layers else self.layer_shift_rows * row_bytes
        self.desc = hs_pool_desc(layers, max_batch, ctx, slots, topk_max, row_bytes, self.host.ptr, layer_stride, 0,
                                 self.hot.data_ptr(), None, None)
        nbytes = hs_meta_bytes(self.desc)
        if nbytes == 0:
            raise HsError(HS_ERR_INVALID_ARG, "hs_meta_bytes")
        self.meta = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        self.desc.meta = self.meta.data_ptr()
        self.layout = hs_get_meta_layout(self.desc)
        self.handle = None
        self._stream = stream

    def upload_noio(self):
        """Copy the host pool into the no-IO device source (call after filling the host pool)."""
        import torch

        if self.noio_src is None:
            raise ValueError("pool was not created with noio=True")
        src = torch.frombuffer(self.host.numpy(), dtype=torch.uint8)
        self.noio_src.copy_(src)
        self.desc.noio_src = self.noio_src.data_ptr()

    def create(self):
        self.handle = hs_pool_create(self.desc, self._stream)
        return self.handle

    def view(self, name):
        """torch view of a metadata array: step, error (int32 scalar), counters [layers][4] (int64 bit pattern),
        tok2slot [layers][max_batch][ctx], slot_tok / slot_stamp [layers][max_batch][slots]."""
        import torch

        off = self.layout[name]
        L, B = self.layers, self.max_batch
        if name in ("step", "error"):
            return self.meta[off:off + 4].view(torch.int32)
        if name == "counters":
            return self.meta[off:off + 32 * L].view(torch.int64).view(L, 4)
        n = self.ctx if name == "tok2slot" else self.slots
        return self.meta[off:off + 4 * L * B * n].view(torch.int32).view(L, B, n)

    def hot_view(self):
        return self.hot.view(self.layers, self.max_batch, self.slots, self.row_bytes)

    def close(self):
        if self.handle:
            hs_pool_destroy(self.handle)
            self.handle = None
