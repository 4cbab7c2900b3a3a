"""ctypes binding of libasp.so: argument marshalling only.

Every function here has the name of the C entry point it wraps (see
include/asp.h) and does nothing but check tensor dtypes/devices/shapes,
collect pointers and sizes, pass the current torch stream, and raise on a
negative status. All arithmetic of the decode path runs in the library's
CUDA kernels; there is no CPU fallback. If libasp.so is missing the import of
any function fails loudly (build it with adaptive_sparse_paged_gb300.build).
"""

from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libasp.so")

ASP_OK, ASP_EINVAL, ASP_EUNSUPPORTED, ASP_EWORKSPACE, ASP_ECUDA, ASP_EDEVICE = 0, -1, -2, -3, -4, -5
ASP_SUMMARIZE_BULK, ASP_SUMMARIZE_APPEND = 0, 1
ASP_DEVERR_PAGE_RANGE, ASP_DEVERR_LIST_RANGE, ASP_DEVERR_LEN_RANGE = 0x1, 0x2, 0x4
ASP_DEVERR_SEQ_RANGE, ASP_DEVERR_TIMEOUT = 0x8, 0x10
ASP_DEVERR_OFFSET_RANGE = 0x20
ASP_MAX_NEW_TOKENS = 1 << 22

#: every symbol include/asp.h declares
EXPORTED = (
    "asp_abi_version",
    "asp_status_string",
    "asp_workspace_size",
    "asp_workspace_init",
    "asp_page_summarize",
    "asp_coverage_select",
    "asp_coverage_select_append",
    "asp_select_plan",
    "asp_page_scores",
    "asp_sparse_decode",
    "asp_get_device_error",
    "asp_coverage_select_noalloc",
    "asp_selftest_wait_timeout",
    "asp_norm_rotate_append",
    "asp_chunk_attention",
    "asp_chunk_weights",
    "asp_decode_weights",
    "asp_weight_evict",
)


class AspPagedKVStruct(ctypes.Structure):
    """Mirror of asp_paged_kv."""
    _fields_ = [
        ("k_cache", ctypes.c_void_p),
        ("v_cache", ctypes.c_void_p),
        ("summaries", ctypes.c_void_p),
        ("block_table", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
        ("batch", ctypes.c_int32),
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("max_pages", ctypes.c_int32),
        ("num_phys_pages", ctypes.c_int32),
    ]


class AspError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_status_string(status)} (status {status})")


_lib = None
_lock = threading.Lock()


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libasp.so once (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"libasp.so not found at {path}; build it with "
                               "`python -m adaptive_sparse_paged_gb300.build`")
        lib = ctypes.CDLL(path)
        vp, sz, i32, u32p = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32, ctypes.POINTER(ctypes.c_uint32)
        kvp = ctypes.POINTER(AspPagedKVStruct)
        sig = {
            "asp_abi_version": ([], i32),
            "asp_status_string": ([i32], ctypes.c_char_p),
            "asp_workspace_size": ([kvp, ctypes.POINTER(sz)], i32),
            "asp_workspace_init": ([vp, sz, vp], i32),
            "asp_page_summarize": ([kvp, i32, vp, vp, vp, sz, vp], i32),
            "asp_coverage_select": ([kvp, vp, ctypes.c_float, i32, vp, vp, vp, sz, vp], i32),
            "asp_page_scores": ([kvp, vp, vp, vp, sz, vp], i32),
            "asp_select_plan": ([kvp, ctypes.c_float, i32, i32, ctypes.POINTER(i32),
                                 ctypes.POINTER(i32)], i32),
            "asp_coverage_select_append": ([kvp, vp, vp, vp, ctypes.c_float, i32, vp, vp, vp,
                                            sz, vp], i32),
            "asp_sparse_decode": ([kvp, vp, vp, vp, ctypes.c_float, vp, vp, vp, sz, vp], i32),
            "asp_get_device_error": ([vp, u32p, vp], i32),
            "asp_coverage_select_noalloc": ([kvp, vp, ctypes.c_float, i32, vp, vp, vp, vp], i32),
            "asp_selftest_wait_timeout": ([vp, sz, vp], i32),
            "asp_norm_rotate_append": ([kvp, vp, vp, i32, vp, vp, vp, ctypes.c_float, vp, i32, i32,
                                        vp, vp, vp, sz, vp], i32),
            "asp_chunk_attention": ([kvp, vp, vp, i32, ctypes.c_float, vp, vp, vp, sz, vp], i32),
            "asp_chunk_weights": ([kvp, vp, vp, i32, vp, ctypes.c_float, ctypes.c_float, vp, vp,
                                   vp, sz, vp], i32),
            "asp_decode_weights": ([kvp, vp, vp, vp, vp, ctypes.c_float, ctypes.c_float, vp, vp,
                                    vp, sz, vp], i32),
            "asp_weight_evict": ([kvp, vp, i32, i32, vp, vp, vp, vp, vp, sz, vp], i32),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def _status_string(status: int) -> str:
    try:
        return load_library().asp_status_string(int(status)).decode()
    except Exception:  # the library itself failed to load
        return "status"


def _check(status: int, where: str) -> None:
    if status != ASP_OK:
        raise AspError(status, where)


def _stream_ptr(device: torch.device, stream=None) -> int:
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


def _run(name: str, device: torch.device, *args) -> None:
    """Calls an entry point with `device` current and raises on its status."""
    fn = getattr(_lib or load_library(), name)
    if torch._C._cuda_getDevice() == device.index:
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status != ASP_OK:
        raise AspError(status, name)


def _need(t: torch.Tensor, name: str, dtype, device, shape=None):
    try:  # what is right is seen first and cheaply; the rest finds out what is not
        if (t.dtype is dtype and t.get_device() == device.index
                and (shape is None or t.shape == shape) and t.is_contiguous()):
            return
    except (AttributeError, RuntimeError):
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


@dataclass
class PagedKV:
    """One layer's paged cache (device tensors), mirrored into asp_paged_kv.

    k_cache, v_cache : bf16 [num_phys_pages, Hkv, P, d]
    summaries        : bf16 [B, Hkv, max_pages, 2, d], logical page order
    block_table      : int32 [B, max_pages]
    seq_lens         : int32 [B]
    num_q_heads      : Hq (query head h reads KV head h // (Hq // Hkv))
    """
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    summaries: torch.Tensor
    block_table: torch.Tensor
    seq_lens: torch.Tensor
    num_q_heads: int

    def __post_init__(self):
        dev = self.k_cache.device
        if dev.type != "cuda":
            raise ValueError("PagedKV tensors must live on a CUDA device")
        n, hkv, p, d = self.k_cache.shape
        _need(self.k_cache, "k_cache", torch.bfloat16, dev)
        _need(self.v_cache, "v_cache", torch.bfloat16, dev, (n, hkv, p, d))
        _need(self.block_table, "block_table", torch.int32, dev)
        b, max_pages = self.block_table.shape
        _need(self.summaries, "summaries", torch.bfloat16, dev, (b, hkv, max_pages, 2, d))
        _need(self.seq_lens, "seq_lens", torch.int32, dev, (b,))
        self.device = dev
        self.batch, self.num_kv_heads, self.page_size, self.head_dim = b, hkv, p, d
        self.max_pages, self.num_phys_pages = max_pages, n
        self.struct = AspPagedKVStruct(
            self.k_cache.data_ptr(), self.v_cache.data_ptr(), self.summaries.data_ptr(),
            self.block_table.data_ptr(), self.seq_lens.data_ptr(), b, int(self.num_q_heads),
            hkv, d, p, max_pages, n)

        # shapes and reference that every call asks for
        self.ref = ctypes.byref(self.struct)
        self.q_shape = (b, int(self.num_q_heads), d)
        self.lens_shape, self.lists_shape = (b, hkv), (b, hkv, max_pages)
        self.offsets_shape = (b + 1,)
        self.weights_shape = (b, hkv, max_pages * p)


def new_summaries(k_cache: torch.Tensor, block_table: torch.Tensor) -> torch.Tensor:
    """Zeroed summaries tensor [B, Hkv, max_pages, 2, d] for this cache and table."""
    _, hkv, _, d = k_cache.shape
    b, max_pages = block_table.shape
    return torch.zeros((b, hkv, max_pages, 2, d), dtype=torch.bfloat16, device=k_cache.device)


# ----------------------------------------------------------- C-ABI mirrors
def asp_abi_version() -> int:
    return int(load_library().asp_abi_version())


def asp_workspace_size(kv: PagedKV) -> int:
    out = ctypes.c_size_t(0)
    _run("asp_workspace_size", kv.device, kv.ref, ctypes.byref(out))
    return int(out.value)


def asp_workspace_init(ws: torch.Tensor, stream=None) -> None:
    _need(ws, "ws", torch.uint8, ws.device)
    _run("asp_workspace_init", ws.device, ws.data_ptr(), ws.numel(), _stream_ptr(ws.device, stream))


def asp_page_summarize(kv: PagedKV, mode: int, k_new, v_new, ws: torch.Tensor, stream=None) -> None:
    if mode == ASP_SUMMARIZE_APPEND:
        shape = (kv.batch, kv.num_kv_heads, kv.head_dim)
        _need(k_new, "k_new", torch.bfloat16, kv.device, shape)
        _need(v_new, "v_new", torch.bfloat16, kv.device, shape)
        kp, vp = k_new.data_ptr(), v_new.data_ptr()
    else:
        kp = vp = None
    _need(ws, "ws", torch.uint8, kv.device)
    _run("asp_page_summarize", kv.device, kv.ref, int(mode), kp, vp, ws.data_ptr(), ws.numel(),
         _stream_ptr(kv.device, stream))


def asp_coverage_select(kv: PagedKV, q: torch.Tensor, gamma: float, budget: int,
                        lists: torch.Tensor, lens: torch.Tensor, ws: torch.Tensor,
                        stream=None) -> None:
    _need(q, "q", torch.float32, kv.device, kv.q_shape)
    _need(lists, "lists", torch.int32, kv.device, kv.lists_shape)
    _need(lens, "lens", torch.int32, kv.device, kv.lens_shape)
    _need(ws, "ws", torch.uint8, kv.device)
    _run("asp_coverage_select", kv.device, kv.ref, q.data_ptr(), float(gamma), int(budget),
         lists.data_ptr(), lens.data_ptr(), ws.data_ptr(), ws.numel(), _stream_ptr(kv.device,
         stream))


def asp_coverage_select_append(kv: PagedKV, k_new: torch.Tensor, v_new: torch.Tensor,
                               q: torch.Tensor, gamma: float, budget: int, lists: torch.Tensor,
                               lens: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """APPEND (k_new, v_new: bf16 [B, Hkv, d]) and coverage selection in one pass."""
    shp = (kv.batch, kv.num_kv_heads, kv.head_dim)
    _need(k_new, "k_new", torch.bfloat16, kv.device, shp)
    _need(v_new, "v_new", torch.bfloat16, kv.device, shp)
    _need(q, "q", torch.float32, kv.device, kv.q_shape)
    _need(lists, "lists", torch.int32, kv.device, kv.lists_shape)
    _need(lens, "lens", torch.int32, kv.device, kv.lens_shape)
    _need(ws, "ws", torch.uint8, kv.device)
    _run("asp_coverage_select_append", kv.device, kv.ref, k_new.data_ptr(), v_new.data_ptr(),
         q.data_ptr(), float(gamma), int(budget), lists.data_ptr(), lens.data_ptr(), ws.data_ptr(),
         ws.numel(), _stream_ptr(kv.device, stream))


def asp_select_plan(kv: PagedKV, gamma: float, budget: int = 0, append: bool = False):
    """(kernels one selection call launches, cluster CTAs per segment or 0)."""
    k, c = ctypes.c_int32(0), ctypes.c_int32(0)
    _run("asp_select_plan", kv.device, kv.ref, float(gamma), int(budget), int(bool(append)),
         ctypes.byref(k), ctypes.byref(c))
    return int(k.value), int(c.value)


def asp_page_scores(kv: PagedKV, q: torch.Tensor, scores: torch.Tensor, ws: torch.Tensor,
                    stream=None) -> None:
    """Per-page scores [B, Hkv, max_pages] fp32 (entries past N_b untouched)."""
    _need(q, "q", torch.float32, kv.device, kv.q_shape)
    _need(scores, "scores", torch.float32, kv.device,
          kv.lists_shape)
    _need(ws, "ws", torch.uint8, kv.device)
    _run("asp_page_scores", kv.device, kv.ref, q.data_ptr(), scores.data_ptr(), ws.data_ptr(),
         ws.numel(), _stream_ptr(kv.device, stream))


def asp_sparse_decode(kv: PagedKV, q: torch.Tensor, lists: torch.Tensor, lens: torch.Tensor,
                      sm_scale: float, out: torch.Tensor, lse: torch.Tensor, ws: torch.Tensor,
                      stream=None) -> None:
    _need(q, "q", torch.float32, kv.device, kv.q_shape)
    _need(lists, "lists", torch.int32, kv.device, kv.lists_shape)
    _need(lens, "lens", torch.int32, kv.device, kv.lens_shape)
    _need(out, "out", torch.float32, kv.device, kv.q_shape)
    _need(lse, "lse", torch.float32, kv.device, (kv.batch, kv.num_q_heads))
    _need(ws, "ws", torch.uint8, kv.device)
    _run("asp_sparse_decode", kv.device, kv.ref, q.data_ptr(), lists.data_ptr(), lens.data_ptr(),
         float(sm_scale), out.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(),
         _stream_ptr(kv.device, stream))


def asp_coverage_select_noalloc(kv: PagedKV, q: torch.Tensor, gamma: float, budget: int,
                                lists: torch.Tensor, lens: torch.Tensor,
                                dev_error: torch.Tensor | None = None, stream=None) -> None:
    """asp_coverage_select with the library's own fixed scratch instead of a workspace.

    For callers that cannot allocate device memory; see include/asp.h for the
    size limit and the rule that overlapping calls must be serialised.
    dev_error: optional int32 [1] device tensor that collects device error bits.
    """
    _need(q, "q", torch.float32, kv.device, kv.q_shape)
    _need(lists, "lists", torch.int32, kv.device, kv.lists_shape)
    _need(lens, "lens", torch.int32, kv.device, kv.lens_shape)
    err_ptr = None
    if dev_error is not None:
        _need(dev_error, "dev_error", torch.int32, kv.device, (1,))
        err_ptr = dev_error.data_ptr()
    _run("asp_coverage_select_noalloc", kv.device, kv.ref, q.data_ptr(), float(gamma), int(budget),
         lists.data_ptr(), lens.data_ptr(), err_ptr, _stream_ptr(kv.device, stream))


def weights_shape(kv: PagedKV):
    """Shape of the attention weights of this cache: [B, Hkv, max_pages * P]."""
    return kv.weights_shape


def new_weights(kv: PagedKV) -> torch.Tensor:
    """Zeroed attention weights [B, Hkv, max_pages * P] fp32 for this cache."""
    return torch.zeros(weights_shape(kv), dtype=torch.float32, device=kv.device)


def _need_rows(kv: PagedKV, t: torch.Tensor, name: str, heads: int) -> int:
    """Packed bf16 rows [num_tokens, heads, d]; returns num_tokens."""
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a tensor [num_tokens, {heads}, {kv.head_dim}]")
    n = t.size(0)
    _need(t, name, torch.bfloat16, kv.device, (n, heads, kv.head_dim))
    return n


def _need_weights(kv: PagedKV, w_in, w_out) -> int | None:
    _need(w_out, "w_out", torch.float32, kv.device, kv.weights_shape)
    if w_in is None:
        return None
    _need(w_in, "w_in", torch.float32, kv.device, kv.weights_shape)
    return w_in.data_ptr()


def asp_norm_rotate_append(kv: PagedKV, qkv: torch.Tensor, q_offsets, positions, q_weight, k_weight,
                           eps: float, inv_freq, interleaved: bool, q_out: torch.Tensor,
                           ws: torch.Tensor, stream=None) -> None:
    """Norms, rotates and writes the new tokens' rows qkv (bf16 [N, Hq + 2 Hkv, d]).

    q_offsets: int32 [B + 1], or None for one row per request; positions: int32
    [N] or None (the slots); q_weight, k_weight: bf16 [d] or None (not normed);
    inv_freq: fp32 [rotary_dim / 2] or None (no rotation); q_out: bf16 or fp32
    [N, Hq, d], the normed and rotated queries."""
    dev = kv.device
    n = _need_rows(kv, qkv, "qkv", kv.num_q_heads + 2 * kv.num_kv_heads)
    offs_ptr = pos_ptr = qw_ptr = kw_ptr = freq_ptr = None
    rotary_dim = 0
    if q_offsets is not None:
        _need(q_offsets, "q_offsets", torch.int32, dev, kv.offsets_shape)
        offs_ptr = q_offsets.data_ptr()
    if positions is not None:
        _need(positions, "positions", torch.int32, dev, (n,))
        pos_ptr = positions.data_ptr() or None
    if q_weight is not None:
        _need(q_weight, "q_weight", torch.bfloat16, dev, (kv.head_dim,))
        qw_ptr = q_weight.data_ptr()
    if k_weight is not None:
        _need(k_weight, "k_weight", torch.bfloat16, dev, (kv.head_dim,))
        kw_ptr = k_weight.data_ptr()
    if inv_freq is not None:
        _need(inv_freq, "inv_freq", torch.float32, dev)
        freq_ptr, rotary_dim = inv_freq.data_ptr(), 2 * inv_freq.numel()
    half = getattr(q_out, "dtype", None) is torch.bfloat16
    _need(q_out, "q_out", torch.bfloat16 if half else torch.float32, dev,
          (n, kv.num_q_heads, kv.head_dim))
    _need(ws, "ws", torch.uint8, dev)
    out_ptr = _rows_ptr(q_out)
    _run("asp_norm_rotate_append", dev, kv.ref, _rows_ptr(qkv), offs_ptr, n, pos_ptr, qw_ptr, kw_ptr,
         float(eps), freq_ptr, rotary_dim, int(bool(interleaved)), out_ptr if half else None,
         None if half else out_ptr, ws.data_ptr(), ws.numel(), _stream_ptr(dev, stream))


def _rows_ptr(t: torch.Tensor) -> int:
    """data_ptr of packed rows; a tensor without rows has none, and the library
    wants an aligned non-null one that it never reads."""
    return t.data_ptr() or 256


def asp_chunk_attention(kv: PagedKV, q: torch.Tensor, q_offsets: torch.Tensor, sm_scale: float,
                        out: torch.Tensor, lse: torch.Tensor, ws: torch.Tensor,
                        stream=None) -> None:
    """Causal attention of the new tokens' rows q (bf16 [N, Hq, d]) over the cache."""
    n = _need_rows(kv, q, "q", kv.num_q_heads)
    _need(q_offsets, "q_offsets", torch.int32, kv.device, kv.offsets_shape)
    _need(out, "out", torch.bfloat16, kv.device, (n, kv.num_q_heads, kv.head_dim))
    _need(lse, "lse", torch.float32, kv.device, (n, kv.num_q_heads))
    _need(ws, "ws", torch.uint8, kv.device)
    _run("asp_chunk_attention", kv.device, kv.ref, _rows_ptr(q), q_offsets.data_ptr(), n,
         float(sm_scale), _rows_ptr(out), _rows_ptr(lse), ws.data_ptr(), ws.numel(),
         _stream_ptr(kv.device, stream))


def asp_chunk_weights(kv: PagedKV, q: torch.Tensor, q_offsets: torch.Tensor, lse: torch.Tensor,
                      sm_scale: float, decay: float, w_in, w_out: torch.Tensor, ws: torch.Tensor,
                      stream=None) -> None:
    """w_out = decay * w_in + the attention weight each cached token got from the rows q."""
    n = _need_rows(kv, q, "q", kv.num_q_heads)
    _need(q_offsets, "q_offsets", torch.int32, kv.device, kv.offsets_shape)
    _need(lse, "lse", torch.float32, kv.device, (n, kv.num_q_heads))
    w_ptr = _need_weights(kv, w_in, w_out)
    _need(ws, "ws", torch.uint8, kv.device)
    _run("asp_chunk_weights", kv.device, kv.ref, _rows_ptr(q), q_offsets.data_ptr(), n,
         _rows_ptr(lse), float(sm_scale), float(decay), w_ptr, w_out.data_ptr(), ws.data_ptr(),
         ws.numel(), _stream_ptr(kv.device, stream))


def asp_decode_weights(kv: PagedKV, q: torch.Tensor, lists, lens, lse: torch.Tensor,
                       sm_scale: float, decay: float, w_in, w_out: torch.Tensor, ws: torch.Tensor,
                       stream=None) -> None:
    """w_out = decay * w_in + the attention weight of a decode step (lists and lens None: every page)."""
    _need(q, "q", torch.float32, kv.device, kv.q_shape)
    lists_ptr = lens_ptr = None
    if lists is not None or lens is not None:
        _need(lists, "lists", torch.int32, kv.device, kv.lists_shape)
        _need(lens, "lens", torch.int32, kv.device, kv.lens_shape)
        lists_ptr, lens_ptr = lists.data_ptr(), lens.data_ptr()
    _need(lse, "lse", torch.float32, kv.device, (kv.batch, kv.num_q_heads))
    w_ptr = _need_weights(kv, w_in, w_out)
    _need(ws, "ws", torch.uint8, kv.device)
    _run("asp_decode_weights", kv.device, kv.ref, q.data_ptr(), lists_ptr, lens_ptr, lse.data_ptr(),
         float(sm_scale), float(decay), w_ptr, w_out.data_ptr(), ws.data_ptr(), ws.numel(),
         _stream_ptr(kv.device, stream))


def asp_weight_evict(kv: PagedKV, weights: torch.Tensor, keep: int, recent: int,
                     dst_table: torch.Tensor, w_out: torch.Tensor, kept: torch.Tensor,
                     new_lens: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """Keeps the `recent` newest and the heaviest other tokens of every head, `keep` in all."""
    _need(weights, "weights", torch.float32, kv.device, kv.weights_shape)
    _need(dst_table, "dst_table", torch.int32, kv.device, (kv.batch, kv.max_pages))
    _need(w_out, "w_out", torch.float32, kv.device, kv.weights_shape)
    _need(kept, "kept", torch.int32, kv.device, (kv.batch, kv.num_kv_heads, int(keep)))
    _need(new_lens, "new_lens", torch.int32, kv.device, (kv.batch,))
    _need(ws, "ws", torch.uint8, kv.device)
    _run("asp_weight_evict", kv.device, kv.ref, weights.data_ptr(), int(keep), int(recent),
         dst_table.data_ptr(), w_out.data_ptr(), kept.data_ptr(), new_lens.data_ptr(),
         ws.data_ptr(), ws.numel(), _stream_ptr(kv.device, stream))


def asp_selftest_wait_timeout(ws: torch.Tensor, stream=None) -> None:
    """Failure-detection self-test: a bounded on-chip wait that runs out (~2 s)
    and sets ASP_DEVERR_TIMEOUT in `ws`'s error word (read it with
    asp_get_device_error)."""
    _need(ws, "ws", torch.uint8, ws.device)
    _run("asp_selftest_wait_timeout", ws.device, ws.data_ptr(), ws.numel(),
         _stream_ptr(ws.device, stream))


def asp_get_device_error(ws: torch.Tensor, stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error mask."""
    code = ctypes.c_uint32(0)
    with torch.cuda.device(ws.device):
        st = load_library().asp_get_device_error(ws.data_ptr(), ctypes.byref(code),
                                                 _stream_ptr(ws.device, stream))
    if st not in (ASP_OK, ASP_EDEVICE):
        _check(st, "asp_get_device_error")
    return int(code.value)


def new_workspace(kv: PagedKV, stream=None) -> torch.Tensor:
    """Allocates (through torch) and zero-initialises a workspace for `kv`'s shape."""
    n = asp_workspace_size(kv)
    ws = torch.empty(n, dtype=torch.uint8, device=kv.device)
    asp_workspace_init(ws, stream)
    return ws
