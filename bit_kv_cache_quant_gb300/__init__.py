"""GB300 compressed KV cache for single-token LLM decode: Python binding.

A thin ctypes layer over ``libkvq.so`` (the C ABI declared in
``include/kvq.h``).  It only marshals arguments: torch tensors become raw
device pointers, the current torch stream becomes the ``cudaStream_t``, and
every step of the path runs in the library's CUDA kernels.  Importing this
package fails loudly when the library has not been built; there is no
fallback of any kind.

The functions named ``kvq_*`` / ``snapkv_*`` mirror the C entry points one
to one; :class:`KVCache` bundles a cache buffer, its handle and a decode
workspace for convenience.  :class:`Rope`, :func:`rope_qk` and
:class:`PagedKVCache` are the rotary and paged-cache calls on torch tensors.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
from ctypes import POINTER, Structure, byref, c_char_p, c_double, c_float, c_int32, c_int64, c_size_t, c_uint64, c_void_p
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkvq.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "kvq.h")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        "libkvq.so is not built; run `python -c 'import __graft_entry__ as g; g.build()'` "
        "(or bit_kv_cache_quant_gb300/build.py) first")

lib = ctypes.CDLL(LIB_PATH)

# ------------------------------------------------------------------ enums --
KVQ_OK = 0
STATUS_NAMES = {0: "KVQ_OK", 1: "KVQ_ERR_INVALID_ARG", 2: "KVQ_ERR_UNSUPPORTED", 3: "KVQ_ERR_CAPACITY",
                4: "KVQ_ERR_DEVICE", 5: "KVQ_ERR_CUDA"}
FORMATS = {"fp16": 0, "kivi_chan": 1, "affine_token": 2, "q4_0": 3, "kivi_block": 4}
LAYOUTS = {"linear": 0, "compact": 1, "ring": 2}
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
EVICT_MIDDLE = 0
EVICT_KEEPSET = 1
APPEND_CALIBRATE_K = 1
APPEND_RECOMPUTE_K = 2
STEP_EARLY_READ = 1
DEV_OK, DEV_OVERFLOW, DEV_BAD_KEEPSET, DEV_TIMEOUT, DEV_BAD_PAGE = 0, 1, 2, 3, 4
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "llama3": 4, "factors": 5}


class kvq_config(Structure):
    _fields_ = [("batch", c_int32), ("n_kv_heads", c_int32), ("head_dim", c_int32), ("capacity", c_int32),
                ("layout", c_int32), ("sink", c_int32), ("window", c_int32),
                ("k_format", c_int32), ("k_bits", c_int32), ("k_group", c_int32),
                ("v_format", c_int32), ("v_bits", c_int32), ("v_group", c_int32),
                ("k_bias", c_void_p)]


class kvq_cache_layout(Structure):
    _fields_ = [("total_bytes", c_size_t), ("cap_alloc", c_int32), ("k_row_bytes", c_int32),
                ("v_row_bytes", c_int32), ("k_n_groups", c_int32), ("v_n_groups", c_int32),
                ("state", c_size_t), ("split_sem", c_size_t),
                ("k_codes", c_size_t), ("k_tok_scale", c_size_t), ("k_tok_zero", c_size_t),
                ("k_ch_scale", c_size_t), ("k_ch_zero", c_size_t), ("k_ch_scale32", c_size_t),
                ("k_ch_zero32", c_size_t), ("k_bias", c_size_t),
                ("v_codes", c_size_t), ("v_tok_scale", c_size_t), ("v_tok_zero", c_size_t),
                ("k_blk_scale", c_size_t), ("k_blk_zero", c_size_t), ("k_tail", c_size_t), ("v_tail", c_size_t)]


class kvq_stats(Structure):
    _fields_ = [("pos", c_int64), ("stored", c_int32), ("capacity", c_int32), ("device_status", c_int32),
                ("k_calibrated", c_int32), ("cache_bytes", c_size_t), ("live_bytes", c_size_t),
                ("tail", c_int32)]


class kvq_rope_config(Structure):
    _fields_ = [("rot_dim", c_int32), ("scaling", c_int32), ("base", c_double), ("factor", c_double),
                ("original_max_position", c_double), ("beta_fast", c_double), ("beta_slow", c_double),
                ("low_freq_factor", c_double), ("high_freq_factor", c_double), ("factors", POINTER(c_double)),
                ("attn_factor", c_double)]


class kvq_rope(Structure):
    _fields_ = [("freqs", c_void_p), ("rot_dim", c_int32), ("interleaved", c_int32), ("attn_factor", c_float)]


class kvq_rows(Structure):
    _fields_ = [("in_", c_void_p), ("out", c_void_p), ("in_tok_stride", c_int64), ("in_head_stride", c_int64),
                ("out_tok_stride", c_int64), ("out_head_stride", c_int64), ("heads", c_int32),
                ("norm_weight", c_void_p)]


class kvq_paged_config(Structure):
    _fields_ = [("n_kv_heads", c_int32), ("head_dim", c_int32), ("page_size", c_int32), ("n_pages", c_int32),
                ("k_format", c_int32), ("k_bits", c_int32), ("k_group", c_int32),
                ("v_format", c_int32), ("v_bits", c_int32), ("v_group", c_int32)]


class kvq_paged_layout(Structure):
    _fields_ = [("total_bytes", c_size_t), ("k_row_bytes", c_int32), ("v_row_bytes", c_int32),
                ("k_n_groups", c_int32), ("v_n_groups", c_int32), ("state", c_size_t), ("k_codes", c_size_t),
                ("k_meta", c_size_t), ("v_codes", c_size_t), ("v_meta", c_size_t)]


class kvq_paged_batch(Structure):
    _fields_ = [("n_seqs", c_int32), ("max_pages", c_int32), ("page_table", c_void_p), ("seq_lens", c_void_p),
                ("max_prefix_pages", c_int32), ("prefix_pages", c_void_p), ("prefix_len", c_void_p)]


def _proto(name, res, *args):
    f = getattr(lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_proto("kvq_cache_layout_query", c_int32, POINTER(kvq_config), POINTER(kvq_cache_layout))
_proto("kvq_cache_init", c_int32, POINTER(kvq_config), c_void_p, c_size_t, c_void_p, POINTER(c_void_p))
_proto("kvq_cache_release", None, c_void_p)
_proto("kvq_append", c_int32, c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p)
_proto("kvq_convert", c_int32, c_void_p, c_void_p, c_void_p, c_int64, c_int32, c_int32, c_int32, c_void_p)
_proto("kvq_evict", c_int32, c_void_p, c_int32, c_void_p, c_int32, c_void_p)
_proto("kvq_decode_workspace_bytes", c_size_t, c_void_p, c_int32)
_proto("kvq_decode_plan_query", c_int32, POINTER(kvq_config), c_int32, c_int32, POINTER(c_int32), POINTER(c_int32),
       POINTER(c_int32))
_proto("kvq_decode_attn", c_int32, c_void_p, c_void_p, c_void_p, c_int32, c_int32, c_float, c_void_p, c_size_t,
       c_void_p)
_proto("kvq_append_decode", c_int32, c_void_p, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_int32, c_int32,
       c_float, c_void_p, c_size_t, c_int32, c_void_p)
_proto("kvq_append_decode_layers", c_int32, c_int32, POINTER(c_void_p), POINTER(c_void_p), POINTER(c_void_p), c_int32,
       POINTER(c_void_p), POINTER(c_void_p), c_int32, c_int32, c_float, POINTER(c_void_p), POINTER(c_size_t), c_int32,
       c_void_p)
_proto("kvq_test_stall_decode_tiles", None, c_int32)
_proto("snapkv_workspace_bytes", c_size_t, c_int32, c_int32, c_int32, c_int32, c_int32)
_proto("snapkv_pool", c_int32, c_void_p, c_void_p, c_int32, c_int32, c_int32, c_int32, c_void_p)
_proto("snapkv_select", c_int32, c_void_p, c_int64, c_int32, c_int32, c_int32, c_int32, c_int32, c_int32, c_int32,
       c_void_p, c_void_p, c_void_p, c_size_t, c_void_p)
_proto("snapkv_topk", c_int32, c_void_p, c_int32, c_int32, c_int32, c_int32, c_int32, c_void_p, c_void_p)
_proto("kvq_rope_table", c_int32, POINTER(kvq_rope_config), POINTER(c_uint64), POINTER(c_float))
# kvq_rows, kvq_rope and kvq_paged_batch arguments: byref(struct), or its bytes
_proto("kvq_rope_qk", c_int32, c_void_p, c_void_p, c_int32, c_int32, c_int32, c_void_p, c_void_p, c_float, c_void_p)
_proto("kvq_paged_layout_query", c_int32, POINTER(kvq_paged_config), POINTER(kvq_paged_layout))
_proto("kvq_paged_init", c_int32, POINTER(kvq_paged_config), c_void_p, c_size_t, c_void_p, POINTER(c_void_p))
_proto("kvq_paged_release", None, c_void_p)
_proto("kvq_paged_append", c_int32, c_void_p, c_void_p, c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_int32,
       c_void_p, c_void_p, c_float, c_void_p)
_proto("kvq_paged_workspace_bytes", c_size_t, c_void_p, c_int32, c_int32, c_int32)
_proto("kvq_paged_decode_attn", c_int32, c_void_p, c_void_p, c_void_p, c_void_p, c_int32, c_int32,
       c_float, c_void_p, c_size_t, c_void_p)
_proto("kvq_paged_status", c_int32, c_void_p, POINTER(c_int32))
_proto("kvq_paged_clear_status", c_int32, c_void_p, c_void_p)
_proto("kvq_stats_read", c_int32, c_void_p, POINTER(kvq_stats))
_proto("kvq_clear_status", c_int32, c_void_p, c_void_p)
_proto("kvq_last_launch_count", c_int32)
_proto("kvq_last_error", c_char_p)
_proto("kvq_abi_version", c_int32)


class KvqError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


def _check(status: int) -> None:
    if status != KVQ_OK:
        raise KvqError(status, (lib.kvq_last_error() or b"").decode())


def declared_functions() -> list:
    """Names of the functions include/kvq.h declares."""
    with open(HEADER_PATH) as f:
        text = f.read()
    return sorted(set(re.findall(r"^\s*(?:kvq_status|size_t|void|int32_t|const char\*)\s+(\w+)\s*\(", text, re.M)))


def _stream(stream=None) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dev_ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def make_config(batch, n_kv_heads, head_dim, capacity, k_format, k_bits, k_group, v_format, v_bits, v_group,
                layout="linear", sink=0, window=0, k_bias: Optional[torch.Tensor] = None) -> kvq_config:
    return kvq_config(batch, n_kv_heads, head_dim, capacity, LAYOUTS[layout], sink, window,
                      FORMATS[k_format], k_bits, k_group, FORMATS[v_format], v_bits, v_group,
                      None if k_bias is None else _dev_ptr(k_bias))


# ------------------------------------------------------- C entry points --

def kvq_cache_layout_query(cfg: kvq_config) -> kvq_cache_layout:
    lay = kvq_cache_layout()
    _check(lib.kvq_cache_layout_query(byref(cfg), byref(lay)))
    return lay


def kvq_cache_init(cfg: kvq_config, buf: torch.Tensor, stream=None) -> c_void_p:
    h = c_void_p()
    _check(lib.kvq_cache_init(byref(cfg), _dev_ptr(buf), buf.numel() * buf.element_size(), _stream(stream),
                              byref(h)))
    return h


def kvq_append(cache, k: torch.Tensor, v: torch.Tensor, n_tokens: int, in_dtype: int, flags: int = 0,
               stream=None) -> None:
    _check(lib.kvq_append(cache, _dev_ptr(k), _dev_ptr(v), n_tokens, in_dtype, flags, _stream(stream)))


def kvq_convert(cache, k: torch.Tensor, v: torch.Tensor, head_stride: int, n_tokens: int, in_dtype: int,
                flags: int = 0, stream=None) -> None:
    _check(lib.kvq_convert(cache, _dev_ptr(k), _dev_ptr(v), head_stride, n_tokens, in_dtype, flags,
                           _stream(stream)))


def kvq_evict(cache, mode: int, keep_idx: Optional[torch.Tensor] = None, n_keep: int = 0, stream=None) -> None:
    _check(lib.kvq_evict(cache, mode, _dev_ptr(keep_idx), n_keep, _stream(stream)))


def kvq_decode_workspace_bytes(cache, n_q_heads: int) -> int:
    return lib.kvq_decode_workspace_bytes(cache, n_q_heads)


def kvq_decode_plan_query(cfg: kvq_config, n_q_heads: int, sms: int):
    """(splits, tensor-core splits, wide) of the decode launch for this configuration and SM count."""
    ns, ntc, wide = c_int32(), c_int32(), c_int32()
    _check(lib.kvq_decode_plan_query(byref(cfg), n_q_heads, sms, byref(ns), byref(ntc), byref(wide)))
    return ns.value, ntc.value, wide.value


def kvq_decode_attn(cache, q: torch.Tensor, out: torch.Tensor, n_q_heads: int, io_dtype: int,
                    softmax_scale: float = 0.0, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.kvq_decode_attn(cache, _dev_ptr(q), _dev_ptr(out), n_q_heads, io_dtype, softmax_scale,
                               _dev_ptr(workspace), ws_bytes, _stream(stream)))


def kvq_append_decode(cache, k: torch.Tensor, v: torch.Tensor, in_dtype: int, q: torch.Tensor, out: torch.Tensor,
                      n_q_heads: int, io_dtype: int, softmax_scale: float = 0.0,
                      workspace: Optional[torch.Tensor] = None, flags: int = 0, stream=None) -> None:
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.kvq_append_decode(cache, _dev_ptr(k), _dev_ptr(v), in_dtype, _dev_ptr(q), _dev_ptr(out), n_q_heads,
                                 io_dtype, softmax_scale, _dev_ptr(workspace), ws_bytes, flags, _stream(stream)))


def kvq_append_decode_layers(caches: list, ks: list, vs: list, in_dtype: int, qs: list, outs: list, n_q_heads: int,
                             io_dtype: int, softmax_scale: float = 0.0, workspaces: Optional[list] = None,
                             flags: int = 0, stream=None) -> None:
    n = len(caches)
    arr = lambda xs: (c_void_p * n)(*xs)
    ws = wsb = None
    if workspaces is not None:
        ws = arr([_dev_ptr(w) for w in workspaces])
        wsb = (c_size_t * n)(*[0 if w is None else w.numel() * w.element_size() for w in workspaces])
    _check(lib.kvq_append_decode_layers(n, arr([c.value for c in caches]), arr([_dev_ptr(t) for t in ks]),
                                        arr([_dev_ptr(t) for t in vs]), in_dtype, arr([_dev_ptr(t) for t in qs]),
                                        arr([_dev_ptr(t) for t in outs]), n_q_heads, io_dtype, softmax_scale, ws, wsb,
                                        flags, _stream(stream)))


class LayerStep:
    """One decode step over a stack of layer caches as one call (kvq_append_decode_layers):
    layer l appends ks[l], vs[l] [B, Hkv, 1, D] to caches[l], evicts, and attends with
    qs[l] [B, Hq, D] into outs[l].  The per-layer pointer arrays are built once here, so the
    tensors must stay alive and in place while the step is in use."""

    def __init__(self, caches: list, ks: list, vs: list, qs: list, outs: list, softmax_scale: float = 0.0):
        n = len(caches)
        if not n or not all(len(x) == n for x in (ks, vs, qs, outs)):
            raise ValueError("one k, v, q and out per cache")
        for c, k, v, q, o in zip(caches, ks, vs, qs, outs):
            c._check_rows(k, v)
            if k.shape[2] != 1:
                raise ValueError("a step takes one token per (batch row, kv head)")
            if q.dim() != 3 or q.shape[0] != c.batch or q.shape[2] != c.head_dim or q.dtype not in DTYPES:
                raise ValueError(f"q must be [{c.batch}, Hq, {c.head_dim}] fp32 / bf16 / fp16")
            if o.shape != q.shape or o.dtype != q.dtype:
                raise ValueError("out must have q's shape and dtype")
        self.n = n
        self.hq = qs[0].shape[1]
        self.in_dtype, self.io_dtype = DTYPES[ks[0].dtype], DTYPES[qs[0].dtype]
        self.softmax_scale = softmax_scale
        ws = [c.workspace(self.hq) for c in caches]
        arr = lambda xs: (c_void_p * n)(*xs)
        self._args = (arr([c.handle.value for c in caches]), arr([_dev_ptr(t) for t in ks]),
                      arr([_dev_ptr(t) for t in vs]), arr([_dev_ptr(t) for t in qs]),
                      arr([_dev_ptr(t) for t in outs]), arr([_dev_ptr(w) for w in ws]),
                      (c_size_t * n)(*[0 if w is None else w.numel() * w.element_size() for w in ws]))
        self._keep = (list(caches), list(ks), list(vs), list(qs), list(outs), ws)
        self._handles = tuple(c.handle for c in caches)   # the handle objects: reset() makes new ones
        self.launches = 0

    def run(self, early_read: bool = False, stream=None) -> None:
        """early_read: the kernel just before this call on the stream writes none of the caches."""
        if any(c.handle is not h for c, h in zip(self._keep[0], self._handles)):
            raise ValueError("a cache of this step was reset or released; build a new LayerStep")
        h, k, v, q, o, ws, wsb = self._args
        _check(lib.kvq_append_decode_layers(self.n, h, k, v, self.in_dtype, q, o, self.hq, self.io_dtype,
                                            self.softmax_scale, ws, wsb, STEP_EARLY_READ if early_read else 0,
                                            _stream(stream)))
        self.launches = kvq_last_launch_count()


def kvq_test_stall_decode_tiles(on: bool) -> None:
    lib.kvq_test_stall_decode_tiles(1 if on else 0)


def snapkv_workspace_bytes(batch, n_kv_heads, S, head_dim, obs_window) -> int:
    return lib.snapkv_workspace_bytes(batch, n_kv_heads, S, head_dim, obs_window)


def snapkv_select(k: torch.Tensor, head_stride: int, batch: int, n_kv_heads: int, S: int, head_dim: int,
                  obs_window: int, budget: int, n_sink: int, scores_out: Optional[torch.Tensor],
                  idx_out: torch.Tensor, workspace: torch.Tensor, stream=None) -> None:
    _check(lib.snapkv_select(_dev_ptr(k), head_stride, batch, n_kv_heads, S, head_dim, obs_window, budget, n_sink,
                             _dev_ptr(scores_out), _dev_ptr(idx_out), _dev_ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream(stream)))


def snapkv_pool(scores: torch.Tensor, pooled: torch.Tensor, kernel_size: int, stream=None) -> torch.Tensor:
    """Max-pool smoothing of scores [B, Hkv, S] (fp32, device) into pooled (same shape)."""
    B, H, S = scores.shape
    _check(lib.snapkv_pool(_dev_ptr(scores), _dev_ptr(pooled), B, H, S, kernel_size, _stream(stream)))
    return pooled


def snapkv_topk(scores: torch.Tensor, batch: int, n_kv_heads: int, S: int, budget: int, n_sink: int,
                idx_out: torch.Tensor, stream=None) -> None:
    _check(lib.snapkv_topk(_dev_ptr(scores), batch, n_kv_heads, S, budget, n_sink, _dev_ptr(idx_out),
                           _stream(stream)))


def kvq_stats_read(cache) -> kvq_stats:
    st = kvq_stats()
    status = lib.kvq_stats_read(cache, byref(st))
    if status not in (KVQ_OK, 4):      # KVQ_ERR_DEVICE still fills the counters
        _check(status)
    return st


def kvq_clear_status(cache, stream=None) -> None:
    _check(lib.kvq_clear_status(cache, _stream(stream)))


def kvq_last_launch_count() -> int:
    return lib.kvq_last_launch_count()


# ------------------------------------------------------------ convenience --

class KVCache:
    """One layer's compressed cache: a device buffer, its handle and a decode workspace."""

    def __init__(self, batch, n_kv_heads, head_dim, capacity, k_format="fp16", k_bits=16, k_group=0,
                 v_format="fp16", v_bits=16, v_group=0, layout="linear", sink=0, window=0,
                 k_bias: Optional[torch.Tensor] = None, device="cuda", stream=None):
        self.cfg = make_config(batch, n_kv_heads, head_dim, capacity, k_format, k_bits, k_group, v_format, v_bits,
                               v_group, layout, sink, window, k_bias)
        self.layout = kvq_cache_layout_query(self.cfg)
        self._bias = k_bias      # kept alive until the stream-ordered copy in kvq_cache_init has run
        self.buf = torch.empty(self.layout.total_bytes, dtype=torch.uint8, device=device)
        self.handle = kvq_cache_init(self.cfg, self.buf, stream)
        self.batch, self.n_kv_heads, self.head_dim = batch, n_kv_heads, head_dim
        self._ws = {}
        self.launches = 0

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            lib.kvq_cache_release(h)
            self.handle = None

    def reset(self, stream=None) -> None:
        """Empties the cache (counters to zero) on the same device buffer."""
        lib.kvq_cache_release(self.handle)
        self.handle = None
        self.handle = kvq_cache_init(self.cfg, self.buf, stream)

    def _check_rows(self, k: torch.Tensor, v: torch.Tensor) -> None:
        """k, v: one shape [B, Hkv, n, D] of this cache and one dtype: the C call gets raw pointers and
        reads both with k's dtype.  One short-circuit test on the common path (eager decode calls it
        once per layer)."""
        s = k.shape
        if (s != v.shape or k.dtype is not v.dtype or len(s) != 4 or s[0] != self.batch
                or s[1] != self.n_kv_heads or s[3] != self.head_dim):
            if s != v.shape or k.dtype is not v.dtype:
                raise ValueError(f"k {tuple(s)} {k.dtype} and v {tuple(v.shape)} {v.dtype} must match")
            raise ValueError(f"k and v must be [{self.batch}, {self.n_kv_heads}, n, {self.head_dim}], "
                             f"got {tuple(s)}")
        if k.dtype not in DTYPES:
            raise ValueError(f"unsupported input dtype {k.dtype}")

    def append(self, k: torch.Tensor, v: torch.Tensor, calibrate_k: bool = False, recompute_k: bool = False,
               stream=None) -> None:
        self._check_rows(k, v)
        n = k.shape[2]
        flags = (APPEND_CALIBRATE_K if calibrate_k else 0) | (APPEND_RECOMPUTE_K if recompute_k else 0)
        kvq_append(self.handle, k, v, n, DTYPES[k.dtype], flags, stream)
        self.launches += kvq_last_launch_count()

    def convert(self, k: torch.Tensor, v: torch.Tensor, n_tokens: int, calibrate_k: bool = False,
                stream=None) -> None:
        """Quantises the first n_tokens tokens of a dense cache k, v [B, Hkv, C, D] (C >= n_tokens,
        rows contiguous) into this cache."""
        if k.shape != v.shape or k.dim() != 4 or not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("k and v must be contiguous [B, Hkv, C, D] tensors of one shape")
        self._check_rows(k, v)
        if not 1 <= n_tokens <= k.shape[2]:
            raise ValueError(f"n_tokens must be in 1..{k.shape[2]}")
        kvq_convert(self.handle, k, v, k.shape[2], n_tokens, DTYPES[k.dtype],
                    APPEND_CALIBRATE_K if calibrate_k else 0, stream)
        self.launches += kvq_last_launch_count()

    def evict_middle(self, stream=None) -> None:
        kvq_evict(self.handle, EVICT_MIDDLE, None, 0, stream)
        self.launches += kvq_last_launch_count()

    def evict_keepset(self, idx: torch.Tensor, stream=None) -> None:
        kvq_evict(self.handle, EVICT_KEEPSET, idx, idx.shape[-1], stream)
        self.launches += kvq_last_launch_count()

    def workspace(self, n_q_heads: int) -> Optional[torch.Tensor]:
        if n_q_heads not in self._ws:
            nb = kvq_decode_workspace_bytes(self.handle, n_q_heads)
            self._ws[n_q_heads] = torch.empty(nb, dtype=torch.uint8, device=self.buf.device) if nb else None
        return self._ws[n_q_heads]

    def decode_attn(self, q: torch.Tensor, out: Optional[torch.Tensor] = None, softmax_scale: float = 0.0,
                    stream=None) -> torch.Tensor:
        s = q.shape
        if len(s) != 3 or s[0] != self.batch or s[2] != self.head_dim or q.dtype not in DTYPES:
            raise ValueError(f"q must be [{self.batch}, Hq, {self.head_dim}] fp32 / bf16 / fp16, "
                             f"got {tuple(q.shape)} {q.dtype}")
        if out is None:
            out = torch.empty_like(q)
        elif out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must have q's shape and dtype")
        hq = q.shape[1]
        kvq_decode_attn(self.handle, q, out, hq, DTYPES[q.dtype], softmax_scale, self.workspace(hq), stream)
        self.launches += kvq_last_launch_count()
        return out

    def append_decode(self, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor, out: Optional[torch.Tensor] = None,
                      softmax_scale: float = 0.0, early_read: bool = False, stream=None) -> torch.Tensor:
        """One decode step: append the token k, v [B, Hkv, 1, D], evict (streaming layouts) and attend
        with q [B, Hq, D] over the cache including that token.  early_read: the kernel just before
        this call on the stream writes neither this cache nor its counters (KVQ_STEP_EARLY_READ)."""
        self._check_rows(k, v)
        if k.shape[2] != 1:
            raise ValueError("append_decode takes one token per (batch row, kv head)")
        s = q.shape
        if len(s) != 3 or s[0] != self.batch or s[2] != self.head_dim or q.dtype not in DTYPES:
            raise ValueError(f"q must be [{self.batch}, Hq, {self.head_dim}] fp32 / bf16 / fp16, "
                             f"got {tuple(q.shape)} {q.dtype}")
        if out is None:
            out = torch.empty_like(q)
        elif out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must have q's shape and dtype")
        hq = q.shape[1]
        kvq_append_decode(self.handle, k, v, DTYPES[k.dtype], q, out, hq, DTYPES[q.dtype], softmax_scale,
                          self.workspace(hq), STEP_EARLY_READ if early_read else 0, stream)
        self.launches += kvq_last_launch_count()
        return out

    def stats(self) -> kvq_stats:
        return kvq_stats_read(self.handle)

    def plane(self, name: str, nbytes: int) -> torch.Tensor:
        """uint8 view of `nbytes` bytes of plane `name` (a kvq_cache_layout field)."""
        off = getattr(self.layout, name)
        return self.buf[off: off + nbytes]


def snapkv(k: torch.Tensor, obs_window: int, budget: int, n_sink: int, want_scores: bool = True, stream=None):
    """Scores and kept indices of fp16 keys k [B, Hkv, S, D]."""
    B, H, S, D = k.shape
    ws = torch.empty(snapkv_workspace_bytes(B, H, S, D, obs_window), dtype=torch.uint8, device=k.device)
    scores = torch.empty((B, H, S), dtype=torch.float32, device=k.device) if want_scores else None
    idx = torch.empty((B, H, min(budget, S)), dtype=torch.int32, device=k.device)
    snapkv_select(k, S, B, H, S, D, obs_window, budget, n_sink, scores, idx, ws, stream)
    return scores, idx


# ---------------------------------------------------- positions, paged cache --

def kvq_paged_layout_query(cfg: kvq_paged_config) -> kvq_paged_layout:
    lay = kvq_paged_layout()
    _check(lib.kvq_paged_layout_query(byref(cfg), byref(lay)))
    return lay


def kvq_rope_table(cfg: kvq_rope_config):
    """(table of rot_dim / 2 unsigned 64-bit turn fractions, magnitude of the sines and cosines)."""
    freqs = (c_uint64 * max(1, cfg.rot_dim // 2))()
    mag = c_float()
    _check(lib.kvq_rope_table(byref(cfg), freqs, byref(mag)))
    return list(freqs), mag.value


# The paged and rotary calls run once per layer of a decode step, whose kernels take a few microseconds: the
# checks below read each tensor's properties once, and arguments go as packed bytes in the C structs' layout.
_cur_device = torch._C._cuda_getDevice
_cur_stream = torch._C._cuda_getCurrentRawStream
_capturing = torch._C._cuda_isCurrentStreamCapturing
_ROWS = struct.Struct("@PPqqqqiP")        # kvq_rows
_BATCH = struct.Struct("@iiPPiPP")        # kvq_paged_batch


def _device_of(first: torch.Tensor, *rest) -> int:
    """Index of the one CUDA device all tensors (or None) are on."""
    dev = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"expected a CUDA tensor on {first.device}, got one on {t.device}: one device per call")
    if dev < 0:
        raise ValueError("expected a CUDA tensor")
    return dev


def _call(dev: int, stream, fn, *args) -> None:
    """fn(*args, raw stream) with device `dev` current; `stream` as in the other calls (None: the current one)."""
    if dev == _cur_device():
        status = fn(*args, _cur_stream(dev) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _stream(stream))
    if status:
        _check(status)


def _empty(shape, dtype, dev, stream):
    """An output allocated on the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


class Rope:
    """A rotation's frequency table on the device (kvq_rope_table): the first rot_dim channels of each head
    turn, in pairs (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved.  scaling: "none", "linear" (factor),
    "ntk" (factor), "yarn" (factor, original_max_position, beta_fast, beta_slow), "llama3" (factor,
    original_max_position, low_freq_factor, high_freq_factor) or "factors" (factors, one per pair)."""

    def __init__(self, rot_dim: int, base: float = 10000.0, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, original_max_position: float = 0.0, beta_fast: float = 32.0,
                 beta_slow: float = 1.0, low_freq_factor: float = 1.0, high_freq_factor: float = 4.0,
                 factors=None, attn_factor: float = 0.0, device="cuda"):
        if scaling not in ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(ROPE_SCALINGS)}")
        arr = None
        if factors is not None:
            factors = [float(f) for f in factors]
            if len(factors) != rot_dim // 2:
                raise ValueError("factors needs one value per pair")
            arr = (c_double * len(factors))(*factors)
        cfg = kvq_rope_config(rot_dim, ROPE_SCALINGS[scaling], base, factor, original_max_position, beta_fast,
                              beta_slow, low_freq_factor, high_freq_factor, arr, attn_factor)
        table, self.attn_factor = kvq_rope_table(cfg)
        self.rot_dim, self.interleaved = rot_dim, bool(interleaved)
        signed = [f - (1 << 64) if f >= 1 << 63 else f for f in table]
        self.freqs = torch.tensor(signed, dtype=torch.int64, device=device)   # the 64 bits of each entry
        if self.freqs.is_cuda:
            torch.cuda.current_stream(self.freqs.device).synchronize()   # usable on every stream from here on
        self.arg = bytes(kvq_rope(self.freqs.data_ptr(), rot_dim, int(self.interleaved), self.attn_factor))


def _rows(name, x: torch.Tensor, out: Optional[torch.Tensor], weight: Optional[torch.Tensor], tokens: int,
          head_dim: int, dtype) -> bytes:
    """kvq_rows of x [tokens, heads, head_dim], as packed bytes."""
    s = x.shape
    if len(s) != 3 or x.dtype is not dtype:
        raise ValueError(f"{name} must be [{tokens}, heads, {head_dim}] {dtype}, got {tuple(s)} {x.dtype}")
    n, heads, d = s
    i0, i1, i2 = x.stride()
    if n != tokens or d != head_dim:
        raise ValueError(f"{name} must be [{tokens}, heads, {head_dim}] {dtype}, got {tuple(s)} {x.dtype}")
    if i2 != 1:
        raise ValueError(f"{name}: the channels of a head must be contiguous")
    o0 = o1 = optr = w = 0
    if out is not None:
        if out.shape != s or out.dtype is not dtype:
            raise ValueError(f"{name}_out must have {name}'s shape and dtype, its channels contiguous")
        o0, o1, o2 = out.stride()
        if o2 != 1:
            raise ValueError(f"{name}_out must have {name}'s shape and dtype, its channels contiguous")
        if (not o0 and n > 1) or (not o1 and heads > 1):
            raise ValueError(f"{name}_out must not be an expanded tensor")
        optr = out.data_ptr()
    if weight is not None:
        if weight.shape != (head_dim,) or weight.dtype is not dtype or not weight.is_contiguous():
            raise ValueError(f"{name}_norm must be a contiguous [{head_dim}] tensor of {name}'s dtype")
        w = weight.data_ptr()
    return _ROWS.pack(x.data_ptr(), optr, i0, i1, o0, o1, heads, w)


def _int32(name, t: Optional[torch.Tensor], n: int, cols: Optional[int] = None) -> int:
    """Pointer of a contiguous int32 tensor of n (or n x cols) entries; 0 for None."""
    if t is None:
        return 0
    if t.dtype is not torch.int32 or t.shape != ((n,) if cols is None else (n, cols)) or not t.is_contiguous():
        want = (n,) if cols is None else (n, cols)
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {want}, got {tuple(t.shape)} {t.dtype}")
    return t.data_ptr()


def rope_qk(q: Optional[torch.Tensor], k: Optional[torch.Tensor], positions: Optional[torch.Tensor],
            rope: Optional[Rope], q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
            q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6,
            stream=None):
    """(q_out, k_out): q and k [T, heads, D] normed (RMS over each head, times q_norm / k_norm [D], where
    given), then rotated by positions int32 [T] (rope None: norm only).  Strided q and k, and outputs that
    are the inputs themselves, are fine; either of q and k may be None."""
    x = q if q is not None else k
    s = None if x is None else x.shape
    if s is None or len(s) != 3 or x.dtype not in DTYPES:
        raise ValueError("q and k must be [T, heads, D] fp32 / bf16 / fp16 tensors")
    tokens, _, head_dim = s
    dt = x.dtype
    dev = _device_of(x, k, positions, q_out, k_out, q_norm, k_norm, None if rope is None else rope.freqs)
    rq = rk = None
    if q is not None:
        if q_out is None:
            q_out = _empty(q.shape, dt, dev, stream)
        rq = _rows("q", q, q_out, q_norm, tokens, head_dim, dt)
    if k is not None:
        if k_out is None:
            k_out = _empty(k.shape, dt, dev, stream)
        rk = _rows("k", k, k_out, k_norm, tokens, head_dim, dt)
    _call(dev, stream, lib.kvq_rope_qk, rq, rk, tokens, head_dim, DTYPES[dt], _int32("positions", positions, tokens),
          None if rope is None else rope.arg, eps)
    return q_out, k_out


class PagedKVCache:
    """One layer's pool of pages and its handle.  Page tables, lengths and the batch's shared prefix are the
    caller's int32 device tensors, common to the pools of all layers, and are read by the kernels: a captured
    graph follows what they hold at replay.

    page_table [B, max_pages], seq_lens [B]: token j of sequence b is row j % page_size of page
    page_table[b, j // page_size].  prefix_pages [n], prefix_len [1]: tokens in front of every sequence.

    decode_attn calls that may run at the same time need workspaces of their own.  Without a `workspace`
    argument (workspace_bytes bytes) the pool keeps one for each stream, and a captured call gets one that no
    other call uses, so that graphs may replay beside one another and beside eager calls."""

    def __init__(self, n_kv_heads, head_dim, page_size, n_pages, k_format="fp16", k_bits=16, k_group=0,
                 v_format="fp16", v_bits=16, v_group=0, buf: Optional[torch.Tensor] = None, device="cuda",
                 stream=None):
        self.cfg = kvq_paged_config(n_kv_heads, head_dim, page_size, n_pages, FORMATS[k_format], k_bits, k_group,
                                    FORMATS[v_format], v_bits, v_group)
        self.layout = kvq_paged_layout_query(self.cfg)
        if buf is None:
            buf = torch.zeros(self.layout.total_bytes, dtype=torch.uint8, device=device)
        if not buf.is_cuda or buf.dtype is not torch.uint8 or not buf.is_contiguous():
            raise ValueError("buf must be a contiguous uint8 CUDA tensor")
        self.buf = buf
        h = c_void_p()
        self._dev = buf.get_device()
        _call(self._dev, stream, lambda st: lib.kvq_paged_init(byref(self.cfg), buf.data_ptr(), buf.numel(), st, byref(h)))
        self.handle = h
        self.n_kv_heads, self.head_dim, self.page_size, self.n_pages = n_kv_heads, head_dim, page_size, n_pages
        self._ws = {}          # raw stream -> workspace
        self._kept = []        # workspaces of captured calls
        self._shapes = {}      # (n_seqs, n_q_heads, prefix pages) -> [workspace bytes, launches]
        self.launches = 0

    def __del__(self):
        h = getattr(self, "handle", None)
        if h:
            lib.kvq_paged_release(h)
            self.handle = None

    def _batch(self, page_table, seq_lens, prefix_pages, prefix_len) -> bytes:
        """kvq_paged_batch, as packed bytes."""
        s, n = page_table.shape, seq_lens.shape
        if len(s) != 2 or len(n) != 1 or s[0] != n[0]:
            raise ValueError("page_table must be [B, max_pages] and seq_lens [B]")
        B, cols = s
        npre = 0 if prefix_pages is None else prefix_pages.numel()
        if npre and prefix_len is None:
            raise ValueError("prefix_pages needs prefix_len")
        return _BATCH.pack(B, cols, _int32("page_table", page_table, B, cols), _int32("seq_lens", seq_lens, B), npre,
                           _int32("prefix_pages", prefix_pages, npre), _int32("prefix_len", prefix_len, 1))

    def append(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
               cu_tokens: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
               rope: Optional[Rope] = None, prefix_len: Optional[torch.Tensor] = None,
               positions: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
               k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
               q_norm: Optional[torch.Tensor] = None, k_norm: Optional[torch.Tensor] = None, eps: float = 1e-6,
               stream=None) -> Optional[torch.Tensor]:
        """Stores the step's new tokens k, v [T, Hkv, D] (k normed and rotated on the way) and returns q [T, Hq, D]
        normed and rotated.  seq_lens counts the new tokens; cu_tokens int32 [B + 1] gives each sequence's run of
        tokens (None: one each).  k_out, v_out: where to leave the values the stored rows stand for."""
        s = k.shape
        if len(s) != 3 or k.dtype not in DTYPES:
            raise ValueError("k and v must be [T, Hkv, D] fp32 / bf16 / fp16 tensors")
        dev = _device_of(self.buf, k, v, page_table, seq_lens, cu_tokens, q, prefix_len, positions, q_out, k_out,
                         v_out, q_norm, k_norm, None if rope is None else rope.freqs)
        tokens, dt, D = s[0], k.dtype, self.head_dim
        rq = None
        if q is not None:
            if q_out is None:
                q_out = _empty(q.shape, dt, dev, stream)
            rq = _rows("q", q, q_out, q_norm, tokens, D, dt)
        _call(dev, stream, lib.kvq_paged_append, self.handle, self._batch(page_table, seq_lens, None, prefix_len), tokens,
              _int32("cu_tokens", cu_tokens, page_table.shape[0] + 1), rq, _rows("k", k, k_out, k_norm, tokens, D, dt),
              _rows("v", v, v_out, None, tokens, D, dt), DTYPES[dt], None if rope is None else rope.arg,
              _int32("positions", positions, tokens), eps)
        self.launches += 1 if tokens else 0
        return q_out

    def workspace_bytes(self, n_seqs: int, n_q_heads: int, max_prefix_pages: int = 0) -> int:
        return lib.kvq_paged_workspace_bytes(self.handle, n_seqs, n_q_heads, max_prefix_pages)

    def _workspace(self, need, stream) -> torch.Tensor:
        if _capturing():
            self._kept.append(_empty((need,), torch.uint8, self._dev, stream))
            return self._kept[-1]
        raw = _cur_stream(self._dev) if stream is None else _stream(stream)
        ws = self._ws.get(raw)
        if ws is None or ws.numel() < need:
            # the smaller one goes back to the allocator, which orders it behind this stream's calls
            ws = self._ws[raw] = _empty((need,), torch.uint8, self._dev, stream)
        return ws

    def decode_attn(self, q: torch.Tensor, page_table: torch.Tensor, seq_lens: torch.Tensor,
                    prefix_pages: Optional[torch.Tensor] = None, prefix_len: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None, softmax_scale: float = 0.0,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Attention of q [B, Hq, D] (bf16 / fp16) over the prefix and each sequence's own tokens."""
        s = q.shape
        if len(s) != 3 or s[2] != self.head_dim or q.dtype not in DTYPES or not q.is_contiguous():
            raise ValueError(f"q must be a contiguous [B, Hq, {self.head_dim}] tensor, got {tuple(s)} {q.dtype}")
        dev = _device_of(self.buf, q, page_table, seq_lens, prefix_pages, prefix_len, out, workspace)
        batch = self._batch(page_table, seq_lens, prefix_pages, prefix_len)
        if s[0] != page_table.shape[0]:
            raise ValueError("q and page_table must have one row per sequence")
        if out is None:
            out = _empty(s, q.dtype, dev, stream)
        elif out.shape != s or out.dtype is not q.dtype or not out.is_contiguous():
            raise ValueError("out must have q's shape and dtype")
        key = (s[0], s[1], 0 if prefix_pages is None else prefix_pages.numel())
        shape = self._shapes.get(key)
        if shape is None:      # workspace and launches go by these alone
            if len(self._shapes) >= 4096:
                self._shapes.clear()
            shape = self._shapes[key] = [max(16, self.workspace_bytes(*key)), None]
        ws = self._workspace(shape[0], stream) if workspace is None else workspace
        _call(dev, stream, lib.kvq_paged_decode_attn, self.handle, batch, q.data_ptr(), out.data_ptr(), s[1],
              DTYPES[q.dtype], softmax_scale, ws.data_ptr(), ws.nbytes)
        if shape[1] is None:
            shape[1] = kvq_last_launch_count()
        self.launches += shape[1]
        return out

    def status(self) -> int:
        """The pool's status word (DEV_*); synchronises."""
        st = c_int32()
        _call(self._dev, None, lambda _: lib.kvq_paged_status(self.handle, byref(st)))
        return st.value

    def clear_status(self, stream=None) -> None:
        _call(self._dev, stream, lib.kvq_paged_clear_status, self.handle)

    def plane(self, name: str) -> torch.Tensor:
        """A view of plane k_codes, v_codes, k_meta or v_meta of the pool: codes fp16 [n_pages, Hkv, page_size, D]
        or uint8 [n_pages, Hkv, page_size, row_bytes]; metadata fp16 [n_pages, Hkv, page_size, groups, 2]."""
        side, what = name.split("_")
        rows = (self.n_pages, self.n_kv_heads, self.page_size)
        count = self.n_pages * self.n_kv_heads * self.page_size
        off = getattr(self.layout, name)
        if what == "codes":
            rb = getattr(self.layout, f"{side}_row_bytes")
            x = self.buf[off:off + count * rb].view(*rows, rb)
            return x.view(torch.float16) if self.cfg.k_format == FORMATS["fp16"] else x
        ng = getattr(self.layout, f"{side}_n_groups")
        return self.buf[off:off + count * ng * 4].view(torch.float16).view(*rows, ng, 2)
