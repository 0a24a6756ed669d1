"""GB300 (sm_103a) FP8 paged-KV decode attention and cache append.

Thin ctypes binding over the C ABI declared in ``include/pa_fp8.h``
(``libpa_fp8.so``). This module only marshals arguments: every step runs in
the library's CUDA kernels. PyTorch supplies device memory and the current
stream. There is no fallback: if the library is missing, calls raise.

Functions take torch CUDA tensors and work in place (outputs are arguments):
  decode(...)              paged FP8 decode attention -> BF16
  cache_scatter(...)       FP8 K/V (+ key_scale) append by slot_mapping
  cache_quant_scatter(...) BF16/FP32 K/V quantised to E4M3 on append
  kv_compress_epilog(...)  BF16 rows to rope (BF16) + grouped E4M3 nope (modes 0/1)
  quantize_rows(...)       per-token E4M3 quantiser (Q, K)
  value_channel_scale(...) per-channel V dequant scale
  mla_sparse_decode(...)   MLA sparse attention over a packed FP8 latent cache
  mla_sparse_decode_kvc(...) the same over rows the KV compress epilog wrote
and a speculative decode step over the same cache:
  qkv_norm_rope_append(...) per-head norm, rotation and quantisation of q and k, K/V append
  tree_decode(...)         attention of a tree of drafted tokens
  tree_verify(...)         drafted tokens against the target's probabilities
  cache_keep_path(...)     the accepted branch kept in the cache
and a ragged serving step (requests bring one token or a prompt's chunk each):
  plan_batch(...)          block tables, slots and positions from request lengths
  qkv_norm_mrope_append(...) the append with several position axes (images, video)
  window_attention(...)    attention to a sliding window and the first tokens
  token_logprobs(...)      log probabilities, ranks, entropy and top alternatives
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading

from . import _build

LAYOUT_BSND = 0
LAYOUT_BNBD = 1
DTYPE_F32 = 0
DTYPE_BF16 = 1
INDEX_I32 = 0
INDEX_I64 = 1

PA_OK = 0
_STATUS_NAMES = {0: "PA_OK", 1: "PA_ERR_NULLPTR", 2: "PA_ERR_INVALID", 3: "PA_ERR_WORKSPACE",
                 4: "PA_ERR_CUDA", 5: "PA_ERR_UNSUPPORTED"}

LIB_PATH = _build.LIB_PATH
_lock = threading.Lock()
_lib = None


class PaError(RuntimeError):
    """A non-PA_OK status from the library."""

    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__("%s: %s (%s)" % (where, _STATUS_NAMES.get(status, status), detail))


class pa_decode_config(ctypes.Structure):
    _fields_ = [("s2_tile", ctypes.c_int), ("num_ctas", ctypes.c_int),
                ("overlap_prologue", ctypes.c_int), ("merge_wait_ns", ctypes.c_int),
                ("wait_limit_ns", ctypes.c_int), ("reserved", ctypes.c_int * 3)]


def build(force: bool = False) -> str:
    """Compile libpa_fp8.so (nvcc, sm_103a) if it is stale."""
    return _build.build(force=force)


def lib():
    """The loaded ctypes library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libpa_fp8.so is not built (%s); run "
                               "fp8_paged_kv_block_gb300.build() first" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        P, i32, i64, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float,
                                ctypes.c_size_t)
        L.pa_status_string.argtypes = [i32]
        L.pa_status_string.restype = ctypes.c_char_p
        L.pa_last_error.argtypes = []
        L.pa_last_error.restype = ctypes.c_char_p
        L.pa_fp8_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32, P,
                                                   ctypes.POINTER(sz)]
        L.pa_fp8_decode_workspace_size.restype = i32
        L.pa_fp8_decode_auto_s2_tile.argtypes = [i32, i32, i32, i64]
        L.pa_fp8_decode_auto_s2_tile.restype = i32
        L.pa_fp8_decode.argtypes = [P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, i64,
                                    i32, i32, f32, P, P, sz, P]
        L.pa_fp8_decode.restype = i32
        L.pa_fp8_cache_scatter.argtypes = [P, P, P, P, P, i32, P, i64, i64, P, i64, i32, i32, i32,
                                           i64, i32, i32, P]
        L.pa_fp8_cache_scatter.restype = i32
        L.pa_fp8_cache_quant_scatter.argtypes = [P, P, i32, P, P, P, i32, P, P, P, i32, i64, i32,
                                                 i32, i64, i32, i32, i32, P]
        L.pa_fp8_cache_quant_scatter.restype = i32
        L.pa_fp8_kv_compress_epilog.argtypes = [P, i64, i32, i64, i32, P, i64, i32, P, i32, i32,
                                                i32, i32, P]
        L.pa_fp8_kv_compress_epilog.restype = i32
        L.pa_fp8_quantize_rows.argtypes = [P, i32, i64, i32, P, P, P]
        L.pa_fp8_quantize_rows.restype = i32
        L.pa_fp8_value_channel_scale.argtypes = [P, i32, P, i32, i64, i32, i32, P, P]
        L.pa_fp8_value_channel_scale.restype = i32
        L.pa_mla_sparse_decode.argtypes = [P, P, P, i64, P, P, P, P, i32, i32, i32, i32, i32, i32,
                                           i64, i32, f32, i32, P, P]
        L.pa_mla_sparse_decode.restype = i32
        L.pa_mla_sparse_decode_kvc.argtypes = [P, P, P, i64, i64, i32, P, P, P, P, i32, i32, i32,
                                               i32, i32, i32, i64, i32, f32, i32, P, P]
        L.pa_mla_sparse_decode_kvc.restype = i32
        L.pa_fp8_qkv_norm_rope_append.argtypes = [
            P, P, P, i32, i64, i64, i64, P, P, i32, f32, P, i32, i64, i32, P, i32, P, P, P, P, P,
            i32, P, P, P, i32, i64, i32, i32, i32, i64, i32, i32, P]
        L.pa_fp8_qkv_norm_rope_append.restype = i32
        L.pa_fp8_tree_decode_workspace_size.argtypes = [i32, i32, i32, i32, i32,
                                                        ctypes.POINTER(sz)]
        L.pa_fp8_tree_decode_workspace_size.restype = i32
        L.pa_fp8_tree_decode.argtypes = [P, P, P, P, P, P, P, P, P, P, i64, P, i32, i32, i32, i32,
                                         i32, i32, i64, i32, i32, f32, P, sz, P]
        L.pa_fp8_tree_decode.restype = i32
        L.pa_tree_verify.argtypes = [P, P, P, P, P, P, i32, i32, i32, P, P, P, P]
        L.pa_tree_verify.restype = i32
        L.pa_fp8_cache_keep_path.argtypes = [P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, i32,
                                             i64, i32, i32, P]
        L.pa_fp8_cache_keep_path.restype = i32
        L.pa_fp8_qkv_norm_mrope_append.argtypes = [
            P, P, P, i32, i64, i64, i64, P, P, i32, f32, P, i32, i64, i32, P, i32, i32, i64, P, P,
            P, P, P, P, i32, P, P, P, i32, i64, i32, i32, i32, i64, i32, i32, P]
        L.pa_fp8_qkv_norm_mrope_append.restype = i32
        L.pa_plan_batch.argtypes = [P, P, P, P, P, P, i32, P, P, P, P, P, i32, i64, i64, i64, i32,
                                    i32, P]
        L.pa_plan_batch.restype = i32
        L.pa_fp8_window_attention_workspace_size.argtypes = [i32, i32, i32, i32,
                                                             ctypes.POINTER(sz)]
        L.pa_fp8_window_attention_workspace_size.restype = i32
        L.pa_fp8_window_attention.argtypes = [P, P, P, P, P, P, P, P, P, P, i32, i64, i32, i32,
                                              i32, i32, i32, i64, i32, i32, i64, i64, f32, P, sz,
                                              P]
        L.pa_fp8_window_attention.restype = i32
        L.pa_token_logprobs.argtypes = [P, i32, i64, P, i32, i64, i32, P, P, P, i32, P, P, P]
        L.pa_token_logprobs.restype = i32
        _lib = L
        return L


def _check(status: int, where: str):
    if status != PA_OK:
        detail = lib().pa_last_error().decode(errors="replace")
        raise PaError(status, where, detail)


def _torch():
    import torch
    return torch


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _need(t, name, dtype=None, contiguous=True):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _fp8_types():
    torch = _torch()
    return (torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2)


def _in_dtype(t):
    torch = _torch()
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError("expected float32 or bfloat16, got %s" % t.dtype)


# --------------------------------------------------------------------------
# Decode attention
# --------------------------------------------------------------------------

_configs = {}


def _config(s2_tile: int, num_ctas: int, overlap_prologue=0, merge_wait_ns=0, wait_limit_ns=0):
    key = (s2_tile, num_ctas, int(overlap_prologue), int(merge_wait_ns), int(wait_limit_ns))
    c = _configs.get(key)
    if c is None:
        c = pa_decode_config()
        c.s2_tile = s2_tile
        c.num_ctas = num_ctas
        c.overlap_prologue = int(overlap_prologue)
        c.merge_wait_ns = int(merge_wait_ns)
        c.wait_limit_ns = int(wait_limit_ns)
        _configs[key] = c
    return c


def auto_s2_tile(S1: int, NQ: int, NKV: int, s2: int) -> int:
    """The s2_tile that s2_tile=0 selects for sequences of capacity s2 (the
    block table's width x block_size): 1024 from 8192 tokens on where at most
    16 query rows share a kv head, else 512 (pa_fp8_decode_auto_s2_tile)."""
    t = lib().pa_fp8_decode_auto_s2_tile(S1, NQ, NKV, s2)
    if t == 0:
        raise ValueError("auto_s2_tile: invalid shape S1=%d NQ=%d NKV=%d s2=%d" % (S1, NQ, NKV, s2))
    return t


def decode_workspace_size(B: int, S1: int, NQ: int, NKV: int, D: int = 128, *,
                          s2_tile: int = 0, num_ctas: int = 0) -> int:
    n = ctypes.c_size_t(0)
    cfg = _config(s2_tile, num_ctas)
    _check(lib().pa_fp8_decode_workspace_size(B, S1, NQ, NKV, D, ctypes.byref(cfg),
                                              ctypes.byref(n)), "pa_fp8_decode_workspace_size")
    return n.value


class DecodeWorkspace:
    """Zero-initialised device scratch for pa_fp8_decode (reusable: every call
    leaves its counters at zero)."""

    def __init__(self, B, S1, NQ, NKV, D=128, *, s2_tile=0, num_ctas=0, device=None):
        torch = _torch()
        self.nbytes = decode_workspace_size(B, S1, NQ, NKV, D, s2_tile=s2_tile, num_ctas=num_ctas)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or "cuda")

    def error_flags(self) -> int:
        """Non-zero if a kernel wait gave up (bitmask of the wait sites)."""
        return int(self.buf[:4].view(_torch().int32).item())

    def clear_error_flags(self) -> None:
        """Zero the error word (on the current stream); the kernel only ever
        sets bits in it."""
        self.buf[:4].zero_()


def decode(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table, kv_act_seqs, out, *,
           S1: int = 1, layout: int = LAYOUT_BSND, s2_tile: int = 0, softmax_scale=None,
           workspace: DecodeWorkspace | None = None, num_ctas: int = 0, stream=None,
           overlap_prologue: int = 0, merge_wait_ns: int = 0, wait_limit_ns: int = 0):
    """Paged FP8 decode attention (in place into ``out``).

    q [B*S1, NQ, D] E4M3 (uint8 or float8_e4m3fn), q_scale float32 [B*S1, NQ],
    k_cache/v_cache E4M3 in ``layout`` ([NB, BS, NKV, D] for BSND,
    [NB, NKV, BS, D] for BNBD), k_scale float32 (cache shape without D),
    v_scale float32 [B, NKV, D], block_table int32 [B, max_blocks],
    kv_act_seqs int32 [B], out bfloat16 [B*S1, NQ, D].
    s2_tile: 0 (automatic, see auto_s2_tile), 128, 256, 512 or 1024.
    overlap_prologue: 1 (or True) lets the kernel's prologue overlap the
    preceding kernel in the stream (that kernel must not write kv_act_seqs,
    block_table, q, q_scale or v_scale); 2 also lets it load the cache blocks
    below each sequence's S1 newest positions early (that kernel must not
    write the cache there); see pa_decode_config.overlap_prologue.
    merge_wait_ns, wait_limit_ns: test and diagnostic knobs, see
    pa_decode_config.
    """
    args, keep = _decode_args(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table,
                              kv_act_seqs, out, S1, layout, s2_tile, softmax_scale, workspace,
                              num_ctas, overlap_prologue, merge_wait_ns, wait_limit_ns, stream)
    _check(lib().pa_fp8_decode(*args, _stream(stream)), "pa_fp8_decode")
    del keep   # (a workspace made here lives until the launch is enqueued)
    return out


def _decode_args(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table, kv_act_seqs, out,
                 S1, layout, s2_tile, softmax_scale, workspace, num_ctas, overlap_prologue,
                 merge_wait_ns, wait_limit_ns, stream, ready=False):
    """pa_fp8_decode's arguments but the stream, validated, and the objects
    they point into."""
    torch = _torch()
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, _fp8_types())
    _need(q_scale, "q_scale", torch.float32)
    _need(k_scale, "k_scale", torch.float32)
    _need(v_scale, "v_scale", torch.float32)
    _need(block_table, "block_table", torch.int32)
    _need(kv_act_seqs, "kv_act_seqs", torch.int32)
    _need(out, "out", torch.bfloat16)
    B = kv_act_seqs.shape[0]
    BS1, NQ, D = q.shape
    if layout == LAYOUT_BSND:
        NB, BS, NKV, _ = k_cache.shape
    else:
        NB, NKV, BS, _ = k_cache.shape
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if workspace is None:
        workspace = _own_workspace(lambda: DecodeWorkspace(B, S1, NQ, NKV, D, s2_tile=s2_tile,
                                                           num_ctas=num_ctas, device=q.device),
                                   stream, ready)
    cfg = _config(s2_tile, num_ctas, overlap_prologue, merge_wait_ns, wait_limit_ns)
    args = (_ptr(q), _ptr(q_scale), _ptr(k_cache), _ptr(k_scale), _ptr(v_cache), _ptr(v_scale),
            _ptr(block_table), _ptr(kv_act_seqs), _ptr(out), B, S1, NQ, NKV, D, BS, NB,
            block_table.shape[1], layout, float(softmax_scale), ctypes.byref(cfg),
            _ptr(workspace.buf), workspace.nbytes)
    keep = (q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table, kv_act_seqs, out,
            workspace, cfg)
    return args, keep


def _own_workspace(make, stream, ready=False):
    """A workspace that the caller did not give, zeroed on the stream that uses
    it and handed back to it. `ready`: the zeroing is waited for, as calls on
    other streams may come (not in a capture, where nothing can be waited for:
    the graph zeroes it)."""
    torch = _torch()
    with torch.cuda.stream(stream):
        workspace = make()
        if ready and not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream().synchronize()
    return workspace


class _Prepared:
    """A library call whose arguments were validated and marshalled once, for
    a loop that makes the same call every step (the buffers' contents may
    change between calls, not their addresses, shapes or dtypes). Runs on the
    stream given when it was made (default: the current stream then), or on
    the stream passed to the call. `scratch` is a workspace that was made for
    this call alone: its memory is not given to others before the streams that
    it ran on are done. (A graph that captured the call does not hold it: the
    callable lives as long as the graph.)"""

    def __init__(self, fn, where, args, keep, stream, scratch=None):
        # a function object of its own that takes ready ctypes values as they are:
        # converting a long argument list anew took longer than a short kernel
        raw = lib()[where]
        raw.restype = fn.restype
        ready = tuple(t(a) if isinstance(a, (int, float)) else a
                      for t, a in zip(fn.argtypes, args))
        self._call = functools.partial(raw, *ready)
        self._where, self._keep = where, keep
        self._stream = _stream(stream)
        self._scratch, self._streams = scratch, {self._stream.value}
        # (torch.cuda.current_device without its checks, which take longer than the rest)
        self._device, self._current = keep[0].device.index, _torch()._C._cuda_getDevice
        self._several = _torch().cuda.device_count() > 1

    def __call__(self, stream=None):
        on = self._stream if stream is None and not self._several else self._checked(stream)
        st = self._call(on)
        if st != PA_OK:
            _check(st, self._where)

    def _checked(self, stream):
        """The handle of the stream to launch on."""
        on = self._stream if stream is None else _stream(stream)
        # a default stream is whichever device's is current: another one's kernel would
        # fault on these buffers (with other streams the launch itself fails)
        if on.value is None and self._several and self._current() != self._device:
            raise ValueError("%s: the buffers are on cuda:%s, the current device is cuda:%d"
                             % (self._where, self._device, self._current()))
        if self._scratch is not None and on.value not in self._streams:
            self._scratch.buf.record_stream(stream)
            self._streams.add(on.value)
        return on


def prepare_decode(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table, kv_act_seqs, out,
                   *, S1: int = 1, layout: int = LAYOUT_BSND, s2_tile: int = 0,
                   softmax_scale=None, workspace: DecodeWorkspace | None = None,
                   num_ctas: int = 0, overlap_prologue: int = 0, stream=None):
    """decode() prepared once: returns a callable that launches the same
    decode on the same buffers (arguments as for decode())."""
    args, keep = _decode_args(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table,
                              kv_act_seqs, out, S1, layout, s2_tile, softmax_scale, workspace,
                              num_ctas, overlap_prologue, 0, 0, stream, ready=True)
    return _Prepared(lib().pa_fp8_decode, "pa_fp8_decode", args, keep, stream,
                     scratch=None if workspace is not None else keep[-2])


# --------------------------------------------------------------------------
# Cache append
# --------------------------------------------------------------------------

def _cache_dims(key_cache, layout):
    if layout == LAYOUT_BNBD:
        NB, H, BS, _ = key_cache.shape
    else:
        NB, BS, H, _ = key_cache.shape
    return NB, H, BS


def _slot_type(slot_mapping):
    torch = _torch()
    if slot_mapping.dtype == torch.int32:
        return INDEX_I32
    if slot_mapping.dtype == torch.int64:
        return INDEX_I64
    raise TypeError("slot_mapping must be int32 or int64")


def cache_scatter(key, value, key_cache, value_cache, slot_mapping, key_scale, key_scale_cache,
                  *, layout: int = LAYOUT_BNBD, stream=None):
    """FP8 K/V + key_scale append by slot_mapping (in place). key_scale may
    have a non-contiguous tail (any 2-D strides)."""
    torch = _torch()
    for t, n in ((key, "key"), (value, "value"), (key_cache, "key_cache"),
                 (value_cache, "value_cache")):
        _need(t, n, _fp8_types())
    _need(slot_mapping, "slot_mapping", (torch.int32, torch.int64))
    _need(key_scale, "key_scale", torch.float32, contiguous=False)
    _need(key_scale_cache, "key_scale_cache", torch.float32)
    T, H, Dk = key.shape
    Dv = value.shape[2]
    NB, _, BS = _cache_dims(key_cache, layout)
    st = lib().pa_fp8_cache_scatter(_ptr(key), _ptr(value), _ptr(key_cache), _ptr(value_cache),
                                    _ptr(slot_mapping), _slot_type(slot_mapping), _ptr(key_scale),
                                    key_scale.stride(0), key_scale.stride(1),
                                    _ptr(key_scale_cache), T, H, Dk, Dv, NB, BS, layout,
                                    _stream(stream))
    _check(st, "pa_fp8_cache_scatter")


def cache_quant_scatter(key, value, key_cache, value_cache, slot_mapping, key_scale_cache,
                        v_scale, token_batch, *, layout: int = LAYOUT_BNBD,
                        overlap_prologue: bool = False, stream=None):
    """BF16/FP32 K/V quantised to E4M3 on append (in place): key per
    (token, head) with scale amax/448 stored to key_scale_cache, value against
    v_scale[token_batch[i]]. overlap_prologue=True launches it with
    programmatic stream serialisation: the inputs are read while the preceding
    kernel may still run (it must not write them), the caches are written after
    it has completed."""
    args, keep = _quant_scatter_args(key, value, key_cache, value_cache, slot_mapping,
                                     key_scale_cache, v_scale, token_batch, layout,
                                     overlap_prologue)
    _check(lib().pa_fp8_cache_quant_scatter(*args, _stream(stream)), "pa_fp8_cache_quant_scatter")
    del keep


def _quant_scatter_args(key, value, key_cache, value_cache, slot_mapping, key_scale_cache,
                        v_scale, token_batch, layout, overlap_prologue):
    torch = _torch()
    _need(key, "key", (torch.float32, torch.bfloat16))
    _need(value, "value", (key.dtype,))
    for t, n in ((key_cache, "key_cache"), (value_cache, "value_cache")):
        _need(t, n, _fp8_types())
    _need(slot_mapping, "slot_mapping", (torch.int32, torch.int64))
    _need(key_scale_cache, "key_scale_cache", torch.float32)
    _need(v_scale, "v_scale", torch.float32)
    _need(token_batch, "token_batch", torch.int32)
    T, H, D = key.shape
    NB, _, BS = _cache_dims(key_cache, layout)
    args = (_ptr(key), _ptr(value), _in_dtype(key), _ptr(key_cache), _ptr(value_cache),
            _ptr(slot_mapping), _slot_type(slot_mapping), _ptr(key_scale_cache), _ptr(v_scale),
            _ptr(token_batch), v_scale.shape[0], T, H, D, NB, BS, layout,
            int(bool(overlap_prologue)))
    keep = (key, value, key_cache, value_cache, slot_mapping, key_scale_cache, v_scale,
            token_batch)
    return args, keep


def prepare_cache_quant_scatter(key, value, key_cache, value_cache, slot_mapping,
                                key_scale_cache, v_scale, token_batch, *,
                                layout: int = LAYOUT_BNBD, overlap_prologue: bool = False,
                                stream=None):
    """cache_quant_scatter() prepared once: returns a callable that launches the
    same append on the same buffers."""
    args, keep = _quant_scatter_args(key, value, key_cache, value_cache, slot_mapping,
                                     key_scale_cache, v_scale, token_batch, layout,
                                     overlap_prologue)
    return _Prepared(lib().pa_fp8_cache_quant_scatter, "pa_fp8_cache_quant_scatter", args, keep,
                     stream)


def kv_compress_epilog(cache, x, slot_mapping, *, quant_group_size: int = 64, quant_mode: int = 1,
                       round_scale: bool = True, stream=None):
    """KV compress epilog (modes 0 and 1), in place: cache uint8
    [block_num, block_size, 1, head_dim] (blocks may be strided), x bfloat16
    [bs, d], slot_mapping int32/int64 [bs]. Each row is written as the rope
    part (last 64 values) in BF16, the rest in E4M3 groups of 64, then the
    group scales (BF16 in mode 0, E8M0 in mode 1)."""
    torch = _torch()
    _need(cache, "cache", (torch.uint8,), contiguous=False)
    _need(x, "x", (torch.bfloat16,))
    _need(slot_mapping, "slot_mapping", (torch.int32, torch.int64))
    if cache.dim() != 4 or cache.shape[2] != 1:
        raise ValueError("cache must be [block_num, block_size, 1, head_dim]")
    NB, BS, _, HD = cache.shape
    if cache.stride(3) != 1 or cache.stride(1) != HD:
        raise ValueError("cache rows must be contiguous within a block")
    bs, d = x.shape
    st = lib().pa_fp8_kv_compress_epilog(_ptr(cache), NB, BS, cache.stride(0), HD, _ptr(x), bs, d,
                                         _ptr(slot_mapping), _slot_type(slot_mapping),
                                         quant_group_size, quant_mode, int(bool(round_scale)),
                                         _stream(stream))
    _check(st, "pa_fp8_kv_compress_epilog")


def quantize_rows(x, codes, scale, *, stream=None):
    """Per-row E4M3 quantiser: x [..., D] float32/bfloat16 -> codes [..., D],
    dequant scale [...] = amax / 448."""
    torch = _torch()
    _need(x, "x", (torch.float32, torch.bfloat16))
    _need(codes, "codes", _fp8_types())
    _need(scale, "scale", torch.float32)
    D = x.shape[-1]
    rows = x.numel() // D
    st = lib().pa_fp8_quantize_rows(_ptr(x), _in_dtype(x), rows, D, _ptr(codes), _ptr(scale),
                                    _stream(stream))
    _check(st, "pa_fp8_quantize_rows")


def value_channel_scale(v, cu_seqlens, v_scale, *, stream=None):
    """v [Ttot, H, D] float32/bfloat16, cu_seqlens int64 [B+1] (device) ->
    v_scale [B, H, D] = per-channel max |v| over each sequence / 448."""
    torch = _torch()
    _need(v, "v", (torch.float32, torch.bfloat16))
    _need(cu_seqlens, "cu_seqlens", torch.int64)
    _need(v_scale, "v_scale", torch.float32)
    T, H, D = v.shape
    B = cu_seqlens.shape[0] - 1
    st = lib().pa_fp8_value_channel_scale(_ptr(v), _in_dtype(v), _ptr(cu_seqlens), B, T, H, D,
                                          _ptr(v_scale), _stream(stream))
    _check(st, "pa_fp8_value_channel_scale")


# --------------------------------------------------------------------------
# Speculative decode step: a tree of drafted tokens for each sequence
# --------------------------------------------------------------------------

def _one_device(**tensors):
    """Every tensor on the current device: the launch goes to that device's
    stream, and a pointer of another device would fault there."""
    torch = _torch()
    cur = torch.cuda.current_device()
    for n, t in tensors.items():
        if t is not None and t.device.index != cur:
            raise ValueError("%s is on %s, the current device is cuda:%d" % (n, t.device, cur))


def _shape(t, name, *want):
    if tuple(t.shape) != tuple(want):
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(want)))


def _norm_rope_args(q, k, v, q_weight, k_weight, cos_sin, positions, q_codes, q_scale, key_cache,
                    value_cache, slot_mapping, key_scale_cache, v_scale, token_batch, eps,
                    interleaved, layout, pair_axis=None):
    """pa_fp8_qkv_norm_rope_append's arguments but the stream, or with pair_axis
    pa_fp8_qkv_norm_mrope_append's, and the objects they point into."""
    torch = _torch()
    floats = (torch.float32, torch.bfloat16)
    e4m3 = (torch.uint8, torch.float8_e4m3fn)            # what is written, whatever holds it
    _need(q, "q", floats, contiguous=False)
    for t, n in ((k, "k"), (v, "v")):
        _need(t, n, (q.dtype,), contiguous=False)
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        if t.dim() != 3 or t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]):
            raise ValueError("%s must be [tokens, heads, head_size] with contiguous heads" % n)
    T, NQ, D = q.shape
    NKV = k.shape[1]
    _shape(k, "k", T, NKV, D)
    _shape(v, "v", T, NKV, D)
    wdt = torch.float32
    for t, n in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if t is not None:
            _need(t, n, floats)
            _shape(t, n, D)
            wdt = t.dtype
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise TypeError("q_weight and k_weight must have one dtype")
    rd = max_pos = pos_type = 0
    if cos_sin is not None:
        _need(cos_sin, "cos_sin", torch.float32)
        max_pos, rd = cos_sin.shape
        if positions is None:
            raise ValueError("cos_sin needs positions")
    axes = ()
    if pair_axis is not None:
        pair_axis = [int(a) for a in pair_axis]
        if len(pair_axis) != rd // 2:
            raise ValueError("pair_axis must name an axis for each of the %d pairs" % (rd // 2))
        _need(positions, "positions", (torch.int32, torch.int64), contiguous=False)
        if positions.dim() != 2:
            raise ValueError("positions must be [axes, tokens]")
        A = positions.shape[0]
        _shape(positions, "positions", A, T)
        if T > 0 and ((T > 1 and positions.stride(1) != 1) or (A > 1 and positions.stride(0) < T)):
            raise ValueError("positions must have contiguous axes that do not overlap")
        if any(not 0 <= a < A for a in pair_axis):
            raise ValueError("pair_axis must be below the number of axes, %d" % A)
        step = positions.stride(0) if A > 1 and T > 0 else T
        host = (ctypes.c_uint8 * max(1, len(pair_axis)))(*pair_axis)
        axes = (A, step, ctypes.addressof(host))
        pair_axis = host
    elif positions is not None:
        _need(positions, "positions", (torch.int32, torch.int64))
        _shape(positions, "positions", T)
    if positions is not None:
        pos_type = INDEX_I64 if positions.dtype == torch.int64 else INDEX_I32
    _need(q_codes, "q_codes", e4m3)
    _shape(q_codes, "q_codes", T, NQ, D)
    _need(q_scale, "q_scale", torch.float32)
    _shape(q_scale, "q_scale", T, NQ)
    for t, n in ((key_cache, "key_cache"), (value_cache, "value_cache")):
        _need(t, n, e4m3)
    _need(slot_mapping, "slot_mapping", (torch.int32, torch.int64))
    _shape(slot_mapping, "slot_mapping", T)
    _need(key_scale_cache, "key_scale_cache", torch.float32)
    _need(v_scale, "v_scale", torch.float32)
    _need(token_batch, "token_batch", torch.int32)
    _shape(token_batch, "token_batch", T)
    NB, H, BS = _cache_dims(key_cache, layout)
    cache = (NB, BS, H) if layout == LAYOUT_BSND else (NB, H, BS)
    _shape(key_cache, "key_cache", *cache, D)
    _shape(value_cache, "value_cache", *cache, D)
    if key_scale_cache.numel() != NB * BS * H or H != NKV:
        raise ValueError("key_scale_cache and the caches must have one scale a row and k's heads")
    _shape(v_scale, "v_scale", v_scale.shape[0], NKV, D)
    _one_device(q=q, k=k, v=v, q_weight=q_weight, k_weight=k_weight, cos_sin=cos_sin,
                positions=positions, q_codes=q_codes, q_scale=q_scale, key_cache=key_cache,
                value_cache=value_cache, slot_mapping=slot_mapping,
                key_scale_cache=key_scale_cache, v_scale=v_scale, token_batch=token_batch)
    step = [t.stride(0) if T > 1 else 0 for t in (q, k, v)]     # (of one token: any)
    args = (_ptr(q), _ptr(k), _ptr(v), _in_dtype(q), *step,
            _ptr(q_weight), _ptr(k_weight), DTYPE_BF16 if wdt == torch.bfloat16 else DTYPE_F32,
            float(eps), _ptr(cos_sin), rd, max_pos, int(bool(interleaved)), _ptr(positions),
            pos_type, *axes, _ptr(q_codes), _ptr(q_scale), _ptr(key_cache), _ptr(value_cache),
            _ptr(slot_mapping), _slot_type(slot_mapping), _ptr(key_scale_cache), _ptr(v_scale),
            _ptr(token_batch), v_scale.shape[0], T, NQ, NKV, D, NB, BS, layout)
    keep = (q, k, v, q_weight, k_weight, cos_sin, positions, q_codes, q_scale, key_cache,
            value_cache, slot_mapping, key_scale_cache, v_scale, token_batch, pair_axis)
    return args, keep


def qkv_norm_rope_append(q, k, v, q_weight, k_weight, cos_sin, positions, q_codes, q_scale,
                         key_cache, value_cache, slot_mapping, key_scale_cache, v_scale,
                         token_batch, *, eps: float = 1e-5, interleaved: bool = False,
                         layout: int = LAYOUT_BNBD, stream=None):
    """Per-head RMSNorm and rotation of q and k, E4M3 quantisation, and the
    append of k and v, in one pass (in place into q_codes, q_scale and the
    caches).

    q [T, NQ, D], k and v [T, NKV, D] float32 or bfloat16, tokens any stride
    apart (views of one projection's output), D 64, 128 or 256; q_weight,
    k_weight [D] float32 or bfloat16 or None (no norm); cos_sin float32
    [max_position, rotary_dim], cosines then sines, or None (no rotation);
    positions int32/int64 [T]; q_codes E4M3 [T, NQ, D], q_scale float32
    [T, NQ]; the caches, slot_mapping, v_scale and token_batch as in
    cache_quant_scatter. interleaved: channels (2i, 2i+1) are a pair instead
    of (i, i + rotary_dim/2)."""
    args, keep = _norm_rope_args(q, k, v, q_weight, k_weight, cos_sin, positions, q_codes,
                                 q_scale, key_cache, value_cache, slot_mapping, key_scale_cache,
                                 v_scale, token_batch, eps, interleaved, layout)
    _check(lib().pa_fp8_qkv_norm_rope_append(*args, _stream(stream)),
           "pa_fp8_qkv_norm_rope_append")
    del keep


def prepare_qkv_norm_rope_append(q, k, v, q_weight, k_weight, cos_sin, positions, q_codes,
                                 q_scale, key_cache, value_cache, slot_mapping, key_scale_cache,
                                 v_scale, token_batch, *, eps: float = 1e-5,
                                 interleaved: bool = False, layout: int = LAYOUT_BNBD,
                                 stream=None):
    """qkv_norm_rope_append() prepared once: returns a callable that launches
    the same call on the same buffers."""
    args, keep = _norm_rope_args(q, k, v, q_weight, k_weight, cos_sin, positions, q_codes,
                                 q_scale, key_cache, value_cache, slot_mapping, key_scale_cache,
                                 v_scale, token_batch, eps, interleaved, layout)
    return _Prepared(lib().pa_fp8_qkv_norm_rope_append, "pa_fp8_qkv_norm_rope_append", args, keep,
                     stream)


def qkv_norm_mrope_append(q, k, v, q_weight, k_weight, cos_sin, positions, q_codes, q_scale,
                          key_cache, value_cache, slot_mapping, key_scale_cache, v_scale,
                          token_batch, *, pair_axis, eps: float = 1e-5, interleaved: bool = False,
                          layout: int = LAYOUT_BNBD, stream=None):
    """qkv_norm_rope_append() for tokens with several positions, as the time,
    height and width of an image's or a video's patches: positions int32/int64
    [axes, T] (up to 4 axes, each contiguous), and pair i of the rotated channels
    takes its angle from positions[pair_axis[i]]. pair_axis: a sequence of
    rotary_dim/2 ints, such as [0] * 16 + [1] * 24 + [2] * 24 for sections of
    axes one behind another. Everything else as there."""
    if pair_axis is None or cos_sin is None:
        raise TypeError("qkv_norm_mrope_append needs pair_axis and cos_sin")
    args, keep = _norm_rope_args(q, k, v, q_weight, k_weight, cos_sin, positions, q_codes,
                                 q_scale, key_cache, value_cache, slot_mapping, key_scale_cache,
                                 v_scale, token_batch, eps, interleaved, layout, pair_axis)
    _check(lib().pa_fp8_qkv_norm_mrope_append(*args, _stream(stream)),
           "pa_fp8_qkv_norm_mrope_append")
    del keep


def prepare_qkv_norm_mrope_append(q, k, v, q_weight, k_weight, cos_sin, positions, q_codes,
                                  q_scale, key_cache, value_cache, slot_mapping, key_scale_cache,
                                  v_scale, token_batch, *, pair_axis, eps: float = 1e-5,
                                  interleaved: bool = False, layout: int = LAYOUT_BNBD,
                                  stream=None):
    """qkv_norm_mrope_append() prepared once: returns a callable that launches
    the same call on the same buffers."""
    if pair_axis is None or cos_sin is None:
        raise TypeError("qkv_norm_mrope_append needs pair_axis and cos_sin")
    args, keep = _norm_rope_args(q, k, v, q_weight, k_weight, cos_sin, positions, q_codes,
                                 q_scale, key_cache, value_cache, slot_mapping, key_scale_cache,
                                 v_scale, token_batch, eps, interleaved, layout, pair_axis)
    return _Prepared(lib().pa_fp8_qkv_norm_mrope_append, "pa_fp8_qkv_norm_mrope_append", args,
                     keep, stream)


def tree_decode_workspace_size(B: int, S1: int, NQ: int, NKV: int, D: int = 128) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().pa_fp8_tree_decode_workspace_size(B, S1, NQ, NKV, D, ctypes.byref(n)),
           "pa_fp8_tree_decode_workspace_size")
    return n.value


class TreeWorkspace:
    """Zero-initialised device scratch for tree_decode (reusable: every call
    leaves what must be zero at zero). Calls that may run at the same time,
    replays of two captured graphs among them, need one each."""

    def __init__(self, B, S1, NQ, NKV, D=128, *, device=None):
        torch = _torch()
        self.nbytes = tree_decode_workspace_size(B, S1, NQ, NKV, D)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or "cuda")

    def error_flags(self) -> int:
        """Non-zero if a kernel wait gave up (bitmask of the wait sites)."""
        return int(self.buf[:4].view(_torch().int32).item())

    def clear_error_flags(self) -> None:
        """Zero the error word (on the current stream)."""
        self.buf[:4].zero_()


def _tree_args(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table, kv_act_seqs,
               tree_mask, out, S1, tree_len, layout, softmax_scale, workspace, stream,
               ready=False):
    torch = _torch()
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, (torch.uint8, torch.float8_e4m3fn))
    for t, n in ((q_scale, "q_scale"), (k_scale, "k_scale"), (v_scale, "v_scale")):
        _need(t, n, torch.float32)
    _need(block_table, "block_table", torch.int32)
    _need(kv_act_seqs, "kv_act_seqs", torch.int32)
    _need(tree_mask, "tree_mask", (torch.bool, torch.uint8), contiguous=False)
    _need(out, "out", torch.bfloat16)
    B = kv_act_seqs.shape[0]
    BS1, NQ, D = q.shape
    if BS1 != B * S1:
        raise ValueError("q has %d tokens, expected B * S1 = %d" % (BS1, B * S1))
    NB, NKV, BS = _cache_dims(k_cache, layout)
    cache = (NB, BS, NKV) if layout == LAYOUT_BSND else (NB, NKV, BS)
    _shape(k_cache, "k_cache", *cache, D)
    _shape(v_cache, "v_cache", *cache, D)
    if k_scale.numel() != NB * BS * NKV:
        raise ValueError("k_scale must have one scale a cache row")
    _shape(q_scale, "q_scale", BS1, NQ)
    _shape(v_scale, "v_scale", B, NKV, D)
    _shape(out, "out", BS1, NQ, D)
    _shape(kv_act_seqs, "kv_act_seqs", B)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks]")
    if tree_mask.dim() == 2:
        tree_mask = tree_mask.unsqueeze(0).expand(B, S1, S1) if tuple(tree_mask.shape) == (S1, S1) \
            else tree_mask
    _shape(tree_mask, "tree_mask", B, S1, S1)
    if B > 0 and ((S1 > 1 and tree_mask.stride(2) != 1) or (S1 > 1 and tree_mask.stride(1) != S1)):
        raise ValueError("tree_mask must have contiguous rows within a sequence")
    if tree_len is not None:
        _need(tree_len, "tree_len", torch.int32)
        _shape(tree_len, "tree_len", B)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if workspace is None:
        workspace = _own_workspace(lambda: TreeWorkspace(B, S1, NQ, NKV, D, device=q.device),
                                   stream, ready)
    _one_device(q=q, q_scale=q_scale, k_cache=k_cache, k_scale=k_scale, v_cache=v_cache,
                v_scale=v_scale, block_table=block_table, kv_act_seqs=kv_act_seqs,
                tree_mask=tree_mask, tree_len=tree_len, out=out, workspace=workspace.buf)
    args = (_ptr(q), _ptr(q_scale), _ptr(k_cache), _ptr(k_scale), _ptr(v_cache), _ptr(v_scale),
            _ptr(block_table), _ptr(kv_act_seqs), _ptr(tree_len), _ptr(tree_mask),
            tree_mask.stride(0), _ptr(out), B, S1, NQ, NKV, D, BS, NB, block_table.shape[1],
            layout, float(softmax_scale), _ptr(workspace.buf), workspace.nbytes)
    keep = (q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table, kv_act_seqs, tree_len,
            tree_mask, out, workspace)
    return args, keep


def tree_decode(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table, kv_act_seqs,
                tree_mask, out, *, S1: int, tree_len=None, layout: int = LAYOUT_BSND,
                softmax_scale=None, workspace: TreeWorkspace | None = None, stream=None):
    """Attention of a tree of drafted tokens over the paged FP8 cache (in place
    into ``out``): each of a sequence's tree_len[b] <= S1 drafted tokens, whose
    K/V are the sequence's last positions, attends to everything before them
    and to the drafted tokens its row of tree_mask names.

    tree_mask bool or uint8 [B, S1, S1], or [S1, S1] for all sequences;
    tree_len int32 [B] or None (all S1); the other arguments as in decode().
    Rows at and behind tree_len[b], and rows that see nothing, get zeros."""
    args, keep = _tree_args(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table,
                            kv_act_seqs, tree_mask, out, S1, tree_len, layout, softmax_scale,
                            workspace, stream)
    _check(lib().pa_fp8_tree_decode(*args, _stream(stream)), "pa_fp8_tree_decode")
    del keep   # (a workspace made here lives until the launch is enqueued)
    return out


def prepare_tree_decode(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table, kv_act_seqs,
                        tree_mask, out, *, S1: int, tree_len=None, layout: int = LAYOUT_BSND,
                        softmax_scale=None, workspace: TreeWorkspace | None = None, stream=None):
    """tree_decode() prepared once: returns a callable that launches the same
    call on the same buffers."""
    args, keep = _tree_args(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table,
                            kv_act_seqs, tree_mask, out, S1, tree_len, layout, softmax_scale,
                            workspace, stream, ready=True)
    return _Prepared(lib().pa_fp8_tree_decode, "pa_fp8_tree_decode", args, keep, stream,
                     scratch=None if workspace is not None else keep[-1])


def _verify_args(target_probs, draft_probs, draft_tokens, parents, uniforms, accepted, path,
                 tokens, tree_len):
    torch = _torch()
    _need(target_probs, "target_probs", torch.float32)
    if target_probs.dim() != 3:
        raise ValueError("target_probs must be [B, S1, V]")
    B, S1, V = target_probs.shape
    if draft_probs is not None:
        _need(draft_probs, "draft_probs", torch.float32)
        _shape(draft_probs, "draft_probs", B, S1, V)
    for t, n in ((draft_tokens, "draft_tokens"), (parents, "parents"), (path, "path"),
                 (tokens, "tokens")):
        _need(t, n, torch.int32)
        _shape(t, n, B, S1)
    _need(uniforms, "uniforms", torch.float32)
    _shape(uniforms, "uniforms", B, S1)
    _need(accepted, "accepted", torch.int32)
    _shape(accepted, "accepted", B)
    if tree_len is not None:
        _need(tree_len, "tree_len", torch.int32)
        _shape(tree_len, "tree_len", B)
    _one_device(target_probs=target_probs, draft_probs=draft_probs, draft_tokens=draft_tokens,
                parents=parents, uniforms=uniforms, accepted=accepted, path=path, tokens=tokens,
                tree_len=tree_len)
    args = (_ptr(target_probs), _ptr(draft_probs), _ptr(draft_tokens), _ptr(parents),
            _ptr(uniforms), _ptr(tree_len), B, S1, V, _ptr(accepted), _ptr(path), _ptr(tokens))
    keep = (target_probs, draft_probs, draft_tokens, parents, uniforms, accepted, path, tokens,
            tree_len)
    return args, keep


def tree_verify(target_probs, draft_probs, draft_tokens, parents, uniforms, accepted, path,
                tokens, *, tree_len=None, stream=None):
    """Verification of drafted tokens against the target's probabilities from
    given random numbers (in place into accepted, path and tokens).

    target_probs float32 [B, S1, V], row s the target's distribution after node
    s; draft_probs float32 [B, S1, V], row s the distribution node s's children
    were drawn from, or None (drafts not drawn at random); draft_tokens, parents
    int32 [B, S1]; uniforms float32 [B, S1] in [0, 1): entry s tests node s,
    entry 0 draws the last token. accepted int32 [B]: nodes on the accepted
    branch, node 0 counted; path int32 [B, S1]: those nodes; tokens int32
    [B, S1]: the new tokens, accepted[b] of them, the last one drawn from what
    is left of the target's distribution; -1 behind."""
    args, keep = _verify_args(target_probs, draft_probs, draft_tokens, parents, uniforms,
                              accepted, path, tokens, tree_len)
    _check(lib().pa_tree_verify(*args, _stream(stream)), "pa_tree_verify")
    del keep


def prepare_tree_verify(target_probs, draft_probs, draft_tokens, parents, uniforms, accepted,
                        path, tokens, *, tree_len=None, stream=None):
    """tree_verify() prepared once: returns a callable that launches the same
    call on the same buffers."""
    args, keep = _verify_args(target_probs, draft_probs, draft_tokens, parents, uniforms,
                              accepted, path, tokens, tree_len)
    return _Prepared(lib().pa_tree_verify, "pa_tree_verify", args, keep, stream)


def _keep_args(key_cache, value_cache, key_scale_cache, block_table, kv_act_seqs, path, accepted,
               new_act_seqs, tree_len, layout):
    torch = _torch()
    for t, n in ((key_cache, "key_cache"), (value_cache, "value_cache")):
        _need(t, n, _fp8_types())
    _need(key_scale_cache, "key_scale_cache", torch.float32)
    for t, n in ((block_table, "block_table"), (kv_act_seqs, "kv_act_seqs"), (path, "path"),
                 (accepted, "accepted"), (new_act_seqs, "new_act_seqs")):
        _need(t, n, torch.int32)
    if layout is None:
        raise TypeError("cache_keep_path needs layout=: no other argument has the caches' heads "
                        "or block size to hold against their shape")
    if path.dim() != 2 or block_table.dim() != 2:
        raise ValueError("path must be [B, S1] and block_table [B, max_blocks]")
    B, S1 = path.shape
    if block_table.shape[0] != B:
        raise ValueError("block_table must have one row a sequence")
    for t, n in ((kv_act_seqs, "kv_act_seqs"), (accepted, "accepted"),
                 (new_act_seqs, "new_act_seqs")):
        _shape(t, n, B)
    if tree_len is not None:
        _need(tree_len, "tree_len", torch.int32)
        _shape(tree_len, "tree_len", B)
    NB, H, BS = _cache_dims(key_cache, layout)
    _shape(value_cache, "value_cache", *key_cache.shape)
    if key_scale_cache.numel() != NB * BS * H:
        raise ValueError("key_scale_cache must have one scale a cache row")
    _one_device(key_cache=key_cache, value_cache=value_cache, key_scale_cache=key_scale_cache,
                block_table=block_table, kv_act_seqs=kv_act_seqs, path=path, accepted=accepted,
                new_act_seqs=new_act_seqs, tree_len=tree_len)
    args = (_ptr(key_cache), _ptr(value_cache), _ptr(key_scale_cache), _ptr(block_table),
            _ptr(kv_act_seqs), _ptr(tree_len), _ptr(path), _ptr(accepted), _ptr(new_act_seqs), B,
            S1, H, key_cache.shape[3], BS, NB, block_table.shape[1], layout)
    keep = (key_cache, value_cache, key_scale_cache, block_table, kv_act_seqs, tree_len, path,
            accepted, new_act_seqs)
    return args, keep


def cache_keep_path(key_cache, value_cache, key_scale_cache, block_table, kv_act_seqs, path,
                    accepted, new_act_seqs, *, tree_len=None, layout: int | None = None,
                    stream=None):
    """The accepted branch kept in the cache, in place: the K/V codes and key
    scales of the drafted nodes path[b][:accepted[b]] (tree_verify's, strictly
    increasing) move to the first drafted positions, and new_act_seqs int32 [B]
    (another tensor than kv_act_seqs) becomes the length that leaves. layout has
    to be given, the one that tree_decode reads the caches in: no default, as the
    cache's shape alone does not tell heads from positions."""
    args, keep = _keep_args(key_cache, value_cache, key_scale_cache, block_table, kv_act_seqs,
                            path, accepted, new_act_seqs, tree_len, layout)
    _check(lib().pa_fp8_cache_keep_path(*args, _stream(stream)), "pa_fp8_cache_keep_path")
    del keep


def prepare_cache_keep_path(key_cache, value_cache, key_scale_cache, block_table, kv_act_seqs,
                            path, accepted, new_act_seqs, *, tree_len=None,
                            layout: int | None = None, stream=None):
    """cache_keep_path() prepared once: returns a callable that launches the
    same call on the same buffers."""
    args, keep = _keep_args(key_cache, value_cache, key_scale_cache, block_table, kv_act_seqs,
                            path, accepted, new_act_seqs, tree_len, layout)
    return _Prepared(lib().pa_fp8_cache_keep_path, "pa_fp8_cache_keep_path", args, keep, stream)


# --------------------------------------------------------------------------
# A ragged serving step
# --------------------------------------------------------------------------

def _plan_args(kv_act_seqs, new_lens, pool, pool_head, block_table, slot_mapping, positions,
               token_batch, cu_tokens, new_act_seqs, new_pool_head, num_blocks, block_size):
    torch = _torch()
    for t, n in ((kv_act_seqs, "kv_act_seqs"), (new_lens, "new_lens"), (pool, "pool"),
                 (pool_head, "pool_head"), (block_table, "block_table"),
                 (positions, "positions"), (token_batch, "token_batch"),
                 (cu_tokens, "cu_tokens"), (new_act_seqs, "new_act_seqs"),
                 (new_pool_head, "new_pool_head")):
        _need(t, n, torch.int32)
    _need(slot_mapping, "slot_mapping", (torch.int32, torch.int64))
    if block_table.dim() != 2 or slot_mapping.dim() != 1 or pool.dim() != 1:
        raise ValueError("block_table must be [B, max_blocks], slot_mapping [tokens] and pool "
                         "[blocks]")
    B, T = block_table.shape[0], slot_mapping.shape[0]
    for t, n in ((kv_act_seqs, "kv_act_seqs"), (new_lens, "new_lens"),
                 (new_act_seqs, "new_act_seqs")):
        _shape(t, n, B)
    for t, n in ((positions, "positions"), (token_batch, "token_batch")):
        _shape(t, n, T)
    _shape(cu_tokens, "cu_tokens", B + 1)
    for t, n in ((pool_head, "pool_head"), (new_pool_head, "new_pool_head")):
        _shape(t, n, 1)
    _one_device(kv_act_seqs=kv_act_seqs, new_lens=new_lens, pool=pool, pool_head=pool_head,
                block_table=block_table, slot_mapping=slot_mapping, positions=positions,
                token_batch=token_batch, cu_tokens=cu_tokens, new_act_seqs=new_act_seqs,
                new_pool_head=new_pool_head)
    args = (_ptr(kv_act_seqs), _ptr(new_lens), _ptr(pool), _ptr(pool_head), _ptr(block_table),
            _ptr(slot_mapping), _slot_type(slot_mapping), _ptr(positions), _ptr(token_batch),
            _ptr(cu_tokens), _ptr(new_act_seqs), _ptr(new_pool_head), B, T, pool.shape[0],
            int(num_blocks), int(block_size), block_table.shape[1])
    keep = (kv_act_seqs, new_lens, pool, pool_head, block_table, slot_mapping, positions,
            token_batch, cu_tokens, new_act_seqs, new_pool_head)
    return args, keep


def plan_batch(kv_act_seqs, new_lens, pool, pool_head, block_table, slot_mapping, positions,
               token_batch, cu_tokens, new_act_seqs, new_pool_head, *, num_blocks: int,
               block_size: int = 128, stream=None):
    """Where a step's new tokens go, from the requests' lengths, on the device
    (in place into block_table and the tensors behind it).

    kv_act_seqs, new_lens int32 [B]: positions in the cache and new tokens of
    each request; pool int32 [blocks]: ids of blocks, those from pool_head[0] on
    free; block_table int32 [B, max_blocks]: gets the new blocks' entries.
    slot_mapping int32/int64, positions and token_batch int32 [T]: of the tokens
    that the requests bring, one request behind another, -1, 0 and 0 behind;
    cu_tokens int32 [B + 1]: the requests' first rows; new_act_seqs int32 [B];
    pool_head, new_pool_head int32 [1]. num_blocks: of the cache.

    A request that does not fit its row of the block table, the T rows or what is
    left of the pool is refused: its slots are -1 and its length stays. The
    outputs overlap neither an input nor one another."""
    args, keep = _plan_args(kv_act_seqs, new_lens, pool, pool_head, block_table, slot_mapping,
                            positions, token_batch, cu_tokens, new_act_seqs, new_pool_head,
                            num_blocks, block_size)
    _check(lib().pa_plan_batch(*args, _stream(stream)), "pa_plan_batch")
    del keep


def prepare_plan_batch(kv_act_seqs, new_lens, pool, pool_head, block_table, slot_mapping,
                       positions, token_batch, cu_tokens, new_act_seqs, new_pool_head, *,
                       num_blocks: int, block_size: int = 128, stream=None):
    """plan_batch() prepared once: returns a callable that launches the same call
    on the same buffers."""
    args, keep = _plan_args(kv_act_seqs, new_lens, pool, pool_head, block_table, slot_mapping,
                            positions, token_batch, cu_tokens, new_act_seqs, new_pool_head,
                            num_blocks, block_size)
    return _Prepared(lib().pa_plan_batch, "pa_plan_batch", args, keep, stream)


def window_attention_workspace_size(max_tokens: int, NQ: int, NKV: int, D: int = 128) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().pa_fp8_window_attention_workspace_size(max_tokens, NQ, NKV, D, ctypes.byref(n)),
           "pa_fp8_window_attention_workspace_size")
    return n.value


class WindowWorkspace:
    """Zero-initialised device scratch for window_attention (reusable: every call
    leaves what must be zero at zero), for calls of at most max_tokens tokens a
    sequence. Calls that may run at the same time, replays of two captured graphs
    among them, need one each."""

    def __init__(self, max_tokens, NQ, NKV, D=128, *, device=None):
        torch = _torch()
        self.nbytes = window_attention_workspace_size(max_tokens, NQ, NKV, D)
        self.buf = torch.zeros(self.nbytes, dtype=torch.uint8, device=device or "cuda")

    def error_flags(self) -> int:
        """Non-zero if a kernel wait gave up (bitmask of the wait sites) or cu_tokens
        decreased (bit 16384)."""
        return int(self.buf[:4].view(_torch().int32).item())

    def clear_error_flags(self) -> None:
        """Zero the error word (on the current stream)."""
        self.buf[:4].zero_()


def _window_args(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table, kv_act_seqs,
                 cu_tokens, out, window, sinks, max_tokens, layout, softmax_scale, workspace,
                 stream, ready=False):
    torch = _torch()
    for t, n in ((q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, (torch.uint8, torch.float8_e4m3fn))
    for t, n in ((q_scale, "q_scale"), (k_scale, "k_scale"), (v_scale, "v_scale")):
        _need(t, n, torch.float32)
    for t, n in ((block_table, "block_table"), (kv_act_seqs, "kv_act_seqs"),
                 (cu_tokens, "cu_tokens")):
        _need(t, n, torch.int32)
    _need(out, "out", torch.bfloat16)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, head_size]")
    T, NQ, D = q.shape
    B = kv_act_seqs.shape[0]
    NB, NKV, BS = _cache_dims(k_cache, layout)
    cache = (NB, BS, NKV) if layout == LAYOUT_BSND else (NB, NKV, BS)
    _shape(k_cache, "k_cache", *cache, D)
    _shape(v_cache, "v_cache", *cache, D)
    if k_scale.numel() != NB * BS * NKV:
        raise ValueError("k_scale must have one scale a cache row")
    _shape(q_scale, "q_scale", T, NQ)
    _shape(v_scale, "v_scale", B, NKV, D)
    _shape(out, "out", T, NQ, D)
    _shape(kv_act_seqs, "kv_act_seqs", B)
    _shape(cu_tokens, "cu_tokens", B + 1)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks]")
    if window is not None and window < 1:
        raise ValueError("window must be 1 or more, or None for all keys")
    if sinks < 0:
        raise ValueError("sinks must be 0 or more")
    if max_tokens is None:
        max_tokens = max(1, T)
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(D)
    if workspace is None:
        workspace = _own_workspace(lambda: WindowWorkspace(max_tokens, NQ, NKV, D,
                                                           device=q.device), stream, ready)
    _one_device(q=q, q_scale=q_scale, k_cache=k_cache, k_scale=k_scale, v_cache=v_cache,
                v_scale=v_scale, block_table=block_table, kv_act_seqs=kv_act_seqs,
                cu_tokens=cu_tokens, out=out, workspace=workspace.buf)
    args = (_ptr(q), _ptr(q_scale), _ptr(k_cache), _ptr(k_scale), _ptr(v_cache), _ptr(v_scale),
            _ptr(block_table), _ptr(kv_act_seqs), _ptr(cu_tokens), _ptr(out), B, T,
            int(max_tokens), NQ, NKV, D, BS, NB, block_table.shape[1], layout,
            0 if window is None else int(window), int(sinks), float(softmax_scale),
            _ptr(workspace.buf), workspace.nbytes)
    keep = (q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table, kv_act_seqs, cu_tokens,
            out, workspace)
    return args, keep


def window_attention(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table, kv_act_seqs,
                     cu_tokens, out, *, window: int | None, sinks: int = 0,
                     max_tokens: int | None = None, layout: int = LAYOUT_BSND,
                     softmax_scale=None, workspace: WindowWorkspace | None = None, stream=None):
    """Causal attention of a ragged batch to a sliding window and to the first
    tokens, over the paged FP8 cache (in place into ``out``): the token at
    position p sees the keys j <= p with p - j < window (all of them with None)
    or j < sinks.

    q [T, NQ, 128] E4M3, q_scale float32 [T, NQ], out bfloat16 [T, NQ, 128]: rows
    cu_tokens[b] .. cu_tokens[b + 1] - 1 (int32 [B + 1]) are the last positions of
    sequence b, which kv_act_seqs int32 [B] counts in; rows behind cu_tokens[B]
    stay as they were. The caches, their scales and the block table as in
    decode(); entries of blocks that no row sees need not be valid. max_tokens:
    the most tokens a sequence has (default T; the scratch and the choice of the
    kernel go by it, and tokens of a sequence behind it get zeros)."""
    args, keep = _window_args(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table,
                              kv_act_seqs, cu_tokens, out, window, sinks, max_tokens, layout,
                              softmax_scale, workspace, stream)
    _check(lib().pa_fp8_window_attention(*args, _stream(stream)), "pa_fp8_window_attention")
    del keep   # (a workspace made here lives until the launch is enqueued)
    return out


def prepare_window_attention(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table,
                             kv_act_seqs, cu_tokens, out, *, window: int | None, sinks: int = 0,
                             max_tokens: int | None = None, layout: int = LAYOUT_BSND,
                             softmax_scale=None, workspace: WindowWorkspace | None = None,
                             stream=None):
    """window_attention() prepared once: returns a callable that launches the same
    call on the same buffers."""
    args, keep = _window_args(q, q_scale, k_cache, k_scale, v_cache, v_scale, block_table,
                              kv_act_seqs, cu_tokens, out, window, sinks, max_tokens, layout,
                              softmax_scale, workspace, stream, ready=True)
    return _Prepared(lib().pa_fp8_window_attention, "pa_fp8_window_attention", args, keep, stream,
                     scratch=None if workspace is not None else keep[-1])


def _logprob_args(logits, tokens, logprobs, ranks, entropy, top_ids, top_logprobs):
    torch = _torch()
    _need(logits, "logits", (torch.float32, torch.bfloat16), contiguous=False)
    if logits.dim() != 2:
        raise ValueError("logits must be [rows, V]")
    R, V = logits.shape
    if (V > 1 and logits.stride(1) != 1) or (R > 1 and logits.stride(0) < V):
        raise ValueError("logits must have contiguous rows that do not overlap")
    _need(tokens, "tokens", (torch.int32, torch.int64))
    _shape(tokens, "tokens", R)
    _need(logprobs, "logprobs", torch.float32)
    _shape(logprobs, "logprobs", R)
    for t, n, dt in ((ranks, "ranks", torch.int32), (entropy, "entropy", torch.float32)):
        if t is not None:
            _need(t, n, dt)
            _shape(t, n, R)
    top = 0
    if (top_ids is None) != (top_logprobs is None):
        raise ValueError("top_ids and top_logprobs go together")
    if top_ids is not None:
        _need(top_ids, "top_ids", torch.int32)
        if top_ids.dim() != 2:
            raise ValueError("top_ids must be [rows, alternatives]")
        top = top_ids.shape[1]
        _shape(top_ids, "top_ids", R, top)
        _need(top_logprobs, "top_logprobs", torch.float32)
        _shape(top_logprobs, "top_logprobs", R, top)
    _one_device(logits=logits, tokens=tokens, logprobs=logprobs, ranks=ranks, entropy=entropy,
                top_ids=top_ids, top_logprobs=top_logprobs)
    args = (_ptr(logits), _in_dtype(logits), logits.stride(0) if R > 1 else V, _ptr(tokens),
            INDEX_I64 if tokens.dtype == torch.int64 else INDEX_I32, R, V, _ptr(logprobs),
            _ptr(ranks), _ptr(entropy), top, _ptr(top_ids), _ptr(top_logprobs))
    keep = (logits, tokens, logprobs, ranks, entropy, top_ids, top_logprobs)
    return args, keep


def token_logprobs(logits, tokens, logprobs, *, ranks=None, entropy=None, top_ids=None,
                   top_logprobs=None, stream=None):
    """Log probabilities of given tokens from logits (in place into logprobs and
    the others that are given).

    logits float32 or bfloat16 [R, V], rows any stride apart (a padded
    vocabulary's view); tokens int32/int64 [R]; logprobs float32 [R]; ranks int32
    [R]: how many logits are larger than the token's; entropy float32 [R];
    top_ids int32 and top_logprobs float32 [R, k], k at most 32: the k most
    probable tokens, of equal ones the lower index first. A logit of -inf has the
    log probability -inf; a row with a NaN or +inf gets NaN, ranks and ids -1, a
    token outside [0, V) NaN and rank -1."""
    args, keep = _logprob_args(logits, tokens, logprobs, ranks, entropy, top_ids, top_logprobs)
    _check(lib().pa_token_logprobs(*args, _stream(stream)), "pa_token_logprobs")
    del keep


def prepare_token_logprobs(logits, tokens, logprobs, *, ranks=None, entropy=None, top_ids=None,
                           top_logprobs=None, stream=None):
    """token_logprobs() prepared once: returns a callable that launches the same
    call on the same buffers."""
    args, keep = _logprob_args(logits, tokens, logprobs, ranks, entropy, top_ids, top_logprobs)
    return _Prepared(lib().pa_token_logprobs, "pa_token_logprobs", args, keep, stream)


__all__ = [
    "LAYOUT_BSND", "LAYOUT_BNBD", "PaError", "build", "lib", "decode", "decode_workspace_size",
    "auto_s2_tile", "prepare_decode", "prepare_cache_quant_scatter",
    "DecodeWorkspace", "cache_scatter", "cache_quant_scatter", "quantize_rows",
    "value_channel_scale", "qkv_norm_rope_append", "prepare_qkv_norm_rope_append",
    "tree_decode", "prepare_tree_decode", "tree_decode_workspace_size", "TreeWorkspace",
    "tree_verify", "prepare_tree_verify", "cache_keep_path", "prepare_cache_keep_path",
    "plan_batch", "prepare_plan_batch", "qkv_norm_mrope_append", "prepare_qkv_norm_mrope_append",
    "window_attention", "prepare_window_attention", "window_attention_workspace_size",
    "WindowWorkspace", "token_logprobs", "prepare_token_logprobs",
]


MLA_ROW_USED = 656


class MlaStatus:
    """A device int the MLA decode kernel ORs a bit into when one of its
    bounded waits gives up (zeroed at creation)."""

    def __init__(self, device=None):
        torch = _torch()
        self.buf = torch.zeros(1, dtype=torch.int32,
                               device=device if device is not None else torch.cuda.current_device())

    def value(self) -> int:
        return int(self.buf.item())


def _mla_args(q_nope, q_rope, topk_indices, block_table, kv_act_seqs, out, S1, softmax_scale):
    torch = _torch()
    _need(q_nope, "q_nope", torch.bfloat16)
    _need(q_rope, "q_rope", torch.bfloat16)
    _need(topk_indices, "topk_indices", torch.int32)
    _need(block_table, "block_table", torch.int32)
    _need(kv_act_seqs, "kv_act_seqs", torch.int32)
    _need(out, "out", torch.bfloat16)
    T, NQ, dn = q_nope.shape
    if dn != 512 or tuple(q_rope.shape) != (T, NQ, 64) or tuple(out.shape) != (T, NQ, 512):
        raise ValueError("q_nope/out must be [T, NQ, 512] and q_rope [T, NQ, 64]")
    B = kv_act_seqs.shape[0]
    if T != B * S1 or topk_indices.shape[0] != T:
        raise ValueError("B*S1 must equal the query token count of q_nope and topk_indices")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(576.0)
    return B, NQ, float(softmax_scale)


def mla_sparse_decode(q_nope, q_rope, nope_cache, topk_indices, block_table, kv_act_seqs, out, *,
                      S1: int, status: MlaStatus, block_size: int = 128, softmax_scale=None,
                      s2_tile: int = 128, stream=None):
    """MLA sparse attention with FP8 anti-quantisation (decode), in place.

    q_nope bfloat16 [B*S1, NQ, 512], q_rope bfloat16 [B*S1, NQ, 64];
    nope_cache uint8 [num_blocks*block_size, row_bytes] packed rows (E4M3 kn |
    BF16 kr | 4 FP32 scales, row_bytes >= 656); topk_indices int32
    [B*S1, topk]; block_table int32 [B, max_blocks]; kv_act_seqs int32 [B];
    out bfloat16 [B*S1, NQ, 512]."""
    torch = _torch()
    B, NQ, sc = _mla_args(q_nope, q_rope, topk_indices, block_table, kv_act_seqs, out, S1,
                          softmax_scale)
    _need(nope_cache, "nope_cache", torch.uint8)
    rows, row_bytes = nope_cache.shape
    if rows % block_size:
        raise ValueError("nope_cache rows must be a multiple of block_size")
    st = lib().pa_mla_sparse_decode(_ptr(q_nope), _ptr(q_rope), _ptr(nope_cache), row_bytes,
                                    _ptr(topk_indices), _ptr(block_table), _ptr(kv_act_seqs),
                                    _ptr(out), B, S1, NQ, 1, topk_indices.shape[1], block_size,
                                    rows // block_size, block_table.shape[1], sc,
                                    s2_tile, _ptr(status.buf), _stream(stream))
    _check(st, "pa_mla_sparse_decode")


def mla_sparse_decode_kvc(q_nope, q_rope, kv_cache, topk_indices, block_table, kv_act_seqs, out,
                          *, quant_mode: int, S1: int, status: MlaStatus, block_size: int = 128,
                          softmax_scale=None, s2_tile: int = 128, stream=None):
    """The MLA sparse decode of ``mla_sparse_decode`` over cache rows written by
    ``kv_compress_epilog`` with d = 576 and the given quant_mode (0: BF16 group
    scales, 1: E8M0 group scales). kv_cache is the epilog's cache, uint8
    [block_num, block_size, 1, head_dim] (blocks may be strided, rows within a
    block contiguous), or [block_num * block_size, head_dim]; head_dim >= 656
    and a multiple of 16."""
    torch = _torch()
    B, NQ, sc = _mla_args(q_nope, q_rope, topk_indices, block_table, kv_act_seqs, out, S1,
                          softmax_scale)
    _need(kv_cache, "kv_cache", torch.uint8, contiguous=False)
    if kv_cache.dim() == 4:
        nb, bs, one, row_bytes = kv_cache.shape
        if one != 1 or bs != block_size or kv_cache.stride(3) != 1 or kv_cache.stride(1) != row_bytes:
            raise ValueError("kv_cache must be [block_num, block_size, 1, head_dim] with "
                             "contiguous rows inside a block")
        stride = kv_cache.stride(0)
    elif kv_cache.dim() == 2 and kv_cache.is_contiguous():
        rows, row_bytes = kv_cache.shape
        if rows % block_size:
            raise ValueError("kv_cache rows must be a multiple of block_size")
        nb, stride = rows // block_size, block_size * row_bytes
    else:
        raise ValueError("kv_cache must be [block_num, block_size, 1, head_dim] or a contiguous "
                         "[block_num * block_size, head_dim]")
    st = lib().pa_mla_sparse_decode_kvc(_ptr(q_nope), _ptr(q_rope), _ptr(kv_cache), row_bytes,
                                        stride, int(quant_mode), _ptr(topk_indices),
                                        _ptr(block_table), _ptr(kv_act_seqs), _ptr(out), B, S1,
                                        NQ, 1, topk_indices.shape[1], block_size, nb,
                                        block_table.shape[1], sc, s2_tile, _ptr(status.buf),
                                        _stream(stream))
    _check(st, "pa_mla_sparse_decode_kvc")
