"""Paged KV-cache decode attention for GB300 (sm_103a): Python binding.

A thin ctypes layer over the C ABI in ``include/pkv.h`` (library
``_lib/libpkv.so``, built in-tree by ``_build.py``).  It only marshals
arguments: torch tensors supply device pointers and the current CUDA
stream; every step of the computation runs in the library's kernels.  There
is no CPU fallback: if the library is missing or the call fails, a
:class:`PkvError` is raised.

Layouts (see the header for the full contract):
  k_cache, v_cache  [S][NB][Hkv][bs][D]  torch.bfloat16, or torch.uint8 holding
                    E4M3 codes (FP8 cache);
  k_scale, v_scale  float32 [S][NB][Hkv] (FP8 cache only);
  q, out            bfloat16 [B][Hq][D];
  block_tables      int32 [B][MB];  context_lens int32 [B];
  kv_group_ptr      host int32 [L] (shared-with pointer per layer);
  tree_mask         int32 [B or 1][T][ceil(T / 32)], the bits of a drafted tree's nodes;
  packed rows       bfloat16 [N][Hq][D], request b's at query_starts[b] ..
                    query_starts[b + 1] - 1 (int32 [B + 1]).

A step of continuous batching (prompts, chunks of them and single tokens in one
batch):
  :func:`extend_tables` (blocks, slots and positions of the packed rows), then
  per layer :func:`rope_append` (norms and rotation of queries and keys, keys
  and values into their slots) and :func:`paged_decode_packed`.

A step of speculative decoding with drafted trees:
  :func:`extend_tables` (blocks and slots for the nodes), :func:`tree_masks`
  (what each node sees, and its position), per layer :func:`rope_append` (or
  :func:`kv_append`) and :func:`paged_decode_tree`, then :func:`verify_tree`
  (the path that the target model's probabilities accept, and the token behind
  it) and :func:`compact_tokens` (with the step's ``new_lens`` and
  ``prev_seq_lens``, so that a request without room keeps its tokens).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libpkv.so")

PKV_OK = 0
STATUS_NAMES = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "alignment", 4: "cuda",
                5: "device index error", 6: "workspace"}
KV_BF16, KV_FP8_E4M3, KV_INT8 = 0, 1, 2
MATH_AUTO, MATH_FFMA, MATH_MMA, MATH_TC = 0, 1, 2, 3
DEVERR_BLOCK_ID, DEVERR_SLOT, DEVERR_CONTEXT_LEN, DEVERR_TIMEOUT = 1, 2, 4, 8
DEVERR_NO_BLOCKS, DEVERR_TREE, DEVERR_QUERY = 16, 32, 64


class PkvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"pkv status {status} ({STATUS_NAMES.get(status, '?')}): {message}")
        self.status = status


class CacheDesc(ctypes.Structure):
    _fields_ = [("num_slots", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class DecodeOpts(ctypes.Structure):
    _fields_ = [("partition_blocks", ctypes.c_int32), ("math", ctypes.c_int32),
                ("warps_per_cta", ctypes.c_int32), ("stages", ctypes.c_int32),
                ("event_decode_start", ctypes.c_void_p), ("event_decode_end", ctypes.c_void_p)]


class DecodePlan(ctypes.Structure):
    _fields_ = [("partition_blocks", ctypes.c_int32), ("max_partitions", ctypes.c_int32),
                ("math", ctypes.c_int32), ("warps_per_cta", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("kernels_per_call", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_size_t), ("smem_bytes_per_cta", ctypes.c_size_t),
                ("query_tokens_per_tile", ctypes.c_int32), ("row_tiles", ctypes.c_int32)]

MAX_QUERY_TOKENS = 512
ABI_VERSION = 2


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return LIB_PATH


def load() -> ctypes.CDLL:
    """Load the built library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise PkvError(4, f"CUDA library not built: {LIB_PATH} is missing "
                              "(run paged_kv_cache_274_gb300._build.build())")
        lib = ctypes.CDLL(LIB_PATH)
        P, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        pdesc, popts = ctypes.POINTER(CacheDesc), ctypes.POINTER(DecodeOpts)
        lib.pkv_kv_append.restype = ctypes.c_int
        lib.pkv_kv_append.argtypes = [pdesc, i32, P, P, P, i32, P, P, P, P, P]
        pf64, i64_ = ctypes.POINTER(ctypes.c_double), ctypes.c_int64
        lib.pkv_rope_append.restype = ctypes.c_int
        lib.pkv_rope_append.argtypes = [pdesc, i32, P, i64_, P, i64_, P, i64_, i32, i32, P, P, f32, P, i32, pf64,
                                        ctypes.POINTER(i32), i32, i32, P, P, i64_, P, P, P, P, P]
        lib.pkv_decode_workspace_bytes.restype = sz
        lib.pkv_decode_workspace_bytes.argtypes = [pdesc, i32, i32, i32, popts]
        lib.pkv_decode_describe.restype = ctypes.c_int
        lib.pkv_decode_describe.argtypes = [pdesc, i32, i32, i32, popts, ctypes.POINTER(DecodePlan)]
        lib.pkv_paged_decode.restype = ctypes.c_int
        lib.pkv_paged_decode.argtypes = [pdesc, P, i32, i32, P, P, P, P, P, i32, P, P, i32, i32,
                                         f32, P, P, sz, popts, P]
        lib.pkv_decode_multi_workspace_bytes.restype = sz
        lib.pkv_decode_multi_workspace_bytes.argtypes = [pdesc, i32, i32, i32, i32, popts]
        lib.pkv_decode_multi_describe.restype = ctypes.c_int
        lib.pkv_decode_multi_describe.argtypes = [pdesc, i32, i32, i32, i32, popts,
                                                  ctypes.POINTER(DecodePlan)]
        lib.pkv_paged_decode_multi.restype = ctypes.c_int
        lib.pkv_paged_decode_multi.argtypes = [pdesc, P, i32, i32, i32, P, P, P, P, P, i32, P, P, i32,
                                               i32, f32, P, P, sz, popts, P]
        lib.pkv_append_and_decode.restype = ctypes.c_int
        lib.pkv_append_and_decode.argtypes = [pdesc, P, P, P, i32, P, i32, i32, i32, P, P, P, P, P, i32, P,
                                              P, i32, i32, f32, P, P, sz, popts, P]
        lib.pkv_paged_decode_tree.restype = ctypes.c_int
        lib.pkv_paged_decode_tree.argtypes = [pdesc, P, i32, i32, i32, P, P, P, P, P, i32, P, P, i32, P, P, i32,
                                              i32, f32, P, P, sz, popts, P]
        lib.pkv_decode_tree_workspace_bytes.restype = sz
        lib.pkv_decode_tree_workspace_bytes.argtypes = [pdesc, i32, i32, i32, i32, popts]
        lib.pkv_decode_tree_describe.restype = ctypes.c_int
        lib.pkv_decode_tree_describe.argtypes = [pdesc, i32, i32, i32, i32, popts, ctypes.POINTER(DecodePlan)]
        lib.pkv_paged_decode_packed.restype = ctypes.c_int
        lib.pkv_paged_decode_packed.argtypes = [pdesc, P, i32, i32, i32, i32, P, P, P, P, P, i32, P, P, P, i32, i32, f32, P, P,
                                                sz, popts, P]
        lib.pkv_decode_packed_workspace_bytes.restype = sz
        lib.pkv_decode_packed_workspace_bytes.argtypes = [pdesc, i32, i32, i32, i32, i32, popts]
        lib.pkv_tree_masks.restype = ctypes.c_int
        lib.pkv_tree_masks.argtypes = [P, P, P, i32, i32, P, P, P]
        lib.pkv_extend_tables.restype = ctypes.c_int
        lib.pkv_extend_tables.argtypes = [i32, i32, i32, i32, P, P, P, P, P, P, P, P, P, P, P, P, P, i32, P]
        lib.pkv_verify_tree.restype = ctypes.c_int
        lib.pkv_verify_tree.argtypes = [P, P, P, P, i64_, P, i64_, i32, i32, i32, P, P, P, P, i32, P, P]
        lib.pkv_compact_tokens.restype = ctypes.c_int
        lib.pkv_compact_tokens.argtypes = [pdesc, P, P, i32, i32, P, P, i32, P, i32, P, P, P, P, P, P]
        lib.pkv_compact_tokens_kept.restype = ctypes.c_int
        lib.pkv_compact_tokens_kept.argtypes = [pdesc, P, P, i32, i32, P, P, i32, P, i32, P, P, P, P, P, P, P, P]
        lib.pkv_paged_decode_static_workspace.restype = ctypes.c_int
        lib.pkv_paged_decode_static_workspace.argtypes = [pdesc, P, i32, i32, P, P, P, P, P, i32, P,
                                                          P, i32, i32, f32, P, popts, P]
        lib.pkv_copy_blocks.restype = ctypes.c_int
        lib.pkv_copy_blocks.argtypes = [pdesc, P, P, P, P, i32, P, P, P, P, i32, P, i32, P]
        lib.pkv_read_probe.restype = ctypes.c_int
        lib.pkv_read_probe.argtypes = [P, sz, P, P]
        lib.pkv_read_device_error.restype = ctypes.c_int
        lib.pkv_read_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32), P]
        lib.pkv_status_string.restype = ctypes.c_char_p
        lib.pkv_status_string.argtypes = [ctypes.c_int]
        lib.pkv_last_error_message.restype = ctypes.c_char_p
        lib.pkv_last_error_message.argtypes = []
        lib.pkv_abi_version.restype = ctypes.c_int32
        lib.pkv_abi_version.argtypes = []
        i64 = ctypes.c_int64
        pi32 = ctypes.POINTER(ctypes.c_int32)
        pi64 = ctypes.POINTER(ctypes.c_int64)
        lib.pkv_prefix_block_hashes.restype = ctypes.c_int
        lib.pkv_prefix_block_hashes.argtypes = [i32, P, i64, P]
        lib.pkv_prefix_cache_create.restype = ctypes.c_int
        lib.pkv_prefix_cache_create.argtypes = [i32, i32, ctypes.POINTER(ctypes.c_void_p)]
        lib.pkv_prefix_cache_destroy.restype = ctypes.c_int
        lib.pkv_prefix_cache_destroy.argtypes = [P]
        lib.pkv_prefix_cache_match.restype = ctypes.c_int
        lib.pkv_prefix_cache_match.argtypes = [P, i32, P, i64, P, i32, pi32]
        lib.pkv_prefix_cache_insert.restype = ctypes.c_int
        lib.pkv_prefix_cache_insert.argtypes = [P, i32, P, i64, P, i32, pi32]
        lib.pkv_prefix_cache_erase.restype = ctypes.c_int
        lib.pkv_prefix_cache_erase.argtypes = [P, i32, P, i32, pi32]
        lib.pkv_prefix_cache_stats.restype = ctypes.c_int
        lib.pkv_prefix_cache_stats.argtypes = [P, i32, pi64, pi64, pi64]
        if lib.pkv_abi_version() != ABI_VERSION:
            raise RuntimeError(f"{LIB_PATH} has ABI version {lib.pkv_abi_version()}, "
                               f"this binding needs {ABI_VERSION}: rebuild")
        _lib = lib
        return lib


def _check(status: int):
    if status != PKV_OK:
        msg = load().pkv_last_error_message().decode(errors="replace")
        raise PkvError(status, msg)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# The current device, and its current stream's handle without a Stream object
# (0.1 us instead of 3), by torch's internal calls where it has them.
_get_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _check_device(device: int):
    """A prepared call launches on the current device: its tensors are there."""
    here = _get_device() if _get_device is not None else torch.cuda.current_device()
    if here != device:
        raise PkvError(1, f"the call's tensors are on cuda:{device}, the current device is cuda:{here}")


def _current_handle(device: int):
    """cudaStream_t of the current stream, for a prepared call whose tensors
    are on this device."""
    _check_device(device)
    return _raw_stream(device) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream


def _prepared_handle(device: int, stream, bound):
    """The stream of a prepared call: the one given, the one it was prepared
    with, or the current one."""
    if stream is None and bound is None:
        return _current_handle(device)
    _check_device(device)
    return bound if stream is None else _stream_handle(stream)


def _need_cuda(name: str, t: torch.Tensor, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise PkvError(1, f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise PkvError(1, f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise PkvError(1, f"{name} must be {dtype}, got {t.dtype}")


def _need_here(name: str, t: torch.Tensor, dtype, shape=None):
    """_need_cuda, on the current device (where the call launches), of this
    shape."""
    _need_cuda(name, t, dtype)
    if t.get_device() != torch.cuda.current_device():
        raise PkvError(1, f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    if shape is not None and tuple(t.shape) != shape:
        raise PkvError(1, f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _allocating_on(stream):
    """Context in which new tensors belong to the stream that a call launches on."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _need_page_params(desc: CacheDesc, t: Optional[torch.Tensor], name: str):
    """E4M3: fp32 [S][NB][Hkv]; INT8: fp32 [S][NB][Hkv][2] (scale, zero)."""
    _need_cuda(name, t, torch.float32)
    want = (desc.num_slots, desc.num_blocks, desc.num_kv_heads)
    if desc.dtype == KV_INT8:
        want = want + (2,)
    if tuple(t.shape) != want:
        raise PkvError(1, f"{name} must have shape {list(want)}")


def cache_desc(k_cache: torch.Tensor) -> CacheDesc:
    """Descriptor of a [S][NB][Hkv][bs][D] cache tensor (bf16, or uint8 = E4M3)."""
    if k_cache.dim() != 5:
        raise PkvError(1, "cache must be 5-D [S][NB][Hkv][bs][D]")
    if k_cache.dtype == torch.bfloat16:
        dt = KV_BF16
    elif k_cache.dtype == torch.uint8:
        dt = KV_FP8_E4M3
    elif k_cache.dtype == torch.int8:
        dt = KV_INT8
    else:
        raise PkvError(1, f"cache dtype {k_cache.dtype} (bfloat16, uint8 E4M3 codes or int8)")
    S, NB, Hkv, bs, D = (int(x) for x in k_cache.shape)
    return CacheDesc(S, NB, bs, Hkv, D, dt)


def kv_append(k: torch.Tensor, v: torch.Tensor, slot_mapping: torch.Tensor,
              k_cache: torch.Tensor, v_cache: torch.Tensor,
              k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
              slot: int = 0, stream=None) -> None:
    """Write new tokens k, v [N][Hkv][D] (bf16) into cache slot ``slot`` at
    ``slot_mapping`` (int64 [N], -1 = skip)."""
    desc = cache_desc(k_cache)
    for n, t in (("k", k), ("v", v)):
        _need_cuda(n, t, torch.bfloat16)
    _need_cuda("slot_mapping", slot_mapping, torch.int64)
    _need_cuda("k_cache", k_cache)
    _need_cuda("v_cache", v_cache, k_cache.dtype)
    N = int(slot_mapping.shape[0])
    if k.shape != (N, desc.num_kv_heads, desc.head_dim) or v.shape != k.shape:
        raise PkvError(1, f"k/v must be [{N}][{desc.num_kv_heads}][{desc.head_dim}]")
    if desc.dtype != KV_BF16:
        _need_page_params(desc, k_scale, "k_scale")
        _need_page_params(desc, v_scale, "v_scale")
    _check(load().pkv_kv_append(ctypes.byref(desc), int(slot), _ptr(k), _ptr(v), _ptr(slot_mapping),
                                N, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                                _stream_handle(stream)))


def _need_rows(name: str, t: torch.Tensor, shape) -> int:
    """A bf16 tensor [N][H][D] on the current device whose heads lie one behind
    the other; returns the elements between its tokens."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise PkvError(1, f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise PkvError(1, f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.get_device() != torch.cuda.current_device():
        raise PkvError(1, f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    if t.dim() != 3 or any(w is not None and n != w for n, w in zip(t.shape, shape)):
        raise PkvError(1, f"{name} must be {''.join('[%s]' % ('H' if w is None else w) for w in shape)}, got {list(t.shape)}")
    N, H, D = t.shape
    if N == 0:
        return H * D
    if (D > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != D):
        raise PkvError(1, f"{name}'s heads must lie one behind the other")
    return t.stride(0) if N > 1 else H * D


def _marshal_rope_append(q, k, v, positions, inv_freq, slot_mapping, k_cache, v_cache, k_scale=None, v_scale=None, slot=0,
                         q_weight=None, k_weight=None, eps=1e-6, freq_axes=None, interleaved=False, out=None, stream=None):
    desc = cache_desc(k_cache)
    D, Hkv = desc.head_dim, desc.num_kv_heads
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise PkvError(1, "q must be [N][Hq][D]")
    N, Hq = q.shape[0], q.shape[1]
    q_stride = _need_rows("q", q, (N, None, D))
    if (k is None) != (v is None):
        raise PkvError(1, "k and v go together")
    k_stride = v_stride = Hkv * D
    _need_here("k_cache", k_cache, k_cache.dtype)
    if k is not None:
        k_stride, v_stride = _need_rows("k", k, (N, Hkv, D)), _need_rows("v", v, (N, Hkv, D))
        _need_here("v_cache", v_cache, k_cache.dtype, tuple(k_cache.shape))
        if desc.dtype != KV_BF16:
            _need_page_params(desc, k_scale, "k_scale")
            _need_page_params(desc, v_scale, "v_scale")
        if slot_mapping is None:
            raise PkvError(1, "slot_mapping is required with k and v")
    if slot_mapping is not None:
        _need_here("slot_mapping", slot_mapping, torch.int64, (N,))
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _need_here(name, w, torch.bfloat16, (D,))
    freqs = [] if inv_freq is None else [float(f) for f in (inv_freq.tolist() if hasattr(inv_freq, "tolist") else inv_freq)]
    axes = 1
    if freqs:
        _need_here("positions", positions, torch.int32)
        if positions.dim() not in (1, 2) or positions.shape[-1] != N:
            raise PkvError(1, f"positions must be [{N}] or [axes][{N}], got {list(positions.shape)}")
        axes = 1 if positions.dim() == 1 else positions.shape[0]
    which = None
    if freq_axes is not None:
        which = [int(x) for x in (freq_axes.tolist() if hasattr(freq_axes, "tolist") else freq_axes)]
        if len(which) != len(freqs):
            raise PkvError(1, f"freq_axes has {len(which)} entries, inv_freq {len(freqs)}")
    if out is None:
        with _allocating_on(stream):
            out = torch.empty((N, Hq, D), dtype=torch.bfloat16, device=q.device)
    out_stride = _need_rows("out", out, (N, Hq, D))
    append = k is not None
    args = (ctypes.byref(desc), int(slot), _ptr(q), q_stride, _ptr(k), k_stride, _ptr(v), v_stride, N, Hq, _ptr(q_weight),
            _ptr(k_weight), float(eps), _ptr(positions) if freqs else None, axes,
            (ctypes.c_double * len(freqs))(*freqs) if freqs else None,
            (ctypes.c_int32 * len(which))(*which) if which else None, 2 * len(freqs), 1 if interleaved else 0,
            _ptr(slot_mapping), _ptr(out), out_stride, _ptr(k_cache) if append else None, _ptr(v_cache) if append else None,
            _ptr(k_scale) if append else None, _ptr(v_scale) if append else None)
    return (load().pkv_rope_append, args, out,
            (q, k, v, positions, slot_mapping, k_cache, v_cache, k_scale, v_scale, q_weight, k_weight))


def rope_append(q: torch.Tensor, k: Optional[torch.Tensor], v: Optional[torch.Tensor], positions: Optional[torch.Tensor],
                inv_freq: Optional[Sequence[float]], slot_mapping: Optional[torch.Tensor], k_cache: torch.Tensor,
                v_cache: torch.Tensor, k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                slot: int = 0, q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                eps: float = 1e-6, freq_axes: Optional[Sequence[int]] = None, interleaved: bool = False,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """A step's queries and keys made ready for the attention in one pass: the
    RMS norm of each head (``q_weight`` / ``k_weight``, bf16 [D]; None: no norm),
    the rotation by ``positions`` (int32 [N] or [axes][N]), and k, v written to
    ``slot_mapping`` as :func:`kv_append` does.  q [N][Hq][D], k and v [N][Hkv][D]
    are bf16 and may be parts of one projection's rows.  ``inv_freq``: radians per
    position of each pair of elements (its length is half of the rotated
    elements; None: no rotation), ``freq_axes`` the position axis of each.
    ``interleaved``: pairs are neighbours instead of halves.  Without k and v the
    queries alone are made.  Tokens with slot -1 are left out.  Returns the
    queries, [N][Hq][D] (``out`` may be q itself)."""
    fn, args, result, _ = _marshal_rope_append(q, k, v, positions, inv_freq, slot_mapping, k_cache, v_cache, k_scale, v_scale,
                                               slot, q_weight, k_weight, eps, freq_axes, interleaved, out, stream)
    _check(fn(*args, _stream_handle(stream)))
    return result


def decode_opts(partition_blocks: int = 0, math: int = MATH_AUTO, warps: int = 0,
                stages: int = 0, event_start=None, event_end=None) -> DecodeOpts:
    """Options of :func:`paged_decode`.  ``event_start`` / ``event_end``:
    optional torch.cuda.Event objects recorded around the decode kernel."""
    def handle(ev):
        return None if ev is None else ctypes.c_void_p(ev.cuda_event)
    return DecodeOpts(int(partition_blocks), int(math), int(warps), int(stages),
                      handle(event_start), handle(event_end))


def decode_workspace_bytes(k_cache: torch.Tensor, batch: int, num_q_heads: int,
                           max_blocks_per_seq: int, opts: Optional[DecodeOpts] = None,
                           query_tokens: int = 1, tree: bool = False) -> int:
    desc = cache_desc(k_cache)
    lib = load()
    fn = lib.pkv_decode_tree_workspace_bytes if tree else lib.pkv_decode_multi_workspace_bytes
    n = fn(ctypes.byref(desc), int(batch), int(query_tokens), int(num_q_heads), int(max_blocks_per_seq),
           ctypes.byref(opts) if opts is not None else None)
    if n == 0:
        raise PkvError(1, "bad arguments for the decode workspace")
    return int(n)


def decode_plan(k_cache: torch.Tensor, batch: int, num_q_heads: int, max_blocks_per_seq: int,
                opts: Optional[DecodeOpts] = None, query_tokens: int = 1, tree: bool = False) -> dict:
    """The resolved launch plan of a decode call (host only, nothing launched)."""
    desc = cache_desc(k_cache)
    plan = DecodePlan()
    lib = load()
    fn = lib.pkv_decode_tree_describe if tree else lib.pkv_decode_multi_describe
    _check(fn(ctypes.byref(desc), int(batch), int(query_tokens), int(num_q_heads), int(max_blocks_per_seq),
              ctypes.byref(opts) if opts is not None else None, ctypes.byref(plan)))
    return {f: getattr(plan, f) for f, _ in DecodePlan._fields_}


def new_decode_workspace(k_cache: torch.Tensor, batch: int, num_q_heads: int,
                         max_blocks_per_seq: int, opts: Optional[DecodeOpts] = None,
                         query_tokens: int = 1, tree: bool = False) -> torch.Tensor:
    """Zero-filled device workspace for :func:`paged_decode` (or, with
    ``query_tokens`` T, :func:`paged_decode_multi`; with ``tree``,
    :func:`paged_decode_tree`)."""
    n = decode_workspace_bytes(k_cache, batch, num_q_heads, max_blocks_per_seq, opts, query_tokens, tree)
    return torch.zeros(n, dtype=torch.uint8, device=k_cache.device)


def _marshal_decode(q, k_cache, v_cache, block_tables, context_lens, kv_group_ptr, layer, scale, out,
                    workspace, k_scale, v_scale, opts, k_new=None, v_new=None, slot_mapping=None,
                    want_dim=None):
    """Check one decode call's arguments and turn them into the C call's
    argument list (without the trailing stream).  Returns (function, args,
    out, workspace)."""
    desc = cache_desc(k_cache)
    _need_cuda("q", q, torch.bfloat16)
    _need_cuda("k_cache", k_cache)
    _need_cuda("v_cache", v_cache, k_cache.dtype)
    _need_cuda("block_tables", block_tables, torch.int32)
    _need_cuda("context_lens", context_lens, torch.int32)
    if want_dim is not None and q.dim() != want_dim:
        raise PkvError(1, "q must be [B][Hq][D]" if want_dim == 3 else "q must be [B][T][Hq][D]")
    if q.dim() == 3:
        B, Hq, D = (int(x) for x in q.shape)
        T = 1
    elif q.dim() == 4:
        B, T, Hq, D = (int(x) for x in q.shape)
    else:
        raise PkvError(1, "q must be [B][Hq][D] or [B][T][Hq][D]")
    if D != desc.head_dim or block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise PkvError(1, "q / block_tables shapes do not match the cache")
    append = k_new is not None or v_new is not None or slot_mapping is not None
    if append:
        _need_cuda("k_new", k_new, torch.bfloat16)
        _need_cuda("v_new", v_new, torch.bfloat16)
        _need_cuda("slot_mapping", slot_mapping, torch.int64)
        N = int(slot_mapping.numel())
        if k_new.shape != (N, desc.num_kv_heads, desc.head_dim) or v_new.shape != k_new.shape:
            raise PkvError(1, "k_new / v_new must be [N][Hkv][D] with N = len(slot_mapping)")
    MB = int(block_tables.shape[1])
    if out is None:
        out = torch.empty_like(q)
    _need_cuda("out", out, torch.bfloat16)
    if out.shape != q.shape:
        raise PkvError(1, "out must be shaped like q")
    if desc.dtype != KV_BF16:
        _need_page_params(desc, k_scale, "k_scale")
        _need_page_params(desc, v_scale, "v_scale")
    if workspace is None:
        workspace = new_decode_workspace(k_cache, B, Hq, MB, opts, T)
    gp = (ctypes.c_int32 * len(kv_group_ptr))(*[int(x) for x in kv_group_ptr])
    if scale is None:
        scale = D ** -0.5
    popts = ctypes.byref(opts) if opts is not None else None
    tail = (_ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_tables), MB,
            _ptr(context_lens), gp, len(kv_group_ptr), int(layer), float(scale), _ptr(out),
            _ptr(workspace), int(workspace.numel()), popts)
    lib = load()
    if append:
        return (lib.pkv_append_and_decode,
                (ctypes.byref(desc), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), N, _ptr(q), B, T, Hq)
                + tail, out, workspace)
    if q.dim() == 4:
        return lib.pkv_paged_decode_multi, (ctypes.byref(desc), _ptr(q), B, T, Hq) + tail, out, workspace
    return lib.pkv_paged_decode, (ctypes.byref(desc), _ptr(q), B, Hq) + tail, out, workspace


def _marshal_tree(q, k_cache, v_cache, block_tables, context_lens, tree_mask, node_counts, kv_group_ptr, layer,
                  scale, out, workspace, k_scale, v_scale, opts, stream=None):
    """As _marshal_decode, for a drafted-tree decode."""
    desc = cache_desc(k_cache)
    _need_here("q", q, torch.bfloat16)
    if q.dim() != 4:
        raise PkvError(1, "q must be [B][T][Hq][D]")
    B, T, Hq, D = q.shape
    if D != desc.head_dim:
        raise PkvError(1, "q does not match the cache's head_dim")
    _need_here("k_cache", k_cache, k_cache.dtype)
    _need_here("v_cache", v_cache, k_cache.dtype, tuple(k_cache.shape))
    _need_here("block_tables", block_tables, torch.int32)
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise PkvError(1, f"block_tables must be [{B}][MB]")
    MB = block_tables.shape[1]
    _need_here("context_lens", context_lens, torch.int32, (B,))
    _need_here("tree_mask", tree_mask, torch.int32)
    if tree_mask.dim() != 3 or tree_mask.shape[0] not in (1, B) or tree_mask.shape[1:] != (T, (T + 31) // 32):
        raise PkvError(1, f"tree_mask must be [{B} or 1][{T}][{(T + 31) // 32}], got {list(tree_mask.shape)}")
    if node_counts is not None:
        _need_here("node_counts", node_counts, torch.int32, (B,))
    if desc.dtype != KV_BF16:
        _need_page_params(desc, k_scale, "k_scale")
        _need_page_params(desc, v_scale, "v_scale")
    with _allocating_on(stream):
        if out is None:
            out = torch.empty_like(q)
        if workspace is None:
            n = decode_workspace_bytes(k_cache, B, Hq, MB, opts, T, tree=True)
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    _need_here("out", out, torch.bfloat16, (B, T, Hq, D))
    _need_here("workspace", workspace, workspace.dtype)
    gp = (ctypes.c_int32 * len(kv_group_ptr))(*[int(x) for x in kv_group_ptr])
    args = (ctypes.byref(desc), _ptr(q), B, T, Hq, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
            _ptr(block_tables), MB, _ptr(context_lens), _ptr(tree_mask), int(tree_mask.shape[0]), _ptr(node_counts),
            gp, len(kv_group_ptr), int(layer), float(D ** -0.5 if scale is None else scale), _ptr(out),
            _ptr(workspace), workspace.numel() * workspace.element_size(),
            ctypes.byref(opts) if opts is not None else None)
    return load().pkv_paged_decode_tree, args, out, workspace


def packed_workspace_bytes(k_cache: torch.Tensor, num_rows: int, batch: int, max_query_tokens: int, num_q_heads: int,
                           max_blocks_per_seq: int, opts: Optional[DecodeOpts] = None) -> int:
    """Workspace bytes of :func:`paged_decode_packed`."""
    desc = cache_desc(k_cache)
    lib = load()
    n = lib.pkv_decode_packed_workspace_bytes(ctypes.byref(desc), int(num_rows), int(batch), int(max_query_tokens), int(num_q_heads),
                                              int(max_blocks_per_seq), ctypes.byref(opts) if opts is not None else None)
    if n == 0:
        raise PkvError(1, f"bad arguments for the workspace: {lib.pkv_last_error_message().decode(errors='replace')}")
    return int(n)


def _marshal_packed(q, k_cache, v_cache, block_tables, context_lens, query_starts, max_query_tokens, kv_group_ptr, layer, scale,
                    out, workspace, k_scale, v_scale, opts, stream=None):
    """As _marshal_decode, for packed rows."""
    desc = cache_desc(k_cache)
    _need_here("q", q, torch.bfloat16)
    if q.dim() != 3:
        raise PkvError(1, "q must be [N][Hq][D]")
    N, Hq, D = q.shape
    if D != desc.head_dim:
        raise PkvError(1, "q does not match the cache's head_dim")
    _need_here("k_cache", k_cache, k_cache.dtype)
    _need_here("v_cache", v_cache, k_cache.dtype, tuple(k_cache.shape))
    _need_here("block_tables", block_tables, torch.int32)
    if block_tables.dim() != 2:
        raise PkvError(1, "block_tables must be [B][MB]")
    B, MB = block_tables.shape
    _need_here("context_lens", context_lens, torch.int32, (B,))
    _need_here("query_starts", query_starts, torch.int32, (B + 1,))
    if desc.dtype != KV_BF16:
        _need_page_params(desc, k_scale, "k_scale")
        _need_page_params(desc, v_scale, "v_scale")
    most = max(1, N) if max_query_tokens is None else int(max_query_tokens)
    with _allocating_on(stream):
        if out is None:
            out = torch.empty_like(q)
        if workspace is None:
            n = packed_workspace_bytes(k_cache, N, B, most, Hq, MB, opts)
            workspace = torch.empty(n, dtype=torch.uint8, device=q.device)
    _need_here("out", out, torch.bfloat16, (N, Hq, D))
    _need_here("workspace", workspace, workspace.dtype)
    gp = (ctypes.c_int32 * len(kv_group_ptr))(*[int(x) for x in kv_group_ptr])
    args = (ctypes.byref(desc), _ptr(q), N, B, most, Hq, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
            _ptr(block_tables), MB, _ptr(context_lens), _ptr(query_starts), gp, len(kv_group_ptr), int(layer),
            float(D ** -0.5 if scale is None else scale), _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
            ctypes.byref(opts) if opts is not None else None)
    return load().pkv_paged_decode_packed, args, out, workspace


def paged_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 block_tables: torch.Tensor, context_lens: torch.Tensor,
                 kv_group_ptr: Sequence[int] = (0,), layer: int = 0,
                 scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None,
                 k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                 opts: Optional[DecodeOpts] = None, stream=None) -> torch.Tensor:
    """One decode step of one layer: returns out [B][Hq][D] (bf16)."""
    fn, args, out, _ = _marshal_decode(q, k_cache, v_cache, block_tables, context_lens, kv_group_ptr, layer,
                                       scale, out, workspace, k_scale, v_scale, opts, want_dim=3)
    _check(fn(*args, _stream_handle(stream)))
    return out


def paged_decode_multi(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       block_tables: torch.Tensor, context_lens: torch.Tensor,
                       kv_group_ptr: Sequence[int] = (0,), layer: int = 0,
                       scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None,
                       k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                       opts: Optional[DecodeOpts] = None, stream=None) -> torch.Tensor:
    """T new query tokens per sequence, q [B][T][Hq][D] (bf16), already
    appended as the last T cached tokens; token t attends causally to the
    first context_lens[b] - T + t + 1 tokens.  Returns out [B][T][Hq][D]."""
    fn, args, out, _ = _marshal_decode(q, k_cache, v_cache, block_tables, context_lens, kv_group_ptr, layer,
                                       scale, out, workspace, k_scale, v_scale, opts, want_dim=4)
    _check(fn(*args, _stream_handle(stream)))
    return out


def append_and_decode(k_new: torch.Tensor, v_new: torch.Tensor, slot_mapping: torch.Tensor,
                      q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      block_tables: torch.Tensor, context_lens: torch.Tensor,
                      kv_group_ptr: Sequence[int] = (0,), layer: int = 0,
                      scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None,
                      k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                      opts: Optional[DecodeOpts] = None, stream=None) -> torch.Tensor:
    """One step in one call: :func:`kv_append` of k_new / v_new [N][Hkv][D]
    at ``slot_mapping`` into cache slot ``kv_group_ptr[layer]``, then
    :func:`paged_decode` (q [B][Hq][D]) or :func:`paged_decode_multi`
    (q [B][T][Hq][D]).  Returns out, shaped like q."""
    if k_new is None or v_new is None or slot_mapping is None:
        raise PkvError(1, "k_new, v_new and slot_mapping are required")
    fn, args, out, _ = _marshal_decode(q, k_cache, v_cache, block_tables, context_lens, kv_group_ptr, layer,
                                       scale, out, workspace, k_scale, v_scale, opts, k_new, v_new,
                                       slot_mapping)
    _check(fn(*args, _stream_handle(stream)))
    return out


def paged_decode_tree(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      block_tables: torch.Tensor, context_lens: torch.Tensor, tree_mask: torch.Tensor,
                      node_counts: Optional[torch.Tensor] = None,
                      kv_group_ptr: Sequence[int] = (0,), layer: int = 0,
                      scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None,
                      k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                      opts: Optional[DecodeOpts] = None, stream=None) -> torch.Tensor:
    """Attention of the nodes of a drafted tree, q [B][T][Hq][D] (bf16): the
    last ``node_counts[b]`` (default T) of the context_lens[b] cached tokens
    are the sequence's nodes; row t attends to every token before them and to
    the nodes whose bits are set in row t of ``tree_mask`` (int32 [B or
    1][T][ceil(T / 32)], see :func:`tree_masks`).  Rows past the count are
    zeros.  Returns out [B][T][Hq][D]."""
    fn, args, out, _ = _marshal_tree(q, k_cache, v_cache, block_tables, context_lens, tree_mask, node_counts,
                                     kv_group_ptr, layer, scale, out, workspace, k_scale, v_scale, opts, stream)
    _check(fn(*args, _stream_handle(stream)))
    return out


def paged_decode_packed(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        block_tables: torch.Tensor, context_lens: torch.Tensor, query_starts: torch.Tensor,
                        max_query_tokens: Optional[int] = None, kv_group_ptr: Sequence[int] = (0,), layer: int = 0,
                        scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None,
                        k_scale: Optional[torch.Tensor] = None, v_scale: Optional[torch.Tensor] = None,
                        opts: Optional[DecodeOpts] = None, stream=None) -> torch.Tensor:
    """Attention of each sequence's new tokens, as many as it has: rows
    query_starts[b] .. query_starts[b + 1] - 1 of q [N][Hq][D] (bf16) are the last
    of the context_lens[b] cached tokens, causal among themselves (the rows that
    :func:`extend_tables` lays out).  ``max_query_tokens``: the most rows of a
    sequence (default N; a tight bound is faster where every sequence has few).
    Rows outside every sequence are left as they were (undefined in a new
    ``out``).  Returns out [N][Hq][D]."""
    fn, args, out, _ = _marshal_packed(q, k_cache, v_cache, block_tables, context_lens, query_starts, max_query_tokens,
                                       kv_group_ptr, layer, scale, out, workspace, k_scale, v_scale, opts, stream)
    _check(fn(*args, _stream_handle(stream)))
    return out


class PreparedDecode:
    """A decode call (:func:`paged_decode`, :func:`paged_decode_multi`,
    :func:`append_and_decode` when ``k_new`` / ``v_new`` / ``slot_mapping``
    are given, :func:`paged_decode_tree` when ``tree_mask`` is, or :func:`paged_decode_packed` when ``query_starts`` is)
    whose arguments were checked and marshalled once.  Each call
    of the object enqueues the same launch again, reading whatever the bound
    tensors hold at that time: the pattern of a serving loop whose step
    buffers stay in place (as under CUDA graph capture) and whose host cost
    per step must stay small.  The object keeps every bound tensor alive.
    ``stream``: the stream bound at preparation (default: the current stream
    at each call); a call may override it."""

    def __init__(self, q, k_cache, v_cache, block_tables, context_lens, kv_group_ptr=(0,), layer=0,
                 scale=None, out=None, workspace=None, k_scale=None, v_scale=None, opts=None,
                 k_new=None, v_new=None, slot_mapping=None, stream=None, tree_mask=None, node_counts=None,
                 query_starts=None, max_query_tokens=None):
        if max_query_tokens is not None and query_starts is None:
            raise PkvError(1, "max_query_tokens without query_starts")
        if query_starts is not None:
            if tree_mask is not None or node_counts is not None or k_new is not None or v_new is not None or slot_mapping is not None:
                raise PkvError(1, "a decode of packed rows neither appends nor takes a tree_mask")
            fn, args, out, workspace = _marshal_packed(q, k_cache, v_cache, block_tables, context_lens, query_starts,
                                                       max_query_tokens, kv_group_ptr, layer, scale, out, workspace,
                                                       k_scale, v_scale, opts, stream)
        elif tree_mask is not None:
            if k_new is not None or v_new is not None or slot_mapping is not None:
                raise PkvError(1, "a drafted-tree decode does not append: call kv_append before it")
            fn, args, out, workspace = _marshal_tree(q, k_cache, v_cache, block_tables, context_lens, tree_mask,
                                                     node_counts, kv_group_ptr, layer, scale, out, workspace,
                                                     k_scale, v_scale, opts, stream)
        elif node_counts is not None:
            raise PkvError(1, "node_counts without tree_mask")
        else:
            fn, args, out, workspace = _marshal_decode(q, k_cache, v_cache, block_tables, context_lens,
                                                       kv_group_ptr, layer, scale, out, workspace, k_scale,
                                                       v_scale, opts, k_new, v_new, slot_mapping)
        self._fn, self._args = fn, args
        self._keep = (q, k_cache, v_cache, block_tables, context_lens, k_scale, v_scale, opts, k_new,
                      v_new, slot_mapping, tree_mask, node_counts, query_starts)
        self.out, self.workspace = out, workspace
        self._stream = None if stream is None else _stream_handle(stream)
        self._device = q.get_device()

    def __call__(self, stream=None) -> torch.Tensor:
        st = self._fn(*self._args, _prepared_handle(self._device, stream, self._stream))
        if st != PKV_OK:
            _check(st)
        return self.out


# ---------------------------------------------------------------------------
# drafted trees and block tables (each _marshal_* checks one call's arguments
# and returns the C function, its arguments without the stream, the result,
# and the tensors to keep alive)
# ---------------------------------------------------------------------------
def _marshal_tree_masks(parents, context_lens=None, node_counts=None, mask=None, positions=None, stream=None):
    _need_here("parents", parents, torch.int32)
    if parents.dim() != 2:
        raise PkvError(1, "parents must be [B][T]")
    B, T = parents.shape
    if not 1 <= T <= MAX_QUERY_TOKENS:
        raise PkvError(1, f"parents must have 1..{MAX_QUERY_TOKENS} nodes, got {T}")
    for name, t in (("context_lens", context_lens), ("node_counts", node_counts)):
        if t is not None:
            _need_here(name, t, torch.int32, (B,))
    W = (T + 31) // 32
    with _allocating_on(stream):
        if mask is None:
            mask = torch.empty((B, T, W), dtype=torch.int32, device=parents.device)
        if positions is None:
            positions = torch.empty((B, T), dtype=torch.int32, device=parents.device)
    _need_here("mask", mask, torch.int32, (B, T, W))
    _need_here("positions", positions, torch.int32, (B, T))
    args = (_ptr(parents), _ptr(context_lens), _ptr(node_counts), B, T, _ptr(mask), _ptr(positions))
    return load().pkv_tree_masks, args, (mask, positions), (parents, context_lens, node_counts)


def tree_masks(parents: torch.Tensor, context_lens: Optional[torch.Tensor] = None,
               node_counts: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
               positions: Optional[torch.Tensor] = None, stream=None):
    """Masks and positions of drafted trees from ``parents`` (int32 [B][T],
    parent of node t in -1..t-1): (mask int32 [B][T][ceil(T / 32)], positions
    int32 [B][T]).  Node t sees itself and what its parent sees; its position
    is the number of tokens before the tree (context_lens[b] - node_counts[b])
    plus its depth."""
    fn, args, result, _ = _marshal_tree_masks(parents, context_lens, node_counts, mask, positions, stream)
    _check(fn(*args, _stream_handle(stream)))
    return result


def new_free_ring(block_ids, num_blocks: int, device="cuda"):
    """(free_ring int32 [num_blocks], free_state int32 [4]) of
    :func:`extend_tables` with these free block ids, first to be taken first."""
    ids = torch.as_tensor(block_ids, dtype=torch.int32).reshape(-1)
    if ids.numel() > num_blocks:
        raise PkvError(1, f"{ids.numel()} free blocks in a pool of {num_blocks}")
    ring = torch.full((int(num_blocks),), -1, dtype=torch.int32)
    ring[:ids.numel()] = ids.cpu()
    state = torch.tensor([0, ids.numel(), 0, 0], dtype=torch.int32)
    return ring.to(device), state.to(device)


def _marshal_extend_tables(seq_lens, new_lens, block_tables, block_counts, free_ring, free_state, block_size, max_tokens,
                           borrowed_counts=None, new_block_counts=None, new_free_state=None, context_lens=None,
                           query_starts=None, slot_mapping=None, positions=None, stream=None):
    i32 = torch.int32
    _need_here("block_tables", block_tables, i32)
    if block_tables.dim() != 2:
        raise PkvError(1, "block_tables must be [B][MB]")
    B, MB = block_tables.shape
    N = int(max_tokens)
    if N < 0:
        raise PkvError(1, f"max_tokens {N} < 0")
    new_block_counts = block_counts if new_block_counts is None else new_block_counts
    new_free_state = free_state if new_free_state is None else new_free_state
    for name, t in (("seq_lens", seq_lens), ("new_lens", new_lens), ("block_counts", block_counts),
                    ("new_block_counts", new_block_counts)):
        _need_here(name, t, i32, (B,))
    if borrowed_counts is not None:
        _need_here("borrowed_counts", borrowed_counts, i32, (B,))
    _need_here("free_ring", free_ring, i32)
    if free_ring.dim() != 1:
        raise PkvError(1, "free_ring must be [NB]")
    _need_here("free_state", free_state, i32, (4,))
    _need_here("new_free_state", new_free_state, i32, (4,))
    dev = block_tables.device
    with _allocating_on(stream):
        if context_lens is None:
            context_lens = torch.empty((B,), dtype=i32, device=dev)
        if query_starts is None:
            query_starts = torch.empty((B + 1,), dtype=i32, device=dev)
        if slot_mapping is None:
            slot_mapping = torch.empty((N,), dtype=torch.int64, device=dev)
        if positions is None:
            positions = torch.empty((N,), dtype=i32, device=dev)
    _need_here("context_lens", context_lens, i32, (B,))
    _need_here("query_starts", query_starts, i32, (B + 1,))
    _need_here("slot_mapping", slot_mapping, torch.int64, (N,))
    _need_here("positions", positions, i32, (N,))
    args = (B, int(block_size), MB, free_ring.shape[0], _ptr(seq_lens), _ptr(new_lens), _ptr(borrowed_counts),
            _ptr(block_tables), _ptr(block_counts), _ptr(new_block_counts), _ptr(free_ring), _ptr(free_state),
            _ptr(new_free_state), _ptr(context_lens), _ptr(query_starts), _ptr(slot_mapping), _ptr(positions), N)
    return (load().pkv_extend_tables, args, (context_lens, query_starts, slot_mapping, positions),
            (seq_lens, new_lens, borrowed_counts, block_tables, block_counts, new_block_counts, free_ring, free_state,
             new_free_state))


def extend_tables(seq_lens: torch.Tensor, new_lens: torch.Tensor, block_tables: torch.Tensor,
                  block_counts: torch.Tensor, free_ring: torch.Tensor, free_state: torch.Tensor, block_size: int,
                  max_tokens: int, borrowed_counts: Optional[torch.Tensor] = None,
                  new_block_counts: Optional[torch.Tensor] = None, new_free_state: Optional[torch.Tensor] = None,
                  context_lens: Optional[torch.Tensor] = None, query_starts: Optional[torch.Tensor] = None,
                  slot_mapping: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None, stream=None):
    """Blocks, slots and positions for the tokens that each request adds this
    step (int32 new_lens [B]; -1: the request has ended and gives its blocks
    back), all on the GPU.  Request b has seq_lens[b] tokens in its
    block_counts[b] blocks; free blocks come from the ring of
    :func:`new_free_ring`.  block_tables and the ring are updated in place,
    the counts and the ring's state too unless ``new_block_counts`` /
    ``new_free_state`` are given.  Returns (context_lens [B], query_starts
    [B + 1], slot_mapping int64 [max_tokens], positions [max_tokens]).  A
    request that cannot be served has context length 0 and slots -1, and
    :func:`read_device_error` says why (see pkv_extend_tables in the header);
    it keeps its blocks and its seq_lens[b] tokens, which the caller passes
    again with the next step."""
    fn, args, result, _ = _marshal_extend_tables(seq_lens, new_lens, block_tables, block_counts, free_ring, free_state,
                                                 block_size, max_tokens, borrowed_counts, new_block_counts,
                                                 new_free_state, context_lens, query_starts, slot_mapping, positions,
                                                 stream)
    _check(fn(*args, _stream_handle(stream)))
    return result


def _need_probs(name: str, t: torch.Tensor, B: int, T: int, V: Optional[int]) -> int:
    """fp32 rows [B][T][V] on the current device at equal distances; returns the
    elements between them."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise PkvError(1, f"{name} must be a CUDA tensor")
    if t.dtype != torch.float32:
        raise PkvError(1, f"{name} must be {torch.float32}, got {t.dtype}")
    if t.get_device() != torch.cuda.current_device():
        raise PkvError(1, f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    if t.dim() != 3 or t.shape[0] != B or t.shape[1] != T or (V is not None and t.shape[2] != V):
        raise PkvError(1, f"{name} must be [{B}][{T}][{'vocab' if V is None else V}], got {list(t.shape)}")
    V = t.shape[2]
    between = t.stride(1) if T > 1 else t.stride(0) if B > 1 else V
    if (V > 1 and t.stride(2) != 1) or (T > 1 and B > 1 and t.stride(0) != T * t.stride(1)):
        raise PkvError(1, f"{name}'s rows must be contiguous and at equal distances")
    return max(between, V) if B * T <= 1 else between


def _marshal_verify_tree(tokens, parents, target_probs, accept_uniforms, sample_uniforms, draft_probs=None, node_counts=None,
                         max_accept=None, accept_idx=None, accept_counts=None, next_tokens=None, stream=None):
    i32 = torch.int32
    _need_here("tokens", tokens, i32)
    if tokens.dim() != 2:
        raise PkvError(1, "tokens must be [B][T]")
    B, T = tokens.shape
    if not 1 <= T <= MAX_QUERY_TOKENS:
        raise PkvError(1, f"tokens must have 1..{MAX_QUERY_TOKENS} nodes, got {T}")
    _need_here("parents", parents, i32, (B, T))
    target_stride = _need_probs("target_probs", target_probs, B, T, None)
    V = target_probs.shape[2]
    draft_stride = 0 if draft_probs is None else _need_probs("draft_probs", draft_probs, B, T, V)
    _need_here("accept_uniforms", accept_uniforms, torch.float32, (B, T))
    _need_here("sample_uniforms", sample_uniforms, torch.float32, (B,))
    if node_counts is not None:
        _need_here("node_counts", node_counts, i32, (B,))
    A = T if max_accept is None else int(max_accept)
    if not 1 <= A <= MAX_QUERY_TOKENS:
        raise PkvError(1, f"max_accept {A} outside 1..{MAX_QUERY_TOKENS}")
    with _allocating_on(stream):
        if accept_idx is None:
            accept_idx = torch.empty((B, A), dtype=i32, device=tokens.device)
        if accept_counts is None:
            accept_counts = torch.empty((B,), dtype=i32, device=tokens.device)
        if next_tokens is None:
            next_tokens = torch.empty((B,), dtype=i32, device=tokens.device)
    _need_here("accept_idx", accept_idx, i32, (B, A))
    _need_here("accept_counts", accept_counts, i32, (B,))
    _need_here("next_tokens", next_tokens, i32, (B,))
    args = (_ptr(tokens), _ptr(parents), _ptr(node_counts), _ptr(target_probs), target_stride, _ptr(draft_probs), draft_stride,
            B, T, V, _ptr(accept_uniforms), _ptr(sample_uniforms), _ptr(accept_idx), _ptr(accept_counts), A, _ptr(next_tokens))
    return (load().pkv_verify_tree, args, (accept_idx, accept_counts, next_tokens),
            (tokens, parents, node_counts, target_probs, draft_probs, accept_uniforms, sample_uniforms))


def verify_tree(tokens: torch.Tensor, parents: torch.Tensor, target_probs: torch.Tensor, accept_uniforms: torch.Tensor,
                sample_uniforms: torch.Tensor, draft_probs: Optional[torch.Tensor] = None,
                node_counts: Optional[torch.Tensor] = None, max_accept: Optional[int] = None,
                accept_idx: Optional[torch.Tensor] = None, accept_counts: Optional[torch.Tensor] = None,
                next_tokens: Optional[torch.Tensor] = None, stream=None):
    """The path of each drafted tree that the target model accepts, and the token
    that follows it.  ``tokens`` and ``parents`` (int32 [B][T]; node 0 is the root,
    parent -1) are the trees, ``target_probs`` (fp32 [B][T][vocab]) the target's
    distribution behind each node, ``draft_probs`` the distribution that each
    node's children were drawn from without replacement (None: children chosen
    without randomness), ``accept_uniforms`` [B][T] and ``sample_uniforms`` [B]
    random numbers in [0, 1).  Returns (accept_idx int32 [B][max_accept],
    accept_counts [B], next_tokens [B]); the first two go to
    :func:`compact_tokens`."""
    fn, args, result, _ = _marshal_verify_tree(tokens, parents, target_probs, accept_uniforms, sample_uniforms, draft_probs,
                                               node_counts, max_accept, accept_idx, accept_counts, next_tokens, stream)
    _check(fn(*args, _stream_handle(stream)))
    return result


def _marshal_compact_tokens(accept_idx, accept_counts, context_lens, block_tables, k_cache, v_cache, num_nodes,
                            node_counts=None, k_scale=None, v_scale=None, seq_lens=None, stream=None, new_lens=None,
                            prev_seq_lens=None):
    desc = cache_desc(k_cache)
    i32 = torch.int32
    _need_here("k_cache", k_cache, k_cache.dtype)
    _need_here("v_cache", v_cache, k_cache.dtype, tuple(k_cache.shape))
    _need_here("accept_idx", accept_idx, i32)
    if accept_idx.dim() != 2:
        raise PkvError(1, "accept_idx must be [B][max_accept]")
    B, A = accept_idx.shape
    _need_here("accept_counts", accept_counts, i32, (B,))
    _need_here("context_lens", context_lens, i32, (B,))
    _need_here("block_tables", block_tables, i32)
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise PkvError(1, f"block_tables must be [{B}][MB]")
    if node_counts is not None:
        _need_here("node_counts", node_counts, i32, (B,))
    if desc.dtype != KV_BF16:
        _need_page_params(desc, k_scale, "k_scale")
        _need_page_params(desc, v_scale, "v_scale")
    if (new_lens is None) != (prev_seq_lens is None):
        raise PkvError(1, "new_lens and prev_seq_lens go together")
    if new_lens is not None:
        _need_here("new_lens", new_lens, i32, (B,))
        _need_here("prev_seq_lens", prev_seq_lens, i32, (B,))
    if seq_lens is None:
        with _allocating_on(stream):
            seq_lens = torch.empty((B,), dtype=i32, device=k_cache.device)
    _need_here("seq_lens", seq_lens, i32, (B,))
    args = (ctypes.byref(desc), _ptr(accept_idx), _ptr(accept_counts), A, B, _ptr(context_lens), _ptr(node_counts),
            int(num_nodes), _ptr(block_tables), block_tables.shape[1], _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
            _ptr(v_scale))
    keep = (accept_idx, accept_counts, context_lens, node_counts, block_tables, k_cache, v_cache, k_scale, v_scale)
    if new_lens is None:
        return load().pkv_compact_tokens, args + (_ptr(seq_lens),), seq_lens, keep
    return (load().pkv_compact_tokens_kept, args + (_ptr(new_lens), _ptr(prev_seq_lens), _ptr(seq_lens)), seq_lens,
            keep + (new_lens, prev_seq_lens))


def compact_tokens(accept_idx: torch.Tensor, accept_counts: torch.Tensor, context_lens: torch.Tensor,
                   block_tables: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, num_nodes: int,
                   node_counts: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                   v_scale: Optional[torch.Tensor] = None, seq_lens: Optional[torch.Tensor] = None,
                   stream=None, new_lens: Optional[torch.Tensor] = None,
                   prev_seq_lens: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Keep the accepted path of each verified tree: the K and V rows of nodes
    accept_idx[b][:accept_counts[b]] (strictly increasing) move, in every
    cache slot, to the positions from the tree's start on.  ``num_nodes`` is T
    of :func:`paged_decode_tree`.  Returns seq_lens [B], the tokens that each
    sequence keeps.

    An inactive sequence (context_lens[b] 0) gets 0.  With ``new_lens`` and
    ``prev_seq_lens``, the new_lens and seq_lens of the step's
    :func:`extend_tables`, that holds for requests that have ended only: those
    that were refused there keep prev_seq_lens[b], whatever their node and
    accept counts hold.  ``seq_lens`` may be ``prev_seq_lens`` itself."""
    fn, args, result, _ = _marshal_compact_tokens(accept_idx, accept_counts, context_lens, block_tables, k_cache, v_cache,
                                                  num_nodes, node_counts, k_scale, v_scale, seq_lens, stream, new_lens,
                                                  prev_seq_lens)
    _check(fn(*args, _stream_handle(stream)))
    return result


class PreparedCall:
    """A call of :func:`tree_masks`, :func:`extend_tables`,
    :func:`compact_tokens`, :func:`rope_append` or :func:`verify_tree` (``op``, then its arguments) checked and marshalled
    once, like :class:`PreparedDecode`: each call of the object enqueues the
    same launch again on whatever the bound tensors hold, and returns the
    bound result tensors."""

    def __init__(self, op, *args, stream=None, **kwargs):
        marshal = {tree_masks: _marshal_tree_masks, extend_tables: _marshal_extend_tables,
                   compact_tokens: _marshal_compact_tokens, rope_append: _marshal_rope_append,
                   verify_tree: _marshal_verify_tree}.get(op)
        if marshal is None:
            raise PkvError(1, "PreparedCall takes tree_masks, extend_tables, compact_tokens, rope_append or verify_tree")
        self._fn, self._args, self.result, self._keep = marshal(*args, stream=stream, **kwargs)
        self._stream = None if stream is None else _stream_handle(stream)
        self._device = self._keep[0].get_device()

    def __call__(self, stream=None):
        st = self._fn(*self._args, _prepared_handle(self._device, stream, self._stream))
        if st != PKV_OK:
            _check(st)
        return self.result


def copy_blocks(src_k: torch.Tensor, src_v: torch.Tensor, dst_k: torch.Tensor,
                dst_v: torch.Tensor, block_pairs: torch.Tensor,
                src_k_scale: Optional[torch.Tensor] = None, src_v_scale: Optional[torch.Tensor] = None,
                dst_k_scale: Optional[torch.Tensor] = None, dst_v_scale: Optional[torch.Tensor] = None,
                stream=None) -> None:
    """Copy blocks ``block_pairs[i] = (src, dst)`` (device int32 [n][2]) from
    one pool ``[NB][Hkv][bs][D]`` to another.  Pools may live in device
    memory or in pinned host memory (``tensor.pin_memory()``)."""
    for n, t in (("src_k", src_k), ("src_v", src_v), ("dst_k", dst_k), ("dst_v", dst_v)):
        if t.dim() != 4 or not t.is_contiguous():
            raise PkvError(1, f"{n} must be a contiguous [NB][Hkv][bs][D] tensor")
        if not (t.is_cuda or t.is_pinned()):
            raise PkvError(1, f"{n} must be a CUDA tensor or pinned host memory")
    if src_k.shape[1:] != dst_k.shape[1:] or src_k.dtype != dst_k.dtype:
        raise PkvError(1, "source and destination pages differ in shape or dtype")
    _need_cuda("block_pairs", block_pairs, torch.int32)
    desc = cache_desc(src_k.unsqueeze(0))
    n = int(block_pairs.shape[0])
    _check(load().pkv_copy_blocks(
        ctypes.byref(desc), _ptr(src_k), _ptr(src_v), _ptr(src_k_scale), _ptr(src_v_scale),
        int(src_k.shape[0]), _ptr(dst_k), _ptr(dst_v), _ptr(dst_k_scale), _ptr(dst_v_scale),
        int(dst_k.shape[0]), _ptr(block_pairs), n, _stream_handle(stream)))


STATIC_WORKSPACE_MAX_BYTES = 16 << 20


def paged_decode_static_workspace(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  block_tables: torch.Tensor, context_lens: torch.Tensor,
                                  kv_group_ptr: Sequence[int] = (0,), layer: int = 0,
                                  scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                                  k_scale: Optional[torch.Tensor] = None,
                                  v_scale: Optional[torch.Tensor] = None,
                                  opts: Optional[DecodeOpts] = None, stream=None) -> torch.Tensor:
    """:func:`paged_decode` for callers that cannot allocate a workspace: the
    library's built-in static device array serves as scratch (at most
    STATIC_WORKSPACE_MAX_BYTES; calls that overlap on the GPU race on it).
    ``out`` must be passed in by a caller that cannot allocate."""
    desc = cache_desc(k_cache)
    _need_cuda("q", q, torch.bfloat16)
    _need_cuda("block_tables", block_tables, torch.int32)
    _need_cuda("context_lens", context_lens, torch.int32)
    B, Hq, D = (int(x) for x in q.shape)
    if out is None:
        out = torch.empty_like(q)
    _need_cuda("out", out, torch.bfloat16)
    gp = (ctypes.c_int32 * len(kv_group_ptr))(*[int(x) for x in kv_group_ptr])
    if scale is None:
        scale = D ** -0.5
    _check(load().pkv_paged_decode_static_workspace(
        ctypes.byref(desc), _ptr(q), B, Hq, _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
        _ptr(v_scale), _ptr(block_tables), int(block_tables.shape[1]), _ptr(context_lens), gp,
        len(kv_group_ptr), int(layer), float(scale), _ptr(out),
        ctypes.byref(opts) if opts is not None else None, _stream_handle(stream)))
    return out


def read_probe(data: torch.Tensor, sum_out: torch.Tensor, stream=None) -> torch.Tensor:
    """Read-only HBM probe (a measurement aid, not part of the decode): one
    launch streams the contiguous CUDA tensor ``data`` once and adds the
    unsigned sum of its 32-bit words, modulo 2^64, to ``sum_out`` (a CUDA
    int64 tensor of one element, holding the bits of a uint64)."""
    if not isinstance(data, torch.Tensor) or not data.is_cuda or not data.is_contiguous():
        raise PkvError(1, "data must be a contiguous CUDA tensor")
    _need_cuda("sum_out", sum_out, torch.int64)
    if sum_out.numel() != 1:
        raise PkvError(1, "sum_out must hold one element")
    _check(load().pkv_read_probe(_ptr(data), int(data.numel() * data.element_size()), _ptr(sum_out),
                                 _stream_handle(stream)))
    return sum_out


def read_device_error(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device error word."""
    flags = ctypes.c_uint32(0)
    st = load().pkv_read_device_error(ctypes.byref(flags), _stream_handle(stream))
    if st not in (PKV_OK, 5):
        _check(st)
    return int(flags.value)


def build(force: bool = False) -> str:
    from . import _build
    return _build.build(force=force)


# ---------------------------------------------------------------------------
# prefix cache (host only; include/pkv_prefix.h)
# ---------------------------------------------------------------------------
def _i32_array(values) -> "ctypes.Array":
    vals = [int(v) for v in values]
    return (ctypes.c_int32 * max(1, len(vals)))(*vals)


def prefix_block_hashes(tokens: Sequence[int], block_size: int) -> list:
    """Cumulative FNV-1a-64 hash of every full block of a token sequence."""
    n = len(tokens)
    nb = n // int(block_size) if block_size > 0 else 0
    out = (ctypes.c_uint64 * max(1, nb))()
    _check(load().pkv_prefix_block_hashes(int(block_size), _i32_array(tokens), n, out))
    return [int(out[j]) for j in range(nb)]


class PrefixCache:
    """Host index from block content to physical block, per layer group:
    ``match`` walks a request's full blocks and returns the physical blocks of
    its cached prefix; ``insert`` registers a sequence's full blocks; ``erase``
    forgets freed blocks."""

    def __init__(self, block_size: int, num_groups: int = 1):
        self._lib = load()
        h = ctypes.c_void_p()
        _check(self._lib.pkv_prefix_cache_create(int(block_size), int(num_groups), ctypes.byref(h)))
        self._h = h
        self.block_size = int(block_size)

    def close(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.pkv_prefix_cache_destroy(self._h)
            self._h = None

    def __del__(self):
        self.close()

    def match(self, tokens: Sequence[int], group: int = 0, max_blocks: Optional[int] = None) -> list:
        nb = len(tokens) // self.block_size
        cap = nb if max_blocks is None else min(nb, int(max_blocks))
        ids = (ctypes.c_int32 * max(1, cap))()
        n = ctypes.c_int32(0)
        _check(self._lib.pkv_prefix_cache_match(self._h, int(group), _i32_array(tokens), len(tokens), ids,
                                                 cap, ctypes.byref(n)))
        return [int(ids[j]) for j in range(n.value)]

    def insert(self, tokens: Sequence[int], block_ids: Sequence[int], group: int = 0) -> int:
        n = ctypes.c_int32(0)
        _check(self._lib.pkv_prefix_cache_insert(self._h, int(group), _i32_array(tokens), len(tokens),
                                                  _i32_array(block_ids), len(block_ids), ctypes.byref(n)))
        return n.value

    def erase(self, block_ids: Sequence[int], group: int = 0) -> int:
        n = ctypes.c_int32(0)
        _check(self._lib.pkv_prefix_cache_erase(self._h, int(group), _i32_array(block_ids), len(block_ids),
                                                 ctypes.byref(n)))
        return n.value

    def stats(self, group: int = 0):
        """(entries, lookups, hits) of one group."""
        e, l, h = ctypes.c_int64(0), ctypes.c_int64(0), ctypes.c_int64(0)
        _check(self._lib.pkv_prefix_cache_stats(self._h, int(group), ctypes.byref(e), ctypes.byref(l),
                                                 ctypes.byref(h)))
        return e.value, l.value, h.value
