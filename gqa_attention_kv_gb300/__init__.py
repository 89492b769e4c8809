"""GB300 grouped-query attention over a decoder KV cache.

A thin ctypes binding over the C ABI in ``include/attn_kv.h`` (library
``libgqa_attn_kv.so``, built in-tree by ``gqa_attention_kv_gb300.build``).
Every function here only marshals arguments -- pointers, sizes and the
current CUDA stream -- and calls the entry point of the same name; all work
runs in the library's kernels.  There is no fallback: if the library is
missing or a call is refused, an exception is raised.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading

import torch

from .synth import LINEAR, PAGED, RING  # noqa: F401  (cache-kind constants)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgqa_attn_kv.so")

ATTN_OK = 0
STATUS_NAMES = {0: "ATTN_OK", 1: "ATTN_ERR_NULL", 2: "ATTN_ERR_SHAPE", 3: "ATTN_ERR_UNSUPPORTED",
                4: "ATTN_ERR_WORKSPACE", 5: "ATTN_ERR_BOUNDS", 6: "ATTN_ERR_TIMEOUT",
                7: "ATTN_ERR_CUDA", 8: "ATTN_ERR_ALIGN", 9: "ATTN_ERR_PAGES"}
for _code, _name in STATUS_NAMES.items():
    globals()[_name] = _code
ATTN_DECODE_TABLES_EARLY = 1  # attn_decode_append flags (include/attn_kv.h)
ATTN_DECODE_CACHE_EARLY = 2
ATTN_KV_BF16, ATTN_KV_FP8_E4M3 = 0, 1  # cache element types (attn_kv_dtype)
ATTN_KV_FP8_E4M3_SCALED, ATTN_KV_INT8_SCALED = 2, 3
_SCALED = (ATTN_KV_FP8_E4M3_SCALED, ATTN_KV_INT8_SCALED)
ATTN_LAYOUT_BSHD, ATTN_LAYOUT_BHSD = 0, 1  # cache layouts (attn_kv_layout)
ATTN_ROPE_PAIRS, ATTN_ROPE_HALF = 0, 1  # which dims turn together (attn_rope_layout)

_BF16, _I32, _I64 = torch.bfloat16, torch.int32, torch.int64
_BYTES = (torch.uint8, torch.int8, torch.float8_e4m3fn)  # what may hold 8-bit codes

_lock = threading.Lock()
_lib = None


class AttnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        extra = ""
        if status == 7:  # ATTN_ERR_CUDA
            extra = f": {lib().attn_last_cuda_error().decode()}"
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} "
                         f"({attn_status_string(status)}{extra})")


class _Cache(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("num_slots", ctypes.c_int64), ("slots_per_seq", ctypes.c_int32),
                ("block_table", ctypes.c_void_p), ("block_size", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("k_ref", ctypes.c_void_p), ("layout", ctypes.c_int32),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("scale_block", ctypes.c_int32)]


# _Cache in its C layout: packing it costs half of what building a ctypes structure does
_PACK = struct.Struct("@iPPqiPiiiPiPPi0P").pack
_PACK_ROPE = struct.Struct("@PiifPPf0P").pack  # an attn_rope


def lib():
    """The loaded library (ctypes.CDLL).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(
                    f"{LIB_PATH} is missing: build it with "
                    "`python -m gqa_attention_kv_gb300.build` (nvcc, sm_103a)")
            L = ctypes.CDLL(LIB_PATH)
            p, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
            cp = p  # attn_kv_cache *: a _Cache by reference, or its bytes
            L.attn_kv_append.argtypes = [p, p, p, i64, cp, i32, i32, p, p]
            L.attn_kv_append.restype = i32
            L.attn_decode_workspace_size.argtypes = [cp, i32, i32, i32, i32, i32, i32, i32]
            L.attn_decode_workspace_size.restype = sz
            L.attn_decode_kernel_launches.argtypes = [cp, i32, i32, i32, i32, i32, i32, i32,
                                                      i32, i32, ctypes.c_uint]
            L.attn_decode_kernel_launches.restype = i32
            L.attn_decode.argtypes = [p, cp, p, p, i32, i32, i32, i32, i32, i32, i32,
                                      ctypes.c_float, p, p, sz, p, p]
            L.attn_decode.restype = i32
            L.attn_decode_append.argtypes = [p, p, p, p, p, cp, p, p, i32, i32, i32, i32, i32,
                                             i32, i32, ctypes.c_float, p, p, sz, p,
                                             ctypes.c_uint, p]
            L.attn_decode_append.restype = i32
            L.attn_decode_noalloc.argtypes = [p, cp, p, p, i32, i32, i32, i32, i32, i32, i32,
                                              ctypes.c_float, p, p, p]
            L.attn_decode_noalloc.restype = i32
            L.attn_kv_reference.argtypes = [p, i64, i32, i32, p, p]
            L.attn_kv_reference.restype = i32
            L.attn_prefill.argtypes = [p, p, p, i32, i32, i32, i32, i32, i32, ctypes.c_float, p,
                                       p, p]
            L.attn_prefill.restype = i32
            L.attn_decode_sinks_workspace_size.argtypes = [cp, i32, i32, i32, i32, i32, i32, i32,
                                                           i32]
            L.attn_decode_sinks_workspace_size.restype = sz
            L.attn_decode_sinks.argtypes = [p, cp, p, p, i32, i32, i32, i32, i32, i32, i32, i32,
                                            ctypes.c_float, p, p, sz, p, p]
            L.attn_decode_sinks.restype = i32
            L.attn_decode_shared_workspace_size.argtypes = [cp, i32, i32, i32, i32, i32, i32, i32,
                                                            i32]
            L.attn_decode_shared_workspace_size.restype = sz
            L.attn_decode_shared.argtypes = [p, cp, i32, p, p, p, p, i32, i32, i32, i32, i32, i32,
                                             i32, i32, ctypes.c_float, p, p, sz, p, p]
            L.attn_decode_shared.restype = i32
            L.attn_qk_rope.argtypes = [p, i64, p, i64, p, i64, p, i32, i32, i32, p, p, p]
            L.attn_qk_rope.restype = i32
            L.attn_qk_rope_append.argtypes = [p, i64, p, i64, p, i64, p, p, i64, p, cp, i32, i32,
                                              i32, p, p, p, p]
            L.attn_qk_rope_append.restype = i32
            L.attn_kv_read.argtypes = [p, i64, cp, i32, i32, p, p, p, p]
            L.attn_kv_read.restype = i32
            L.attn_prefill_sinks.argtypes = [p, p, p, i32, i32, i32, i32, i32, i32, i32,
                                             ctypes.c_float, p, p, p]
            L.attn_prefill_sinks.restype = i32
            L.attn_pages_free.argtypes = [p, i32, i32, p, p, p, i32, p, i32, p, p]
            L.attn_pages_free.restype = i32
            L.attn_pages_reserve.argtypes = [p, i32, i32, p, p, p, i32, p, i32, p, p]
            L.attn_pages_reserve.restype = i32
            L.attn_pages_fork.argtypes = [p, i32, i32, p, p, p, i32, i32, p, i32, p, i32, p, p, p]
            L.attn_pages_fork.restype = i32
            L.attn_pages_workspace_size.argtypes = [i32]
            L.attn_pages_workspace_size.restype = sz
            L.attn_pages_compact.argtypes = [p, i32, i32, i32, p, i32, p, i32, p, p, p, sz, p, p]
            L.attn_pages_compact.restype = i32
            L.attn_pages_copy.argtypes = [cp, i32, i32, i32, p, p, i32, p, p]
            L.attn_pages_copy.restype = i32
            L.attn_status_string.argtypes = [i32]
            L.attn_status_string.restype = ctypes.c_char_p
            L.attn_version.restype = ctypes.c_char_p
            L.attn_last_cuda_error.restype = ctypes.c_char_p
            _lib = L
    return _lib


def attn_status_string(status: int) -> str:
    return lib().attn_status_string(int(status)).decode()


def attn_version() -> str:
    return lib().attn_version().decode()


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it (3 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is None:
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _raw_stream(_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _made(make, like, stream, *args):
    """make(like, *args), a tensor of the call's own, made on the stream that uses
    it: ready for it, and not handed on before it is done."""
    if stream is None:
        return make(like, *args)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream) if isinstance(stream, int)
                           else stream):
        return make(like, *args)


def _zeroed(like, nbytes):
    return torch.zeros(nbytes, dtype=torch.uint8, device=like.device)


def _check(rc, where):
    if rc != ATTN_OK:
        raise AttnError(rc, where)


def _want(where, device, dtype, *tensors):
    """Refuses tensors that a kernel would misread: of another type, strided, or
    not on the device that the call launches on."""
    for t in tensors:
        if t.dtype is not dtype or t.get_device() != device or not t.is_contiguous():
            raise AttnError(ATTN_ERR_UNSUPPORTED,
                            f"{where}: a {t.dtype} tensor of shape {tuple(t.shape)} is not a "
                            f"contiguous {dtype} tensor on the current device")


class KVCache:
    """One layer's cache: k, v [num_slots, n_kv_heads, head_dim] on the device,
    bf16, or uint8 E4M3 codes for an FP8 cache (dtype ATTN_KV_FP8_E4M3, whose
    keys are stored relative to k_ref, float32 [n_kv_heads, head_dim] or None).
    layout ATTN_LAYOUT_BHSD: k, v are [num_slots // rows, n_kv_heads, rows,
    head_dim] (rows = slots_per_seq, or block_size when paged); slots are
    numbered as in the slot-major layout.

    dtypes ATTN_KV_FP8_E4M3_SCALED (uint8 codes) and ATTN_KV_INT8_SCALED (int8):
    scale_block consecutive slots of a head share the scales k_scale and
    v_scale, float32 [num_slots // scale_block, n_kv_heads], which
    attn_kv_append keeps.

    kind LINEAR: slots_per_seq = per-request capacity.
    kind PAGED : block_table int32 [batch, max_blocks_per_seq] (device), block_size.
    kind RING  : slots_per_seq = ring size.
    """

    def __init__(self, kind, k, v, slots_per_seq=0, block_table=None, block_size=0,
                 dtype=ATTN_KV_BF16, k_ref=None, layout=ATTN_LAYOUT_BSHD, k_scale=None,
                 v_scale=None, scale_block=0):
        self.__dict__.update(
            kind=int(kind), k=k, v=v, slots_per_seq=int(slots_per_seq), block_table=block_table,
            block_size=int(block_size), dtype=int(dtype), k_ref=k_ref, layout=int(layout),
            k_scale=k_scale, v_scale=v_scale, scale_block=int(scale_block),
            _usable=None, _table=None)  # (a setattr each would cost 2 us)
        if self.dtype in _SCALED and self.scale_block > 0 and \
                (isinstance(k_scale, torch.Tensor) or isinstance(v_scale, torch.Tensor)):
            shape = (self.num_slots // self.scale_block, self.n_kv_heads)
            for t in (k_scale, v_scale):
                if not isinstance(t, torch.Tensor) or t.shape != shape or \
                        t.dtype is not torch.float32 or not t.is_contiguous():
                    raise AttnError(ATTN_ERR_SHAPE, f"KVCache: k_scale and v_scale are contiguous "
                                                    f"float32 tensors of shape {shape}")

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        seen = self.__dict__  # looked at again by the next call
        seen["_usable"] = seen["_table"] = None

    def _want_usable(self, where, device):
        """Refuses k, v, scales and reference that a kernel would read or write out
        of their place: of another type, size, order or device.  Returns what holds
        until a field is set or a tensor is put elsewhere: (device, addresses of k
        and v, their bytes, addresses of the scales, of k_ref, the shape of k and v,
        the bytes of the C structure without the block table)."""
        k, v, ks, vs, ref = self.k, self.v, self.k_scale, self.v_scale, self.k_ref
        store = _BF16 if self.dtype == ATTN_KV_BF16 else k.dtype if k.dtype in _BYTES else \
            torch.uint8
        _want(where, device, store, k, v)
        if k.shape != v.shape or k.dim() != (4 if self.layout == ATTN_LAYOUT_BHSD else 3):
            raise AttnError(ATTN_ERR_SHAPE, f"{where}: k and v are of one shape, [num_slots, "
                                            "n_kv_heads, head_dim] slot-major, of four "
                                            "dimensions head-major")
        scales = ()
        if self.dtype in _SCALED:
            if ks is None or vs is None:
                raise AttnError(ATTN_ERR_NULL, f"{where}: a scaled cache without its scales")
            _want(where, device, torch.float32, ks, vs, *(() if ref is None else (ref,)))
            shape = (self.num_slots // max(1, self.scale_block), self.n_kv_heads)
            if ks.shape != shape or vs.shape != shape or \
                    (ref is not None and ref.numel() != self.n_kv_heads * self.head_dim):
                raise AttnError(ATTN_ERR_SHAPE, f"{where}: k_scale and v_scale are {shape}, "
                                                "k_ref is [n_kv_heads, head_dim]")
            scales = (ks.data_ptr(), vs.data_ptr())
        at = 0 if ref is None else ref.data_ptr()
        known = (device, k.data_ptr(), v.data_ptr(), k.nbytes, scales, at, tuple(k.shape),
                 _PACK(self.kind, k.data_ptr(), v.data_ptr(), self.num_slots, self.slots_per_seq,
                       0, self.block_size, 0, self.dtype, at, self.layout,
                       *(scales or (0, 0)), self.scale_block))
        self.__dict__["_usable"] = known
        return known

    def _known(self, where, device):
        """_want_usable, if it has not been asked since the last change."""
        u, k, v, ref = self._usable, self.k, self.v, self.k_ref
        if u is None or u[0] != device or u[1] != k.data_ptr() or u[2] != v.data_ptr() or \
                u[3] != k.nbytes or u[3] != v.nbytes or \
                (u[4] and u[4] != (self.k_scale.data_ptr(), self.v_scale.data_ptr())) or \
                (ref is not None and u[5] != ref.data_ptr()):
            u = self._want_usable(where, device)
        return u

    def _with_table(self, where, device, batch):
        """The bytes of the C structure, with a block table that has `batch` rows."""
        u, bt, t = self._known(where, device), self.block_table, self._table
        if self.kind != PAGED or bt is None:
            return u[7]
        if t is None or t[0] is not u or t[1] != bt.data_ptr() or t[2] != bt.nbytes:
            _want(where, device, _I32, bt)
            t = (u, bt.data_ptr(), bt.nbytes, bt.numel() // max(1, bt.shape[-1]), self.packed())
            self.__dict__["_table"] = t
        if t[3] < batch:
            raise AttnError(ATTN_ERR_SHAPE, f"{where}: block_table has fewer rows than {batch}")
        return t[4]

    @property
    def n_kv_heads(self):
        return self.k.shape[1]

    @property
    def head_dim(self):
        return self.k.shape[-1]

    @property
    def num_slots(self):
        return self.k.shape[0] * (self.k.shape[2] if self.layout == ATTN_LAYOUT_BHSD else 1)

    def packed(self) -> bytes:
        """struct(), as the bytes of the C structure."""
        bt, ref, ks, vs = self.block_table, self.k_ref, self.k_scale, self.v_scale
        shape = self.k.shape
        return _PACK(self.kind, self.k.data_ptr(), self.v.data_ptr(),
                     shape[0] * (shape[2] if self.layout == ATTN_LAYOUT_BHSD else 1),
                     self.slots_per_seq, 0 if bt is None else bt.data_ptr(), self.block_size,
                     0 if bt is None else bt.shape[-1], self.dtype,
                     0 if ref is None else ref.data_ptr(), self.layout,
                     0 if ks is None else ks.data_ptr(), 0 if vs is None else vs.data_ptr(),
                     self.scale_block)

    def struct(self) -> _Cache:
        return _Cache.from_buffer_copy(self.packed())


def _want_new_rows(where, cache, k_new, v_new, slots, n):
    """The n rows of an append to a scaled cache; returns its C structure's bytes."""
    device = _device()
    u = cache._known(where, device)
    if not (k_new.dtype is v_new.dtype is _BF16 and slots.dtype is _I64 and
            k_new.get_device() == v_new.get_device() == slots.get_device() == device and
            k_new.is_contiguous() and v_new.is_contiguous() and slots.is_contiguous()):
        _want(where, device, _BF16, k_new, v_new)
        _want(where, device, _I64, slots)
    shape, of_k, of_v = u[6], k_new.shape, v_new.shape
    if (of_k != of_v or of_k != (n, shape[1], shape[-1])) and \
            (min(k_new.numel(), v_new.numel()) < n * shape[1] * shape[-1] or
             of_k[-1] != shape[-1] or of_v[-1] != shape[-1]) or slots.numel() < n:
        raise AttnError(ATTN_ERR_SHAPE, f"{where}: k_new and v_new are [n, {shape[1]}, "
                                        f"{shape[-1]}], slot_mapping [n]")
    return u[7]


def _want_decode(where, cache, q, out, seq_lens, positions, workspace):
    """What a decode over a scaled cache, or under a window with sinks, reads and
    writes; returns the cache's C structure's bytes."""
    device = _device()
    B, R, _, D = shape = q.shape
    c = cache._with_table(where, device, B)
    if not (q.dtype is out.dtype is _BF16 and seq_lens.dtype is positions.dtype is _I32 and
            q.get_device() == out.get_device() == seq_lens.get_device() ==
            positions.get_device() == workspace.get_device() == device and
            q.is_contiguous() and out.is_contiguous() and seq_lens.is_contiguous() and
            positions.is_contiguous() and workspace.is_contiguous()):
        _want(where, device, _BF16, q, out)
        _want(where, device, _I32, seq_lens, positions)
        _want(where, device, workspace.dtype, workspace)
    if seq_lens.numel() < B or positions.numel() < B * R or D != cache.head_dim or \
            (out is not q and out.shape != shape and out.numel() < q.numel()):
        raise AttnError(ATTN_ERR_SHAPE, f"{where}: q and out are [B, R, n_q_heads, "
                                        f"{cache.head_dim}], seq_lens [B], positions [B * R]")
    return c


def attn_kv_append(k_new, v_new, slot_mapping, cache: KVCache, err=None, stream=None):
    """cache.k[slot_mapping[i]] = k_new[i] (same for v); slot_mapping int64 [n]."""
    n, shape = slot_mapping.shape[0], cache.k.shape
    c = _want_new_rows("attn_kv_append", cache, k_new, v_new, slot_mapping, n) \
        if cache.dtype in _SCALED else cache.packed()
    rc = lib().attn_kv_append(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), n, c, shape[1],
                              shape[-1],
                              _ptr(err), _stream(stream))
    _check(rc, "attn_kv_append")


def attn_kv_reference(k, ref=None, stream=None):
    """Per-head mean of bf16 keys k [n, Hkv, D] as float32 [Hkv, D] (the FP8
    cache's reference vector).  Writes into ref if given."""
    n, Hkv, D = k.shape
    if ref is None:
        ref = torch.empty(Hkv, D, dtype=torch.float32, device=k.device)
    rc = lib().attn_kv_reference(_ptr(k), n, Hkv, D, _ptr(ref), _stream(stream))
    _check(rc, "attn_kv_reference")
    return ref


def attn_decode_workspace_size(cache: KVCache, batch, q_rows, n_q_heads, max_seq_len,
                               window=0) -> int:
    c = cache.packed()
    n = lib().attn_decode_workspace_size(c, batch, q_rows, n_q_heads,
                                         cache.n_kv_heads, cache.head_dim, max_seq_len, window)
    if n == ctypes.c_size_t(-1).value:
        raise AttnError(ATTN_ERR_SHAPE, "attn_decode_workspace_size")
    return int(n)


def attn_decode_kernel_launches(cache: KVCache, batch, q_rows, n_q_heads, max_seq_len,
                                window=0, with_append=False, with_rope=False,
                                tables_early=False) -> int:
    """Kernels one attn_decode (with_append: attn_decode_append; with_rope:
    with a rotary embedding; tables_early: with ATTN_DECODE_TABLES_EARLY)
    call of this shape launches (host-side plan; nothing runs on the device)."""
    c = cache.packed()
    n = lib().attn_decode_kernel_launches(c, batch, q_rows, n_q_heads,
                                          cache.n_kv_heads, cache.head_dim, max_seq_len, window,
                                          int(bool(with_append)), int(bool(with_rope)),
                                          ATTN_DECODE_TABLES_EARLY if tables_early else 0)
    if n < 0:
        raise AttnError(ATTN_ERR_SHAPE, "attn_decode_kernel_launches")
    return int(n)


def attn_decode(q, cache: KVCache, seq_lens, positions, max_seq_len, window, scale, out=None,
                workspace=None, err=None, stream=None):
    """Decode attention.  q bf16 [B, R, Hq, D]; seq_lens int32 [B]; positions int32 [B*R].
    Returns out (bf16 [B, R, Hq, D]).  A workspace (zero-filled uint8 device
    tensor of at least attn_decode_workspace_size bytes) is allocated if not
    given; one kept across calls needs no clearing."""
    B, R, Hq, D = q.shape
    if out is None:
        out = _made(torch.empty_like, q, stream)
    if workspace is None:
        need = attn_decode_workspace_size(cache, B, R, Hq, max_seq_len, window)
        if need > 0:
            workspace = _made(_zeroed, q, stream, need)
    c = _want_decode("attn_decode", cache, q, out, seq_lens, positions, workspace) \
        if cache.dtype in _SCALED and workspace is not None else cache.packed()
    rc = lib().attn_decode(_ptr(q), c, _ptr(seq_lens), _ptr(positions), B, R,
                           int(max_seq_len), int(window), Hq, cache.n_kv_heads, D, float(scale),
                           _ptr(out), _ptr(workspace),
                           0 if workspace is None else workspace.nbytes,
                           _ptr(err), _stream(stream))
    _check(rc, "attn_decode")
    return out


def attn_decode_append(q, k_new, v_new, slot_mapping, cache: KVCache, seq_lens, positions,
                       max_seq_len, window, scale, out=None, workspace=None, err=None,
                       stream=None, rope_inv_freq=None, tables_early=False, cache_early=False):
    """The step's KV append and its decode in one launch: same result as
    attn_kv_append(k_new, v_new, slot_mapping, cache) then attn_decode(...)
    when new row b*R + r is the key at position seq_lens[b] - R + r.
    k_new / v_new bf16 [B*R, Hkv, D]; slot_mapping int64 [B*R].  With
    rope_inv_freq (float32 [D/2] on the device), q and k_new are first rotated
    at their positions (interleaved pairs).  tables_early: seq_lens,
    positions and the block table were not written by the kernel launched
    just before on this stream (ATTN_DECODE_TABLES_EARLY); cache_early: nor
    are the cache's other rows (ATTN_DECODE_CACHE_EARLY, implies tables_early)."""
    B, R, Hq, D = q.shape
    if out is None:
        out = _made(torch.empty_like, q, stream)
    if workspace is None:
        need = attn_decode_workspace_size(cache, B, R, Hq, max_seq_len, window)
        if need > 0:
            workspace = _made(_zeroed, q, stream, need)
    if cache.dtype in _SCALED and workspace is not None:
        c = _want_decode("attn_decode_append", cache, q, out, seq_lens, positions, workspace)
        _want_new_rows("attn_decode_append", cache, k_new, v_new, slot_mapping, B * R)
    else:
        c = cache.packed()
    rc = lib().attn_decode_append(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(slot_mapping), _ptr(rope_inv_freq),
        c, _ptr(seq_lens),
        _ptr(positions), B, R, int(max_seq_len), int(window), Hq, cache.n_kv_heads, D,
        float(scale), _ptr(out), _ptr(workspace),
        0 if workspace is None else workspace.nbytes, _ptr(err),
        (ATTN_DECODE_TABLES_EARLY if tables_early else 0) |
        (ATTN_DECODE_CACHE_EARLY if cache_early else 0), _stream(stream))
    _check(rc, "attn_decode_append")
    return out


def attn_prefill(q, k, v, window, scale, out=None, err=None, stream=None):
    """Causal prefill.  q bf16 [B, T, Hq, D], k/v bf16 [B, T, Hkv, D] -> out [B, T, Hq, D]."""
    B, T, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    rc = lib().attn_prefill(_ptr(q), _ptr(k), _ptr(v), B, T, int(window), Hq, k.shape[2], D,
                            float(scale), _ptr(out), _ptr(err), _stream(stream))
    _check(rc, "attn_prefill")
    return out


def attn_decode_noalloc(q, cache: KVCache, seq_lens, positions, max_seq_len, window, scale,
                        out=None, err=None, stream=None):
    """attn_decode without a workspace argument, for callers that cannot
    allocate device memory: the library uses its own fixed scratch array
    (ATTN_DECODE_NOALLOC_SCRATCH_BYTES per GPU).  Calls that overlap on the
    GPU share that array and race; order them on one stream."""
    f = lib().attn_decode_noalloc
    B, R, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    c = cache.packed()
    rc = f(_ptr(q), c, _ptr(seq_lens), _ptr(positions), B, R, int(max_seq_len),
           int(window), Hq, cache.n_kv_heads, D, float(scale), _ptr(out), _ptr(err),
           _stream(stream))
    _check(rc, "attn_decode_noalloc")
    return out


def attn_decode_sinks_workspace_size(cache: KVCache, batch, q_rows, n_q_heads, max_seq_len,
                                     window, n_sinks) -> int:
    c = cache.packed()
    n = lib().attn_decode_sinks_workspace_size(c, batch, q_rows, n_q_heads,
                                               cache.n_kv_heads, cache.head_dim, max_seq_len,
                                               window, n_sinks)
    if n == ctypes.c_size_t(-1).value:
        raise AttnError(ATTN_ERR_SHAPE, "attn_decode_sinks_workspace_size")
    return int(n)


def attn_decode_sinks(q, cache: KVCache, seq_lens, positions, max_seq_len, window, n_sinks, scale,
                      out=None, workspace=None, err=None, stream=None):
    """attn_decode under a sliding window whose first n_sinks tokens stay
    visible: a row at position pos attends t <= pos with t < n_sinks or
    pos - t < window (window <= 0: every t).  RING caches keep the sinks in
    each request's first n_sinks slots and turn the others.  A workspace (at
    least attn_decode_sinks_workspace_size bytes, zero-filled before its first
    use) is allocated if not given."""
    B, R, Hq, D = q.shape
    if out is None:
        out = _made(torch.empty_like, q, stream)
    if workspace is None:
        need = attn_decode_sinks_workspace_size(cache, B, R, Hq, max_seq_len, window, n_sinks)
        if need > 0:
            workspace = _made(_zeroed, q, stream, need)
    c = _want_decode("attn_decode_sinks", cache, q, out, seq_lens, positions, workspace) \
        if workspace is not None else cache.packed()
    rc = lib().attn_decode_sinks(
        _ptr(q), c, _ptr(seq_lens), _ptr(positions), B, R, int(max_seq_len),
        int(window), int(n_sinks), Hq, cache.n_kv_heads, D, float(scale), _ptr(out),
        _ptr(workspace),
        0 if workspace is None else workspace.nbytes, _ptr(err),
        _stream(stream))
    _check(rc, "attn_decode_sinks")
    return out


def attn_prefill_sinks(q, k, v, window, n_sinks, scale, out=None, err=None, stream=None):
    """attn_prefill under a sliding window whose first n_sinks tokens of each
    sequence stay visible.  Shapes as attn_prefill's."""
    B, T, Hq, D = q.shape
    if out is None:
        out = _made(torch.empty_like, q, stream)
    _want("attn_prefill_sinks", _device(), torch.bfloat16, q, k, v, out)
    if k.shape != v.shape or k.shape[:2] != q.shape[:2] or k.shape[3] != D:
        raise AttnError(ATTN_ERR_SHAPE, "attn_prefill_sinks: k and v are [B, T, Hkv, D]")
    rc = lib().attn_prefill_sinks(_ptr(q), _ptr(k), _ptr(v), B, T, int(window), int(n_sinks), Hq,
                                  k.shape[2], D, float(scale), _ptr(out), _ptr(err),
                                  _stream(stream))
    _check(rc, "attn_prefill_sinks")
    return out


def attn_decode_shared_workspace_size(cache: KVCache, batch, q_rows, n_q_heads, max_seq_len,
                                      max_prefix_len, window=0) -> int:
    n = lib().attn_decode_shared_workspace_size(cache.packed(), batch, q_rows, n_q_heads,
                                                cache.n_kv_heads, cache.head_dim, max_seq_len,
                                                max_prefix_len, window)
    if n == ctypes.c_size_t(-1).value:
        raise AttnError(ATTN_ERR_SHAPE, "attn_decode_shared_workspace_size")
    return int(n)


def attn_decode_shared(q, cache: KVCache, seq_lens, positions, prefix_rows, prefix_lens,
                       max_seq_len, max_prefix_len, window, scale, out=None, workspace=None,
                       err=None, stream=None):
    """attn_decode for a batch whose requests share prefixes: key position
    t < prefix_lens[b] of request b is read where row prefix_rows[b] (of the
    block table, or a window of a linear cache) has it, once for all
    neighbouring requests with that row and length.  prefix_rows, prefix_lens
    int32 [B]; max_prefix_len bounds the lengths (it and max_seq_len decide how the
    GPU is shared out: loose bounds cost time).  Worth it for 16 requests from about
    2,000 shared bf16 keys on, for 64 from 500.  A workspace (at least
    attn_decode_shared_workspace_size bytes, zero-filled before its first use)
    is allocated if not given."""
    B, R, Hq, D = q.shape
    if out is None:
        out = _made(torch.empty_like, q, stream)
    if workspace is None:
        need = attn_decode_shared_workspace_size(cache, B, R, Hq, max_seq_len, max_prefix_len,
                                                 window)
        if need > 0:
            workspace = _made(_zeroed, q, stream, need)
    if workspace is not None:
        c = _want_decode("attn_decode_shared", cache, q, out, seq_lens, positions, workspace)
        if not (prefix_rows.dtype is prefix_lens.dtype is _I32 and
                prefix_rows.get_device() == prefix_lens.get_device() == q.get_device() and
                prefix_rows.is_contiguous() and prefix_lens.is_contiguous()):
            _want("attn_decode_shared", _device(), _I32, prefix_rows, prefix_lens)
        if prefix_rows.numel() < B or prefix_lens.numel() < B:
            raise AttnError(ATTN_ERR_SHAPE, "attn_decode_shared: prefix_rows and prefix_lens are "
                                            "[B]")
    else:
        c = cache.packed()
    if cache.kind == PAGED:
        t = cache.block_table
        n_rows = 0 if t is None else t.numel() // max(1, t.shape[-1])
    else:
        n_rows = min(cache.num_slots // max(1, cache.slots_per_seq), (1 << 31) - 1)
    rc = lib().attn_decode_shared(
        _ptr(q), c, n_rows, _ptr(seq_lens), _ptr(positions), _ptr(prefix_rows),
        _ptr(prefix_lens), B, R, int(max_seq_len), int(max_prefix_len), int(window), Hq,
        cache.n_kv_heads, D, float(scale), _ptr(out), _ptr(workspace),
        0 if workspace is None else workspace.nbytes, _ptr(err), _stream(stream))
    _check(rc, "attn_decode_shared")
    return out


def rope_frequencies(rot_dim, base=10000.0, scaling=None, factor=1.0, original_len=0,
                     beta_fast=32.0, beta_slow=1.0, device=None):
    """(inv_freq, factor) of a Rope: base ** (-2 i / rot_dim), i < rot_dim / 2, as
    float32 on `device`, changed for contexts `factor` times as long as a model was
    trained on by `scaling`:
      None      as they are
      "linear"  all divided by factor (positions interpolated)
      "ntk"     base * factor ** (rot_dim / (rot_dim - 2)), so that the slowest is
                divided by factor and the fastest keeps its value
      "yarn"    those that turn less than beta_slow times in original_len tokens
                divided by factor, those that turn more than beta_fast times kept, a
                linear ramp between (over i), and cosines and sines times
                0.1 ln(factor) + 1 (YaRN, arXiv 2309.00071)"""
    half = rot_dim // 2
    if rot_dim < 0 or rot_dim % 2 or not base > 1 or not factor > 0 or \
            scaling not in (None, "linear", "ntk", "yarn") or \
            (scaling == "ntk" and rot_dim < 4) or \
            (scaling == "yarn" and not (original_len > 0 and factor >= 1 and
                                        beta_fast > beta_slow > 0)):
        raise AttnError(ATTN_ERR_SHAPE, "rope_frequencies")
    i = torch.arange(half, dtype=torch.float64)
    times = 1.0
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    inv = float(base) ** (-i / max(1, half))
    if scaling == "linear":
        inv = inv / factor
    elif scaling == "yarn":
        def turns_at(turns):  # the (fractional) i that turns so often in original_len
            return half * math.log(original_len / (turns * 2 * math.pi)) / math.log(base)

        lo = max(math.floor(turns_at(beta_fast)), 0)
        hi = max(min(math.ceil(turns_at(beta_slow)), rot_dim - 1), lo + 1e-3)
        slow = ((i - lo) / (hi - lo)).clamp(0, 1)
        inv = inv * (1 - slow) + inv / factor * slow
        times = 0.1 * math.log(factor) + 1.0
    return inv.float().to(device), times


class Rope:
    """What attn_qk_rope does to a head's rows: rotary embedding of the first
    2 * len(inv_freq) dims (inv_freq float32 on the device, None: no rotation),
    paired as layout says, cosines and sines times factor; RMS norms with q_weight
    and k_weight (float32 [head_dim], None: not normalised) and eps."""

    def __init__(self, inv_freq, layout=ATTN_ROPE_HALF, factor=1.0, q_weight=None, k_weight=None,
                 eps=1e-6):
        self.inv_freq, self.layout, self.factor = inv_freq, int(layout), float(factor)
        self.q_weight, self.k_weight, self.eps = q_weight, k_weight, float(eps)

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        self.__dict__["_usable"] = None  # looked at again by the next call

    @property
    def rot_dim(self):
        return 0 if self.inv_freq is None else 2 * self.inv_freq.numel()

    def _packed(self, where, device, head_dim):
        """The bytes of an attn_rope, its tensors looked at again when one is set or put
        elsewhere."""
        u, f, q, k = self._usable, self.inv_freq, self.q_weight, self.k_weight
        at = (device, head_dim, 0 if f is None else f.data_ptr(),
              0 if q is None else q.data_ptr(), 0 if k is None else k.data_ptr(),
              0 if f is None else f.nbytes)
        if u is None or u[0] != at:
            _want(where, device, torch.float32, *(t for t in (f, q, k) if t is not None))
            for t in (q, k):
                if t is not None and t.numel() != head_dim:
                    raise AttnError(ATTN_ERR_SHAPE,
                                    f"{where}: q_weight and k_weight are [{head_dim}]")
            u = (at, _PACK_ROPE(at[2], self.rot_dim, self.layout, self.factor, at[3], at[4],
                                self.eps))
            self.__dict__["_usable"] = u
        return u[1]


def _want_heads(where, device, n, dim, *tensors):
    """Refuses q, k or v that are not bf16 rows [n, heads, head_dim] whose heads stand
    next to each other; returns the strides of their tokens."""
    strides = []
    for t in tensors:
        if t.dtype is not _BF16 or t.get_device() != device or t.dim() != 3:
            raise AttnError(ATTN_ERR_UNSUPPORTED, f"{where}: q, k and v are bf16 [n, heads, "
                                                  "head_dim] on the current device")
        rows, heads, last = t.shape
        if rows != n or last != dim:
            raise AttnError(ATTN_ERR_SHAPE, f"{where}: q, k and v have n rows and one head_dim")
        step, of_head, of_dim = t.stride()
        if n and ((dim > 1 and of_dim != 1) or (heads > 1 and of_head != dim)):
            raise AttnError(ATTN_ERR_UNSUPPORTED, f"{where}: a token's heads are not contiguous")
        strides.append(step if n > 1 else heads * dim)
    return strides


def _new_like(t, shape):
    return torch.empty(shape, dtype=t.dtype, device=t.device)


def attn_qk_rope(q, k, positions, rope: Rope, q_out=None, k_out=None, stream=None):
    """Norms and rotary embedding of q bf16 [n, Hq, D] and k bf16 [n, Hkv, D] at
    positions int32 [n] (what Rope says, in one pass).  The tokens of q and k may be
    any stride apart (views of a fused projection).  Returns (q_out, k_out),
    contiguous; either may be its input (in place)."""
    where, device = "attn_qk_rope", _device()
    of_q, of_k = q.shape, k.shape
    if len(of_q) != 3 or len(of_k) != 3:
        raise AttnError(ATTN_ERR_SHAPE, f"{where}: q and k are [n, heads, head_dim]")
    n, Hq, D = of_q
    qs, ks = _want_heads(where, device, n, D, q, k)
    if q_out is None:
        q_out = _made(_new_like, q, stream, of_q)
    if k_out is None:
        k_out = _made(_new_like, k, stream, of_k)
    if not (q_out.dtype is k_out.dtype is _BF16 and positions.dtype is _I32 and
            q_out.get_device() == k_out.get_device() == positions.get_device() == device and
            q_out.is_contiguous() and k_out.is_contiguous() and positions.is_contiguous()):
        _want(where, device, _BF16, q_out, k_out)
        _want(where, device, _I32, positions)
    if q_out.shape != of_q or k_out.shape != of_k or positions.numel() < n:
        raise AttnError(ATTN_ERR_SHAPE, f"{where}: q_out and k_out are shaped like q and k, "
                                        "positions is [n]")
    rc = lib().attn_qk_rope(q.data_ptr(), qs, k.data_ptr(), ks, positions.data_ptr(), n,
                            rope._packed(where, device, D), Hq, of_k[1], D, q_out.data_ptr(),
                            k_out.data_ptr(), _stream(stream))
    _check(rc, where)
    return q_out, k_out


def attn_qk_rope_append(q, k, v, positions, slot_mapping, cache: KVCache, rope: Rope, q_out=None,
                        k_out=None, err=None, stream=None):
    """attn_qk_rope, then attn_kv_append of the new keys and of v bf16 [n, Hkv, D]
    at slot_mapping int64 [n], in one launch (two for caches with scales).  k_out, if
    given, receives the new keys too.  Returns q_out."""
    where, device = "attn_qk_rope_append", _device()
    of_q, of_k = q.shape, k.shape
    if len(of_q) != 3 or len(of_k) != 3:
        raise AttnError(ATTN_ERR_SHAPE, f"{where}: q and k are [n, heads, head_dim]")
    n, Hq, D = of_q
    scaled = cache.dtype in _SCALED
    if scaled and n > 1 and not v.is_contiguous():
        v = _made(torch.Tensor.contiguous, v, stream)
    qs, ks, vs = _want_heads(where, device, n, D, q, k, v)
    if q_out is None:
        q_out = _made(_new_like, q, stream, of_q)
    if k_out is None and scaled:
        k_out = _made(_new_like, k, stream, of_k)
    if not (q_out.dtype is _BF16 and positions.dtype is _I32 and slot_mapping.dtype is _I64 and
            q_out.get_device() == positions.get_device() == slot_mapping.get_device() == device and
            q_out.is_contiguous() and positions.is_contiguous() and slot_mapping.is_contiguous()):
        _want(where, device, _BF16, q_out)
        _want(where, device, _I32, positions)
        _want(where, device, _I64, slot_mapping)
    if k_out is not None:
        _want(where, device, _BF16, k_out)
    known = cache._known(where, device)
    _want_ref(where, cache, device)
    if of_k != v.shape or of_k[1] != known[6][1] or D != known[6][-1]:
        raise AttnError(ATTN_ERR_SHAPE, f"{where}: k and v are [n, {known[6][1]}, {known[6][-1]}]")
    if q_out.shape != of_q or (k_out is not None and k_out.shape != of_k) or \
            positions.numel() < n or slot_mapping.numel() < n:
        raise AttnError(ATTN_ERR_SHAPE, f"{where}: q_out and k_out are shaped like q and k, "
                                        "positions and slot_mapping are [n]")
    rc = lib().attn_qk_rope_append(
        q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, positions.data_ptr(),
        slot_mapping.data_ptr(), n, rope._packed(where, device, D), known[7], Hq, of_k[1], D,
        q_out.data_ptr(), _ptr(k_out), _ptr(err), _stream(stream))
    _check(rc, where)
    return q_out


def attn_kv_read(slot_mapping, cache: KVCache, k_out=None, v_out=None, err=None, stream=None):
    """(k_out, v_out) bf16 [n, Hkv, D]: the cache's rows at slot_mapping int64 [n], for
    8-bit caches the values of their codes (keys plus k_ref).  Slots outside the cache
    give zeros and ATTN_ERR_BOUNDS in err."""
    where, device = "attn_kv_read", _device()
    known = cache._known(where, device)
    _want_ref(where, cache, device)
    if not (slot_mapping.dtype is _I64 and slot_mapping.get_device() == device and
            slot_mapping.is_contiguous()):
        _want(where, device, _I64, slot_mapping)
    shape = (slot_mapping.numel(), known[6][1], known[6][-1])
    if k_out is None:
        k_out = _made(_rows_like, slot_mapping, stream, shape)
    if v_out is None:
        v_out = _made(_rows_like, slot_mapping, stream, shape)
    if not (k_out.dtype is v_out.dtype is _BF16 and
            k_out.get_device() == v_out.get_device() == device and
            k_out.is_contiguous() and v_out.is_contiguous()):
        _want(where, device, _BF16, k_out, v_out)
    if k_out.shape != shape or v_out.shape != shape:
        raise AttnError(ATTN_ERR_SHAPE, f"{where}: k_out and v_out are {shape}")
    rc = lib().attn_kv_read(slot_mapping.data_ptr(), shape[0], known[7], shape[1], shape[2],
                            k_out.data_ptr(), v_out.data_ptr(), _ptr(err), _stream(stream))
    _check(rc, where)
    return k_out, v_out


def _want_ref(where, cache, device):
    """The reference vector of an unscaled E4M3 cache (a scaled one's is looked at with
    its scales)."""
    if cache.dtype == ATTN_KV_FP8_E4M3 and cache.k_ref is not None:
        _want(where, device, torch.float32, cache.k_ref)
        if cache.k_ref.numel() != cache.n_kv_heads * cache.head_dim:
            raise AttnError(ATTN_ERR_SHAPE, f"{where}: k_ref is [n_kv_heads, head_dim]")


def _rows_like(t, shape):
    return torch.empty(shape, dtype=_BF16, device=t.device)


def _want_rows(where, block_table, refs, rows, a, b):
    _want(where, _device(), torch.int32, block_table, refs, rows, a, b)
    if block_table.dim() != 2 or not rows.shape == a.shape == b.shape:
        raise AttnError(ATTN_ERR_SHAPE, f"{where}: block_table is [rows, max_blocks], the row "
                                        "arguments are of one length")


def _want_moves(where, moves, n_moves):
    _want(where, _device(), torch.int32, moves, n_moves)
    if moves.dim() != 2 or moves.shape[1] != 3 or n_moves.numel() < 1:
        raise AttnError(ATTN_ERR_SHAPE, f"{where}: moves is [n, 3], n_moves [1]")


def attn_pages_free(block_table, refs, rows, from_block, to_block, err=None, stream=None):
    """Entries from_block[i] .. to_block[i] - 1 of row rows[i] of block_table
    (int32 [table_rows, max_blocks]) give their page back (refs, int32
    [num_pages], counts a page's entries) and become -1.  rows, from_block,
    to_block: int32 [n] on the device."""
    _want_rows("attn_pages_free", block_table, refs, rows, from_block, to_block)
    rc = lib().attn_pages_free(_ptr(block_table), block_table.shape[1], block_table.shape[0],
                               _ptr(rows), _ptr(from_block), _ptr(to_block), rows.shape[0],
                               _ptr(refs), refs.shape[0], _ptr(err), _stream(stream))
    _check(rc, "attn_pages_free")


def attn_pages_reserve(block_table, refs, rows, from_block, to_block, err=None, stream=None):
    """Entries from_block[i] .. to_block[i] - 1 of row rows[i] that are -1 take
    the lowest free pages (refs 0), in order.  ATTN_ERR_PAGES in err when the
    pool runs out."""
    _want_rows("attn_pages_reserve", block_table, refs, rows, from_block, to_block)
    rc = lib().attn_pages_reserve(_ptr(block_table), block_table.shape[1], block_table.shape[0],
                                  _ptr(rows), _ptr(from_block), _ptr(to_block), rows.shape[0],
                                  _ptr(refs), refs.shape[0], _ptr(err), _stream(stream))
    _check(rc, "attn_pages_reserve")


def attn_pages_fork(block_table, refs, src_rows, dst_rows, seq_lens, block_size, moves, n_moves,
                    err=None, stream=None):
    """Row dst_rows[i] becomes the first seq_lens[i] tokens of row src_rows[i]:
    full pages shared, a partial last page replaced by a free one.  moves (int32
    [at least n, 3]) and n_moves (int32 [1]) receive the copies to carry out
    with attn_pages_copy."""
    _want_rows("attn_pages_fork", block_table, refs, src_rows, dst_rows, seq_lens)
    _want_moves("attn_pages_fork", moves, n_moves)
    rc = lib().attn_pages_fork(_ptr(block_table), block_table.shape[1], block_table.shape[0],
                               _ptr(src_rows), _ptr(dst_rows), _ptr(seq_lens), src_rows.shape[0],
                               int(block_size), _ptr(refs), refs.shape[0], _ptr(moves),
                               moves.shape[0], _ptr(n_moves), _ptr(err), _stream(stream))
    _check(rc, "attn_pages_fork")


def attn_pages_workspace_size(num_pages) -> int:
    n = lib().attn_pages_workspace_size(int(num_pages))
    if n == ctypes.c_size_t(-1).value:
        raise AttnError(ATTN_ERR_SHAPE, "attn_pages_workspace_size")
    return int(n)


def attn_pages_compact(block_table, refs, block_size, moves, n_moves, used, workspace=None,
                       err=None, stream=None):
    """Pages in use move to the lowest page ids: block_table and refs follow,
    used (int32 [1]) receives how many pages are in use, moves / n_moves the
    copies to carry out with attn_pages_copy."""
    _want("attn_pages_compact", _device(), torch.int32, block_table, refs, used)
    _want_moves("attn_pages_compact", moves, n_moves)
    if block_table.dim() != 2 or used.numel() < 1:
        raise AttnError(ATTN_ERR_SHAPE, "attn_pages_compact: block_table is [rows, max_blocks]")
    if workspace is None:
        workspace = _made(_zeroed, refs, stream, attn_pages_workspace_size(refs.shape[0]))
    _want("attn_pages_compact", _device(), workspace.dtype, workspace)
    rc = lib().attn_pages_compact(_ptr(block_table), block_table.shape[1], block_table.shape[0],
                                  int(block_size), _ptr(refs), refs.shape[0], _ptr(moves),
                                  moves.shape[0], _ptr(n_moves), _ptr(used), _ptr(workspace),
                                  workspace.nbytes, _ptr(err),
                                  _stream(stream))
    _check(rc, "attn_pages_compact")


def attn_pages_copy(caches, moves, n_moves, err=None, stream=None):
    """Carries out n_moves (int32 [1], device) page copies listed in moves in
    each of the paged caches (a KVCache, or a list of them, one per layer)."""
    if isinstance(caches, KVCache):
        caches = [caches]
    _want_moves("attn_pages_copy", moves, n_moves)
    device, shape, packed = _device(), None, []
    for c in caches:
        known = c._known("attn_pages_copy", device)
        if shape is None:
            shape = known[6]
        elif known[6] != shape:
            raise AttnError(ATTN_ERR_SHAPE, "attn_pages_copy: caches of different shapes")
        packed.append(known[7])
    Hkv, D = (shape[1], shape[-1]) if shape else (1, 128)
    rc = lib().attn_pages_copy(b"".join(packed), len(packed), Hkv, D, _ptr(moves), _ptr(n_moves),
                               moves.shape[0], _ptr(err), _stream(stream))
    _check(rc, "attn_pages_copy")
