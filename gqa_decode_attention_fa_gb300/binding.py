"""Thin ctypes binding over libgqa_decode.so (include/gqa_decode.h, gqa_prefill.h, gqa_q4.h,
gqa_rope.h, gqa_tree.h, gqa_pages.h, gqa_q8.h,
gqa_packed.h).

Argument marshalling only: every step of the decode path runs in the library's CUDA
kernels.  Device tensors are torch tensors (device memory and streams come from torch);
host buffers are numpy arrays or CPU torch tensors.  ``load()`` raises if the library
cannot be loaded -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import os
import re
import threading
from typing import Optional

import numpy as np

from . import build as _build

(GQA_OK, GQA_ERR_INVALID_ARG, GQA_ERR_UNSUPPORTED, GQA_ERR_CUDA, GQA_ERR_WORKSPACE,
 GQA_ERR_SCRATCH_LIMIT) = range(6)
STATIC_SCRATCH_BYTES = 32 << 20
DEVERR_POSITION, DEVERR_SEQLEN, DEVERR_PAGE, DEVERR_TIMEOUT, DEVERR_LAUNCH = 0x1, 0x2, 0x4, 0x8, 0x10
DEVERR_NOPAGE, DEVERR_CONFLICT = 0x20, 0x40
MAX_TREE, MAX_POOLS, MAX_PAGE_PAIRS = 256, 256, 4096
HEADER = os.path.join(_build.ROOT, "include", "gqa_decode.h")
HEADERS = _build.HEADERS

_lock = threading.Lock()
_lib = None


class GqaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class PlanDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "batch", "num_q_heads", "num_kv_heads", "head_dim", "block_size", "max_seq_len",
        "num_cache_blocks", "num_workers", "device", "cluster_size", "ordered_start")]


class PrefillDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "batch", "num_q_heads", "num_kv_heads", "head_dim", "chunk_len", "block_size", "max_seq_len",
        "num_cache_blocks", "device")]


class RopeDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "batch", "num_q_heads", "num_kv_heads", "head_dim", "num_tokens", "block_size", "max_seq_len",
        "num_cache_blocks", "device", "q_stride", "k_stride", "v_stride")]


class TreeDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "batch", "num_q_heads", "num_kv_heads", "head_dim", "tree_len", "block_size", "max_seq_len",
        "num_cache_blocks", "device")]


class PagesDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("batch", "max_blocks", "num_blocks", "device")]


class KeepDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "batch", "max_keep", "max_seq_len", "block_size", "num_blocks", "device")]


class Q8Desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "batch", "num_q_heads", "num_kv_heads", "head_dim", "format", "num_tokens", "block_size", "max_seq_len",
        "num_cache_blocks", "device", "k_stride", "v_stride")]


class PackedDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "batch", "num_q_heads", "num_kv_heads", "head_dim", "num_queries", "num_keys", "causal", "device", "q_stride",
        "k_stride", "v_stride")]


class Pool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("row_bytes", ctypes.c_longlong)]


class Rope(ctypes.Structure):
    """A rotary embedding (gqa_rope_t, include/gqa_rope.h): layout "half" or "interleaved",
    scaling None, "linear", "banded", "yarn" or "custom" (with ``freqs``, one per pair)."""

    _fields_ = [("layout", ctypes.c_int), ("rotary_dim", ctypes.c_int), ("scaling", ctypes.c_int),
                ("original_max_len", ctypes.c_int), ("theta", ctypes.c_float), ("factor", ctypes.c_float),
                ("low_freq_factor", ctypes.c_float), ("high_freq_factor", ctypes.c_float),
                ("beta_fast", ctypes.c_float), ("beta_slow", ctypes.c_float), ("magnitude", ctypes.c_float),
                ("freqs", ctypes.c_void_p)]
    LAYOUTS = {"half": 0, "interleaved": 1}
    SCALINGS = {None: 0, "linear": 1, "banded": 2, "yarn": 3, "custom": 4}

    def __init__(self, theta: float = 1e6, rotary_dim: int = 128, layout: str = "half", scaling: Optional[str] = None,
                 factor: float = 1.0, low_freq_factor: float = 1.0, high_freq_factor: float = 4.0,
                 beta_fast: float = 32.0, beta_slow: float = 1.0, original_max_len: int = 0, magnitude: float = 0.0,
                 freqs=None):
        if layout not in self.LAYOUTS or scaling not in self.SCALINGS:
            raise ValueError(f"rope layout {layout!r} or scaling {scaling!r} is not known")
        self._freqs = None if freqs is None else np.ascontiguousarray(np.asarray(freqs, dtype=np.float64))
        if self._freqs is not None and self._freqs.shape != (int(rotary_dim) // 2,):
            raise ValueError("freqs: one frequency per pair, [rotary_dim / 2]")
        super().__init__(self.LAYOUTS[layout], int(rotary_dim), self.SCALINGS[scaling], int(original_max_len),
                         float(theta), float(factor), float(low_freq_factor), float(high_freq_factor),
                         float(beta_fast), float(beta_slow), float(magnitude),
                         None if self._freqs is None else self._freqs.ctypes.data)

    def frequencies(self):
        """([rotary_dim / 2] float64 frequencies after scaling, magnitude): gqa_rope_freqs."""
        out, mag = np.zeros(max(0, self.rotary_dim // 2)), ctypes.c_double()
        _check(load().gqa_rope_freqs(ctypes.byref(self), out.ctypes.data, ctypes.byref(mag)), "gqa_rope_freqs")
        return out, mag.value


def header_functions() -> list:
    """Names of the functions the headers under include/ declare."""
    names = set()
    for path in HEADERS:
        text = re.sub(r"/\*.*?\*/", "", open(path).read(), flags=re.S)
        names.update(re.findall(r"\b(gqa_[a-z0-9_]+)\s*\(", text))
    return sorted(names)


def load(build: bool = True):
    """Load the library (building it first when stale); raises on failure."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.build() if build else _build.LIB
        if not os.path.exists(path):
            raise RuntimeError(f"libgqa_decode.so is missing ({path}); build it with "
                               "gqa_decode_attention_fa_gb300.build.build()")
        lib = ctypes.CDLL(path)
        P, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        lib.gqa_plan_create.argtypes = [ctypes.POINTER(PlanDesc), P, ctypes.POINTER(P)]
        lib.gqa_plan_destroy.argtypes = [P]
        lib.gqa_plan_num_workers.argtypes = [P]
        lib.gqa_plan_num_workers.restype = I
        lib.gqa_plan_describe.argtypes = [ctypes.POINTER(PlanDesc), P, I, P, P, P, P]
        lib.gqa_plan_describe.restype = I
        lib.gqa_plan_set_ordered_start.argtypes = [P, I]
        lib.gqa_plan_set_ordered_start.restype = I
        lib.gqa_plan_num_splits.argtypes = [P]
        lib.gqa_plan_num_splits.restype = I
        lib.gqa_plan_cluster_size.argtypes = [P]
        lib.gqa_plan_cluster_size.restype = I
        lib.gqa_plan_workspace_bytes.argtypes = [P]
        lib.gqa_plan_workspace_bytes.restype = ctypes.c_size_t
        step = [P, P, P, P, P, P, P, P, P, P, P, F, F]
        lib.gqa_decode_attn.argtypes = step + [P, P]
        lib.gqa_decode_attn_host.argtypes = step + [P, P]
        lib.gqa_attention_splitkv.argtypes = [P, P, P, P, P, P, P, P, P, P, P, F, F, P]
        lib.gqa_combine.argtypes = [P, P, P, P]
        lib.gqa_plan_read_q_rot.argtypes = [P, P]
        lib.gqa_plan_device_errors.argtypes = [P, ctypes.POINTER(ctypes.c_uint32), I]
        lib.gqa_partition_describe.argtypes = [P, I, I, I, I, P]
        lib.gqa_partition_describe.restype = ctypes.c_longlong
        lib.gqa_decode_attn_static.argtypes = [ctypes.POINTER(PlanDesc)] + step[1:] + [P, P, P]
        lib.gqa_prefill_attn.argtypes = [ctypes.POINTER(PrefillDesc)] + [P] * 9 + [F, F, P, P, P]
        lib.gqa_q4_codebook.argtypes = [P]
        lib.gqa_decode_attn_q4.argtypes = [P] * 15 + [F, F, P, P]
        lib.gqa_rope_freqs.argtypes = [P, P, P]
        lib.gqa_rope_append.argtypes = [P] * 13 + [F, P, P, P]
        lib.gqa_tree_prepare.argtypes = [I, I, P, P, P, P, P, I, P, P]
        lib.gqa_tree_workspace_bytes.argtypes = [P, P]
        lib.gqa_tree_attn.argtypes = [P] * 12
        lib.gqa_pages_fork.argtypes = [P] * 6 + [I, P, P]
        lib.gqa_pages_resize.argtypes = [P] * 9
        lib.gqa_pages_copy.argtypes = [P, I, I, P, P, I, I, P, P]
        lib.gqa_cache_keep_rows.argtypes = [P, P, I] + [P] * 6
        lib.gqa_q8_append.argtypes = [P] * 12
        lib.gqa_q8_read.argtypes = [P] * 12
        lib.gqa_q8_workspace_bytes.argtypes = [P, P]
        lib.gqa_q8_attn.argtypes = [P] * 12
        lib.gqa_packed_attn.argtypes = [P] * 9
        lib.gqa_status_string.argtypes = [I]
        lib.gqa_status_string.restype = ctypes.c_char_p
        for name in ("gqa_plan_create", "gqa_plan_destroy", "gqa_decode_attn", "gqa_decode_attn_host",
                     "gqa_attention_splitkv", "gqa_combine", "gqa_plan_read_q_rot",
                     "gqa_plan_device_errors", "gqa_decode_attn_static", "gqa_prefill_attn", "gqa_q4_codebook",
                     "gqa_decode_attn_q4", "gqa_rope_freqs", "gqa_rope_append", "gqa_tree_prepare",
                     "gqa_tree_workspace_bytes", "gqa_tree_attn", "gqa_pages_fork", "gqa_pages_resize",
                     "gqa_pages_copy", "gqa_cache_keep_rows", "gqa_q8_append", "gqa_q8_read",
                     "gqa_q8_workspace_bytes", "gqa_q8_attn", "gqa_packed_attn"):
            getattr(lib, name).restype = I
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    try:
        return load(build=False).gqa_status_string(int(status)).decode()
    except Exception:  # noqa: BLE001 - only used to format an error message
        return "status"


def _check(status: int, what: str):
    if status != GQA_OK:
        raise GqaError(status, what)


def _dptr(t) -> Optional[int]:
    """Device pointer of a torch tensor (None passes NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return t.data_ptr()


def _hptr(a) -> Optional[int]:
    """Host pointer of a numpy array or CPU torch tensor."""
    if a is None:
        return None
    if isinstance(a, np.ndarray):
        if not a.flags["C_CONTIGUOUS"]:
            raise ValueError("expected a C-contiguous array")
        return a.ctypes.data
    if a.is_cuda or not a.is_contiguous():
        raise ValueError("expected a contiguous host tensor")
    return a.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return int(stream) if isinstance(stream, int) else stream.cuda_stream


def partition_describe(seq_lens, num_kv_heads: int, max_seq_len: int, num_workers: int):
    """Host view of the split-KV partition: (total tiles, [W, 2] worker ranges)."""
    sl = np.ascontiguousarray(np.asarray(seq_lens, dtype=np.int32))
    rng = np.zeros((num_workers, 2), dtype=np.int64)
    T = load().gqa_partition_describe(sl.ctypes.data, len(sl), int(num_kv_heads), int(max_seq_len),
                                      int(num_workers), rng.ctypes.data)
    if T < 0:
        raise ValueError("bad partition arguments")
    return int(T), rng


GB300_SMS = 152
# clusters of 1, 2, ..., 16 single-launch CTAs resident at once on GB300 (cudaOccupancyMaxActiveClusters)
GB300_CLUSTER_CAPACITY = (152, 76, 46, 36, 28, 23, 15, 15, 15, 13, 8, 8, 7, 7, 7, 7)


def plan_describe(batch: int, num_q_heads: int, num_kv_heads: int, max_seq_len: int, *, block_size: int = 0,
                  num_cache_blocks: int = 0, num_workers: int = 0, cluster_size: int = 0, seq_lens_host=None,
                  num_sms: int = GB300_SMS, cluster_capacity=GB300_CLUSTER_CAPACITY, head_dim: int = 128,
                  ordered_start: bool = False):
    """The planner's choices without a GPU (gqa_plan_describe): (workers, cluster size, splits)."""
    desc = PlanDesc(int(batch), int(num_q_heads), int(num_kv_heads), int(head_dim), int(block_size),
                    int(max_seq_len), int(num_cache_blocks), int(num_workers), 0, int(cluster_size),
                    int(bool(ordered_start)))
    sl = None if seq_lens_host is None else np.ascontiguousarray(np.asarray(seq_lens_host, dtype=np.int32))
    cap = np.ascontiguousarray(np.asarray(cluster_capacity, dtype=np.int32))
    if cap.shape != (16,):
        raise ValueError("cluster_capacity: 16 counts, for clusters of 1 .. 16 CTAs")
    out = np.zeros(3, dtype=np.int32)
    _check(load().gqa_plan_describe(ctypes.byref(desc), None if sl is None else sl.ctypes.data, int(num_sms),
                                    cap.ctypes.data, out[0:].ctypes.data, out[1:].ctypes.data,
                                    out[2:].ctypes.data), "gqa_plan_describe")
    return int(out[0]), int(out[1]), int(out[2])


def decode_attn_static(batch: int, num_q_heads: int, num_kv_heads: int, max_seq_len: int, q_new, k_new, v_new,
                       k_cache, v_cache, page_table, seq_lens, positions, q_norm_w, k_norm_w, rope_theta: float,
                       eps: float, out, *, block_size: int = 0, num_cache_blocks: int = 0, head_dim: int = 128,
                       num_workers: int = 0, cluster_size: int = 0, device: int = 0, device_errors=None,
                       stream=None, ordered_start: bool = False):
    """One decode step through gqa_decode_attn_static: no plan, no device allocation; the
    workspace is the library's fixed static scratch of the device.  `device_errors` is an
    optional int32/uint32 device tensor of one element the kernels OR error bits into."""
    desc = PlanDesc(int(batch), int(num_q_heads), int(num_kv_heads), int(head_dim), int(block_size),
                    int(max_seq_len), int(num_cache_blocks), int(num_workers), int(device), int(cluster_size),
                    int(bool(ordered_start)))
    _check(load().gqa_decode_attn_static(
        ctypes.byref(desc), _dptr(q_new), _dptr(k_new), _dptr(v_new), _dptr(k_cache), _dptr(v_cache),
        _dptr(page_table), _dptr(seq_lens), _dptr(positions), _dptr(q_norm_w), _dptr(k_norm_w), float(rope_theta),
        float(eps), _dptr(out), _dptr(device_errors), _stream(stream)), "gqa_decode_attn_static")


def decode_attn_static_workload(w, out, *, num_workers: int = 0, cluster_size: int = 0, device: int = 0,
                                device_errors=None, stream=None):
    """gqa_decode_attn_static on a workload's tensors (see workloads.Workload)."""
    decode_attn_static(w.B, w.Hq, w.Hkv, w.max_seq, w.q_new, w.k_new, w.v_new, w.k_cache, w.v_cache, w.page_table,
                       w.seq_lens, w.positions, w.q_norm_w, w.k_norm_w, w.rope_theta, w.eps, out,
                       block_size=w.block_size, num_cache_blocks=w.num_blocks, num_workers=num_workers,
                       cluster_size=cluster_size, device=device, device_errors=device_errors, stream=stream)


def prefill_attn(batch: int, num_q_heads: int, num_kv_heads: int, chunk_len: int, max_seq_len: int, q_new, k_new,
                 v_new, k_cache, v_cache, page_table, q_start, q_norm_w, k_norm_w, rope_theta: float, eps: float, out,
                 *, block_size: int = 0, num_cache_blocks: int = 0, head_dim: int = 128, device: int = 0,
                 device_errors=None, stream=None):
    """One chunk of causal prefill through gqa_prefill_attn (include/gqa_prefill.h)."""
    desc = PrefillDesc(int(batch), int(num_q_heads), int(num_kv_heads), int(head_dim), int(chunk_len),
                       int(block_size), int(max_seq_len), int(num_cache_blocks), int(device))
    _check(load().gqa_prefill_attn(
        ctypes.byref(desc), _dptr(q_new), _dptr(k_new), _dptr(v_new), _dptr(k_cache), _dptr(v_cache),
        _dptr(page_table), _dptr(q_start), _dptr(q_norm_w), _dptr(k_norm_w), float(rope_theta), float(eps),
        _dptr(out), _dptr(device_errors), _stream(stream)), "gqa_prefill_attn")


def prefill_attn_workload(w, out, *, device: int = 0, device_errors=None, stream=None):
    """gqa_prefill_attn on a prefill workload's tensors (see workloads.PrefillWorkload)."""
    prefill_attn(w.B, w.Hq, w.Hkv, w.T, w.max_seq, w.q_new, w.k_new, w.v_new, w.k_cache, w.v_cache, w.page_table,
                 w.q_start, w.q_norm_w, w.k_norm_w, w.rope_theta, w.eps, out, block_size=w.block_size,
                 num_cache_blocks=w.num_blocks, device=device, device_errors=device_errors, stream=stream)


# ------------------- rotary append, draft trees, cache pages, 8-bit caches, packed prompts

# These calls come once a layer and step, so their wrappers keep to a few microseconds: one check
# a tensor, and the descriptors of the geometries in use are kept (the library reads them during a
# call only).

class _Torch:
    """What the wrappers need of torch, looked up at the first call (importing the binding
    does not import torch)."""

    ready = False

    @classmethod
    def load(cls):
        import torch
        cls.i32, cls.bf16, cls.u8, cls.f32 = torch.int32, torch.bfloat16, torch.uint8, torch.float32
        cls.codes = {"e4m3": (torch.float8_e4m3fn, torch.uint8), "int8": (torch.int8, torch.uint8)}
        cls.word32, cls.word64 = (torch.int32, torch.uint32), (torch.int64, torch.uint64)
        cls.empty = torch.empty
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the handle without a Stream object
        cls.stream = staticmethod(raw or (lambda d: torch.cuda.current_stream(d).cuda_stream))
        cls.ready = True


def _torch():
    if not _Torch.ready:
        _Torch.load()
    return _Torch


def _on(device: int, stream) -> int:
    """The stream a call on `device` is queued on: the caller's, else torch's current one there."""
    if stream is None:
        return _torch().stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dev(t, name: str, dtype, shape, device: int, optional: bool = False) -> Optional[int]:
    """Device pointer of a dense tensor of the dtype and shape the call needs (`dtype` a torch
    dtype or a tuple of them; a `shape` of None takes any)."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is missing")
    if t.get_device() != device:
        raise ValueError(f"{name}: expected a tensor on cuda:{device}, got {t.device}")
    d = t.dtype
    if d is not dtype and not (isinstance(dtype, tuple) and d in dtype):
        raise ValueError(f"{name}: expected {dtype}, got {d}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _err(t, device: int) -> Optional[int]:
    return None if t is None else _dev(t, "device_errors", _torch().word32, (1,), device)


@functools.lru_cache(maxsize=1024)
def _desc(kind, *fields):
    """A reference to the descriptor with these fields (ctypes would drop the upper bits of larger ones)."""
    if any(not -2**31 <= int(x) < 2**31 for x in fields):
        raise ValueError(f"{kind.__name__}: a field of {fields} does not fit 32 bits")
    return ctypes.byref(kind(*fields))


def _cache(name: str, t, rows: int, num_kv_heads: int, device: int) -> int:
    p = _dev(t, name, _torch().bf16, None, device)
    if t.numel() != rows * num_kv_heads * 128:
        raise ValueError(f"{name}: expected {rows} rows of {num_kv_heads} x 128, got shape {tuple(t.shape)}")
    return p


def _tokens(t, name: str, batch: int, tokens: int, heads: int, device: int):
    """(pointer, stride in elements between tokens) of a [B, T, H, 128] tensor whose heads are
    dense and whose tokens are evenly spaced -- dense, or a slice of a wider projection."""
    if t is None or t.get_device() != device or t.dtype is not _torch().bf16:
        raise ValueError(f"{name}: expected a bfloat16 tensor on cuda:{device}")
    if t.shape != (batch, tokens, heads, 128):
        raise ValueError(f"{name}: expected shape {(batch, tokens, heads, 128)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), heads * 128
    sb, st, sh, sd = t.stride()
    if tokens == 1:
        st = sb
    step = heads * 128 if batch == 1 and tokens == 1 else st
    if sd != 1 or (heads > 1 and sh != 128) or (batch > 1 and sb != step * tokens) or step < heads * 128:
        raise ValueError(f"{name}: heads must be dense and tokens evenly spaced, got strides {t.stride()}")
    return t.data_ptr(), step


def rope_append(batch: int, num_q_heads: int, num_kv_heads: int, num_tokens: int, max_seq_len: int, q, k, v, k_cache,
                v_cache, page_table, slot_start, positions, counts, q_norm_w, k_norm_w, rope: Rope, eps: float, q_out,
                *, block_size: int = 0, num_cache_blocks: int = 0, head_dim: int = 128, device: int = 0,
                device_errors=None, stream=None):
    """QK-norm, rotation and append of [B, T] tokens (gqa_rope_append, include/gqa_rope.h).  q, k
    and v may be slices of one projection (token strides are taken from the tensors)."""
    tt = _torch()
    i32 = tt.i32
    qp, qs = _tokens(q, "q", batch, num_tokens, num_q_heads, device)
    kp, ks = _tokens(k, "k", batch, num_tokens, num_kv_heads, device)
    vp, vs = _tokens(v, "v", batch, num_tokens, num_kv_heads, device)
    rows = num_cache_blocks * 64 if block_size else batch * max_seq_len
    desc = _desc(RopeDesc, batch, num_q_heads, num_kv_heads, head_dim, num_tokens, block_size, max_seq_len,
                 num_cache_blocks, device, qs, ks, vs)
    _check(load().gqa_rope_append(
        desc, qp, kp, vp, _cache("k_cache", k_cache, rows, num_kv_heads, device),
        _cache("v_cache", v_cache, rows, num_kv_heads, device),
        _dev(page_table, "page_table", i32, (batch, (max_seq_len + 63) // 64), device, True),
        _dev(slot_start, "slot_start", i32, (batch,), device),
        _dev(positions, "positions", i32, (batch, num_tokens), device, True),
        _dev(counts, "counts", i32, (batch,), device, True),
        _dev(q_norm_w, "q_norm_w", tt.bf16, (128,), device, True),
        _dev(k_norm_w, "k_norm_w", tt.bf16, (128,), device, True), ctypes.byref(rope), float(eps),
        _dev(q_out, "q_out", tt.bf16, (batch, num_tokens, num_q_heads, 128), device),
        _err(device_errors, device), _on(device, stream)),
        "gqa_rope_append")


def tree_prepare(parents, ctx_lens, counts, mask, positions, *, device: int = 0, device_errors=None, stream=None):
    """The masks (int64 words) and positions of draft trees from their parents [B, T]
    (gqa_tree_prepare, include/gqa_tree.h)."""
    tt = _torch()
    i32 = tt.i32
    if parents.dim() != 2:
        raise ValueError("parents: expected [batch, tree_len]")
    batch, tree_len = parents.shape
    pp = _dev(parents, "parents", i32, None, device)
    _check(load().gqa_tree_prepare(
        batch, tree_len, pp, _dev(ctx_lens, "ctx_lens", i32, (batch,), device),
        _dev(counts, "counts", i32, (batch,), device, True),
        _dev(mask, "mask", tt.word64, (batch, tree_len, (tree_len + 63) // 64), device),
        _dev(positions, "positions", i32, (batch, tree_len), device), device,
        _err(device_errors, device), _on(device, stream)),
        "gqa_tree_prepare")


def tree_workspace_bytes(batch: int, num_q_heads: int, num_kv_heads: int, tree_len: int, max_seq_len: int, *,
                         block_size: int = 0, num_cache_blocks: int = 0, head_dim: int = 128, device: int = 0) -> int:
    return _workspace_of(batch, num_q_heads, num_kv_heads, head_dim, tree_len, block_size, max_seq_len, num_cache_blocks,
                         device)


@functools.lru_cache(maxsize=1024)
def _workspace_of(*fields) -> int:
    n = ctypes.c_size_t(0)
    _check(load().gqa_tree_workspace_bytes(_desc(TreeDesc, *fields), ctypes.byref(n)), "gqa_tree_workspace_bytes")
    return int(n.value)


def tree_workspace(batch: int, num_q_heads: int, num_kv_heads: int, tree_len: int, max_seq_len: int, *,
                   block_size: int = 0, num_cache_blocks: int = 0, head_dim: int = 128, device: int = 0):
    """A workspace for gqa_tree_attn calls of this geometry that do not overlap.  Its size does not depend
    on the cache's layout, but the limit on a cache's rows does: a page table whose batch *
    max_seq_len passes 2^31 - 1 (a pool smaller than every sequence at full length) needs the paged layout here."""
    tt = _torch()
    return tt.empty(tree_workspace_bytes(batch, num_q_heads, num_kv_heads, tree_len, max_seq_len, block_size=block_size,
                                         num_cache_blocks=num_cache_blocks, head_dim=head_dim, device=device),
                    dtype=tt.u8, device=f"cuda:{device}")


def tree_attn(batch: int, num_q_heads: int, num_kv_heads: int, tree_len: int, max_seq_len: int, q, k_cache, v_cache,
              page_table, ctx_lens, counts, mask, out, *, block_size: int = 0, num_cache_blocks: int = 0,
              head_dim: int = 128, workspace=None, device: int = 0, device_errors=None, stream=None):
    """Attention of draft-tree nodes over the cache (gqa_tree_attn, include/gqa_tree.h).
    ``workspace``: a uint8 tensor of tree_workspace_bytes; None takes one from torch's allocator
    for this call (which knows the current stream only: give one with an explicit ``stream``)."""
    tt = _torch()
    i32 = tt.i32
    rows = num_cache_blocks * 64 if block_size else batch * max_seq_len
    fields = (batch, num_q_heads, num_kv_heads, head_dim, tree_len, block_size, max_seq_len, num_cache_blocks, device)
    need = _workspace_of(*fields)
    if workspace is None:
        if stream is not None:
            raise ValueError("a call on an explicit stream needs a workspace")
        workspace = tt.empty(need, dtype=tt.u8, device=f"cuda:{device}")
    ws = _dev(workspace, "workspace", tt.u8, None, device)
    if workspace.numel() < need:
        raise ValueError(f"workspace: {need} bytes needed, got {workspace.numel()}")
    shape = (batch, tree_len, num_q_heads, 128)
    qp, op = _dev(q, "q", tt.bf16, shape, device), _dev(out, "out", tt.bf16, shape, device)
    if qp == op:
        raise ValueError("out: must not be q, which other CTAs still read")
    _check(load().gqa_tree_attn(
        _desc(TreeDesc, *fields), qp,
        _cache("k_cache", k_cache, rows, num_kv_heads, device),
        _cache("v_cache", v_cache, rows, num_kv_heads, device),
        _dev(page_table, "page_table", i32, (batch, (max_seq_len + 63) // 64), device, True),
        _dev(ctx_lens, "ctx_lens", i32, (batch,), device), _dev(counts, "counts", i32, (batch,), device, True),
        _dev(mask, "mask", tt.word64, (batch, tree_len, (tree_len + 63) // 64), device),
        op, ws, _err(device_errors, device), _on(device, stream)),
        "gqa_tree_attn")


class CachePools:
    """The pools of a cache that share a page table (K and V of every layer; the index and scale
    tensors of a 4-bit cache whose num_kv_heads is a multiple of 4): tensors of `rows` rows of a multiple
    of 16 bytes, paged with num_blocks * 64 rows, else contiguous.  Keeps the tensors alive."""

    def __init__(self, tensors, num_blocks: int = 0, rows: int = 0):
        tensors = list(tensors)
        self.num_blocks, self.rows = int(num_blocks), int(rows) or int(num_blocks) * 64
        if not 1 <= len(tensors) <= MAX_POOLS or self.rows < 1 or (num_blocks and self.rows != num_blocks * 64):
            raise ValueError(f"1 to {MAX_POOLS} pools, of num_blocks pages or of rows rows")
        self.device = tensors[0].device.index
        self.array = (Pool * len(tensors))()
        for i, t in enumerate(tensors):
            if not t.is_cuda or t.device.index != self.device or not t.is_contiguous():
                raise ValueError("pools: contiguous tensors on one CUDA device")
            size = t.numel() * t.element_size()
            if size == 0 or size % self.rows:
                raise ValueError(f"pool {i}: {size} bytes are not {self.rows} rows")
            if size // self.rows % 16 or size // self.rows > 1 << 20:
                raise ValueError(f"pool {i}: rows of {size // self.rows} bytes; the page calls move rows of a multiple of 16, up "
                                 "to 2^20 (the scales of a 4-bit cache: num_kv_heads a multiple of 4)")
            self.array[i] = Pool(t.data_ptr(), size // self.rows)
        spans = sorted((p.base, p.row_bytes * self.rows) for p in self.array)
        if any(a + size > b for (a, size), (b, _) in zip(spans, spans[1:])):
            raise ValueError("pools: two of the tensors overlap, their rows would be moved twice")
        self.tensors = tensors

    def __len__(self):
        return len(self.tensors)


def _page_state(ref_counts, page_table, seq_lens, device: int):
    i32 = _torch().i32
    if ref_counts.dim() != 1 or page_table.dim() != 2:
        raise ValueError("ref_counts [num_blocks], page_table [batch, max_blocks]")
    batch, max_blocks = page_table.shape
    ptrs = (_dev(ref_counts, "ref_counts", i32, None, device), _dev(page_table, "page_table", i32, None, device),
            _dev(seq_lens, "seq_lens", i32, (batch,), device))
    return _desc(PagesDesc, batch, max_blocks, ref_counts.shape[0], device), ptrs


def pages_fork(ref_counts, page_table, seq_lens, src, dst, *, device: int = 0, device_errors=None, stream=None):
    """Sequences dst[i] share the pages of sequences src[i] (gqa_pages_fork, include/gqa_pages.h)."""
    i32 = _torch().i32
    desc, ptrs = _page_state(ref_counts, page_table, seq_lens, device)
    n = src.shape[0]
    _check(load().gqa_pages_fork(
        desc, *ptrs, _dev(src, "src", i32, (n,), device), _dev(dst, "dst", i32, (n,), device),
        n, _err(device_errors, device), _on(device, stream)),
        "gqa_pages_fork")


def pages_resize(ref_counts, page_table, seq_lens, new_lens, cow_src, cow_dst, *, device: int = 0, device_errors=None,
                 stream=None):
    """Grow, shrink or free sequences (gqa_pages_resize); cow_src / cow_dst [B] receive the pages to
    copy before the sequences are written to (pages_copy), or -1."""
    i32 = _torch().i32
    desc, ptrs = _page_state(ref_counts, page_table, seq_lens, device)
    shape = (page_table.shape[0],)
    _check(load().gqa_pages_resize(
        desc, *ptrs, _dev(new_lens, "new_lens", i32, shape, device),
        _dev(cow_src, "cow_src", i32, shape, device), _dev(cow_dst, "cow_dst", i32, shape, device),
        _err(device_errors, device), _on(device, stream)),
        "gqa_pages_resize")


def pages_copy(pools: CachePools, src, dst, *, device_errors=None, stream=None):
    """Page dst[i] := page src[i] in every pool; src[i] < 0 is skipped (gqa_pages_copy)."""
    i32, n, device = _torch().i32, src.shape[0], pools.device
    _check(load().gqa_pages_copy(
        pools.array, len(pools), pools.num_blocks, _dev(src, "src", i32, (n,), device),
        _dev(dst, "dst", i32, (n,), device), n, device,
        _err(device_errors, device), _on(device, stream)),
        "gqa_pages_copy")


def cache_keep_rows(pools: CachePools, page_table, start, keep, counts, *, max_seq_len: int, device_errors=None,
                    stream=None):
    """Rows start[b] + keep[b][i] move to start[b] + i in every pool (gqa_cache_keep_rows)."""
    i32, device = _torch().i32, pools.device
    if keep.dim() != 2:
        raise ValueError("keep: expected [batch, max_keep]")
    batch, width = keep.shape
    kp = _dev(keep, "keep", i32, None, device)
    paged = page_table is not None
    if paged != (pools.num_blocks > 0) or (not paged and pools.rows != batch * max_seq_len):
        raise ValueError("a page table goes with paged pools; contiguous ones have batch * max_seq_len rows")
    desc = _desc(KeepDesc, batch, width, max_seq_len, 64 if paged else 0, pools.num_blocks, device)
    _check(load().gqa_cache_keep_rows(
        desc, pools.array, len(pools),
        _dev(page_table, "page_table", i32, (batch, (max_seq_len + 63) // 64), device, True),
        _dev(start, "start", i32, (batch,), device), kp, _dev(counts, "counts", i32, (batch,), device),
        _err(device_errors, device), _on(device, stream)),
        "gqa_cache_keep_rows")


Q8_FORMATS = {"e4m3": 0, "int8": 1}


def _q8_cache(k_codes, v_codes, k_scale, v_scale, fmt: str, rows: int, num_kv_heads: int, device: int):
    """Pointers of an 8-bit cache's four tensors: `rows` rows of num_kv_heads x 128 codes and num_kv_heads scales."""
    tt = _torch()
    codes, n = tt.codes.get(fmt), rows * num_kv_heads
    if codes is None:
        raise ValueError(f"fmt: one of {sorted(Q8_FORMATS)}, got {fmt!r}")
    ptrs = (_dev(k_codes, "k_codes", codes, None, device), _dev(v_codes, "v_codes", codes, None, device),
            _dev(k_scale, "k_scale", tt.f32, None, device), _dev(v_scale, "v_scale", tt.f32, None, device))
    if not (k_scale.numel() == n == v_scale.numel() and k_codes.numel() == n * 128 == v_codes.numel()):
        shapes = [tuple(t.shape) for t in (k_codes, v_codes, k_scale, v_scale)]
        raise ValueError(f"cache: expected {rows} rows of {num_kv_heads} x 128 codes and {num_kv_heads} scales, got shapes {shapes}")
    return ptrs


def _packed(t, name: str, tokens: int, heads: int, device: int):
    """(pointer, stride in elements between tokens) of a packed [N, H, 128] tensor whose heads are
    dense -- dense, or a slice of a wider projection."""
    if t is None or t.get_device() != device or t.dtype is not _torch().bf16:
        raise ValueError(f"{name}: expected a bfloat16 tensor on cuda:{device}")
    if t.shape != (tokens, heads, 128):
        raise ValueError(f"{name}: expected shape {(tokens, heads, 128)}, got {tuple(t.shape)}")
    if t.is_contiguous():
        return t.data_ptr(), heads * 128
    st, sh, sd = t.stride()
    if tokens == 1:
        st = heads * 128
    if sd != 1 or (heads > 1 and sh != 128) or st < heads * 128:
        raise ValueError(f"{name}: heads must be dense and tokens evenly spaced, got strides {t.stride()}")
    return t.data_ptr(), st


def q8_append(batch: int, num_kv_heads: int, num_tokens: int, max_seq_len: int, k, v, k_codes, v_codes, k_scale, v_scale,
              page_table, offsets, slot_start, *, fmt: str = "e4m3", block_size: int = 0, num_cache_blocks: int = 0,
              head_dim: int = 128, device: int = 0, device_errors=None, stream=None):
    """Quantise and store packed rows (gqa_q8_append, include/gqa_q8.h): k and v [N, H_kv, 128], the rows
    offsets[b] .. offsets[b + 1] - 1 those of sequence b (offsets None: one row a sequence), to the slots
    from slot_start[b] on.  fmt "e4m3" (codes float8_e4m3fn or uint8) or "int8" (int8 or uint8)."""
    i32 = _torch().i32
    kp, ks = _packed(k, "k", num_tokens, num_kv_heads, device)
    vp, vs = _packed(v, "v", num_tokens, num_kv_heads, device)
    kc, vc, kf, vf = _q8_cache(k_codes, v_codes, k_scale, v_scale, fmt,
                               num_cache_blocks * 64 if block_size else batch * max_seq_len, num_kv_heads, device)
    _check(load().gqa_q8_append(
        _desc(Q8Desc, batch, 0, num_kv_heads, head_dim, Q8_FORMATS[fmt], num_tokens, block_size, max_seq_len,
              num_cache_blocks, device, ks, vs), kp, vp, kc, vc, kf, vf,
        _dev(page_table, "page_table", i32, (batch, (max_seq_len + 63) // 64), device, True),
        _dev(offsets, "offsets", i32, (batch + 1,), device, True), _dev(slot_start, "slot_start", i32, (batch,), device),
        _err(device_errors, device), _on(device, stream)),
        "gqa_q8_append")


def q8_read(batch: int, num_kv_heads: int, num_tokens: int, max_seq_len: int, k_codes, v_codes, k_scale, v_scale,
            page_table, offsets, slot_start, k_out, v_out, *, fmt: str = "e4m3", block_size: int = 0,
            num_cache_blocks: int = 0, head_dim: int = 128, device: int = 0, device_errors=None, stream=None):
    """Rows of an 8-bit cache as packed bf16 (gqa_q8_read): row offsets[b] + i of k_out and v_out [N, H_kv, 128]
    receives slot slot_start[b] + i of sequence b (slot_start None: from slot 0 on)."""
    i32 = _torch().i32
    kp, ks = _packed(k_out, "k_out", num_tokens, num_kv_heads, device)
    vp, vs = _packed(v_out, "v_out", num_tokens, num_kv_heads, device)
    kc, vc, kf, vf = _q8_cache(k_codes, v_codes, k_scale, v_scale, fmt,
                               num_cache_blocks * 64 if block_size else batch * max_seq_len, num_kv_heads, device)
    _check(load().gqa_q8_read(
        _desc(Q8Desc, batch, 0, num_kv_heads, head_dim, Q8_FORMATS[fmt], num_tokens, block_size, max_seq_len,
              num_cache_blocks, device, ks, vs), kc, vc, kf, vf,
        _dev(page_table, "page_table", i32, (batch, (max_seq_len + 63) // 64), device, True),
        _dev(offsets, "offsets", i32, (batch + 1,), device, True),
        _dev(slot_start, "slot_start", i32, (batch,), device, True), kp, vp,
        _err(device_errors, device), _on(device, stream)),
        "gqa_q8_read")


@functools.lru_cache(maxsize=1024)
def _q8_workspace_of(batch, num_q_heads, num_kv_heads, max_seq_len, block_size, num_cache_blocks, head_dim, device) -> int:
    n = ctypes.c_size_t(0)
    _check(load().gqa_q8_workspace_bytes(_desc(Q8Desc, batch, num_q_heads, num_kv_heads, head_dim, 0, 0, block_size,
                                               max_seq_len, num_cache_blocks, device, 0, 0), ctypes.byref(n)),
           "gqa_q8_workspace_bytes")
    return int(n.value)


def q8_workspace_bytes(batch: int, num_q_heads: int, num_kv_heads: int, max_seq_len: int, *, block_size: int = 0,
                       num_cache_blocks: int = 0, head_dim: int = 128, device: int = 0) -> int:
    return _q8_workspace_of(batch, num_q_heads, num_kv_heads, max_seq_len, block_size, num_cache_blocks, head_dim, device)


def q8_workspace(batch: int, num_q_heads: int, num_kv_heads: int, max_seq_len: int, *, block_size: int = 0,
                 num_cache_blocks: int = 0, head_dim: int = 128, device: int = 0):
    """A workspace for gqa_q8_attn calls of this geometry that do not overlap."""
    tt = _torch()
    return tt.empty(q8_workspace_bytes(batch, num_q_heads, num_kv_heads, max_seq_len, block_size=block_size,
                                       num_cache_blocks=num_cache_blocks, head_dim=head_dim, device=device),
                    dtype=tt.u8, device=f"cuda:{device}")


def q8_attn(batch: int, num_q_heads: int, num_kv_heads: int, max_seq_len: int, q, k_codes, v_codes, k_scale, v_scale,
            page_table, seq_lens, out, *, fmt: str = "e4m3", block_size: int = 0, num_cache_blocks: int = 0,
            head_dim: int = 128, workspace=None, device: int = 0, device_errors=None, stream=None):
    """Attention of one new token a sequence over an 8-bit cache (gqa_q8_attn, include/gqa_q8.h): q and out [B, H_q,
    128], slots 0 .. seq_lens[b] - 1.  ``workspace``: a uint8 tensor of q8_workspace_bytes; None takes one from torch's
    allocator for this call (which knows the current stream only: give one with an explicit ``stream``)."""
    tt = _torch()
    i32 = tt.i32
    rows = num_cache_blocks * 64 if block_size else batch * max_seq_len
    need = _q8_workspace_of(batch, num_q_heads, num_kv_heads, max_seq_len, block_size, num_cache_blocks, head_dim, device)
    if workspace is None:
        if stream is not None:
            raise ValueError("a call on an explicit stream needs a workspace")
        workspace = tt.empty(need, dtype=tt.u8, device=f"cuda:{device}")
    ws = _dev(workspace, "workspace", tt.u8, None, device)
    if workspace.numel() < need:
        raise ValueError(f"workspace: {need} bytes needed, got {workspace.numel()}")
    shape = (batch, num_q_heads, 128)
    qp, op = _dev(q, "q", tt.bf16, shape, device), _dev(out, "out", tt.bf16, shape, device)
    if qp == op:
        raise ValueError("out: must not be q, which other CTAs still read")
    cp = _q8_cache(k_codes, v_codes, k_scale, v_scale, fmt, rows, num_kv_heads, device)
    _check(load().gqa_q8_attn(
        _desc(Q8Desc, batch, num_q_heads, num_kv_heads, head_dim, Q8_FORMATS[fmt], 0, block_size, max_seq_len,
              num_cache_blocks, device, 0, 0), qp, *cp,
        _dev(page_table, "page_table", i32, (batch, (max_seq_len + 63) // 64), device, True),
        _dev(seq_lens, "seq_lens", i32, (batch,), device), op, ws, _err(device_errors, device), _on(device, stream)),
        "gqa_q8_attn")


def packed_attn(q, k, v, q_offsets, k_offsets, out, *, causal: bool = True, device: int = 0, device_errors=None,
                stream=None):
    """Attention over packed prompts (gqa_packed_attn, include/gqa_packed.h): q [N_q, H_q, 128], k and v [N_k, H_kv,
    128] (slices of one projection are taken as they are), out [N_q, H_q, 128] dense; sequence b has the queries
    q_offsets[b] .. q_offsets[b + 1] - 1 and the keys of k_offsets (None: the same), both ending at one token."""
    tt = _torch()
    if q.dim() != 3 or k.dim() != 3 or q_offsets.dim() != 1:
        raise ValueError("q [N_q, H_q, 128], k and v [N_k, H_kv, 128], q_offsets [B + 1]")
    (nq, hq, _), (nk, hkv, _) = q.shape, k.shape
    offsets = q_offsets.shape
    qp, qs = _packed(q, "q", nq, hq, device)
    kp, ks = _packed(k, "k", nk, hkv, device)
    vp, vs = _packed(v, "v", nk, hkv, device)
    op = _dev(out, "out", tt.bf16, (nq, hq, 128), device)
    if qp == op:
        raise ValueError("out: must not be q, which other CTAs still read")
    _check(load().gqa_packed_attn(
        _desc(PackedDesc, offsets[0] - 1, hq, hkv, 128, nq, nk, int(bool(causal)), device, qs, ks, vs), qp, kp, vp,
        _dev(q_offsets, "q_offsets", tt.i32, None, device), _dev(k_offsets, "k_offsets", tt.i32, offsets, device, True), op,
        _err(device_errors, device), _on(device, stream)),
        "gqa_packed_attn")


def q4_codebook() -> np.ndarray:
    """The 16 Lloyd-Max levels of N(0,1) as bf16 bit patterns (gqa_q4_codebook)."""
    out = np.zeros(16, dtype=np.uint16)
    _check(load().gqa_q4_codebook(out.ctypes.data), "gqa_q4_codebook")
    return out


class Plan:
    """A gqa_plan_t: geometry, split-worker count and the workspace (allocated once)."""

    def __init__(self, batch: int, num_q_heads: int, num_kv_heads: int, max_seq_len: int, *,
                 block_size: int = 0, num_cache_blocks: int = 0, head_dim: int = 128, num_workers: int = 0,
                 device: int = 0, seq_lens_host=None, cluster_size: int = 0, ordered_start: bool = False):
        self._lib = load()
        self.desc = PlanDesc(int(batch), int(num_q_heads), int(num_kv_heads), int(head_dim), int(block_size),
                             int(max_seq_len), int(num_cache_blocks), int(num_workers), int(device),
                             int(cluster_size), int(bool(ordered_start)))
        sl = None
        if seq_lens_host is not None:
            sl = np.ascontiguousarray(np.asarray(seq_lens_host, dtype=np.int32))
        self._h = ctypes.c_void_p()
        _check(self._lib.gqa_plan_create(ctypes.byref(self.desc), None if sl is None else sl.ctypes.data,
                                         ctypes.byref(self._h)), "gqa_plan_create")

    @classmethod
    def for_workload(cls, w, num_workers: int = 0, device: int = 0, cluster_size: int = 0) -> "Plan":
        return cls(w.B, w.Hq, w.Hkv, w.max_seq, block_size=w.block_size, num_cache_blocks=w.num_blocks,
                   num_workers=num_workers, device=device, seq_lens_host=w.seq_lens.cpu().numpy(),
                   cluster_size=cluster_size)

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            _check(self._lib.gqa_plan_destroy(self._h), "gqa_plan_destroy")
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:  # noqa: BLE001 - interpreter shutdown
            pass

    @property
    def handle(self):
        return self._h

    @property
    def num_workers(self) -> int:
        return self._lib.gqa_plan_num_workers(self._h)

    def set_ordered_start(self, ordered: bool = True):
        """Launch each step's first kernel in plain stream order (gqa_plan_set_ordered_start)."""
        _check(self._lib.gqa_plan_set_ordered_start(self._h, int(bool(ordered))), "gqa_plan_set_ordered_start")

    @property
    def num_splits(self) -> int:
        return self._lib.gqa_plan_num_splits(self._h)

    @property
    def cluster_size(self) -> int:
        """The single-launch form's cluster size, 0 for split-KV + combine."""
        return self._lib.gqa_plan_cluster_size(self._h)

    @property
    def workspace_bytes(self) -> int:
        return self._lib.gqa_plan_workspace_bytes(self._h)

    # ------------------------------------------------------------------ the step
    def decode_attn(self, q_new, k_new, v_new, k_cache, v_cache, page_table, seq_lens, positions,
                    q_norm_w, k_norm_w, rope_theta: float, eps: float, out, stream=None):
        _check(self._lib.gqa_decode_attn(
            self._h, _dptr(q_new), _dptr(k_new), _dptr(v_new), _dptr(k_cache), _dptr(v_cache), _dptr(page_table),
            _dptr(seq_lens), _dptr(positions), _dptr(q_norm_w), _dptr(k_norm_w), float(rope_theta), float(eps),
            _dptr(out), _stream(stream)), "gqa_decode_attn")

    def decode_attn_host(self, q_new, k_new, v_new, k_cache, v_cache, page_table, seq_lens, positions,
                         q_norm_w, k_norm_w, rope_theta: float, eps: float, out, stream=None):
        """q/k/v_new, seq_lens, positions and out are host buffers; caches, page table and
        norm weights are device tensors.  Synchronise the stream before reading `out`."""
        _check(self._lib.gqa_decode_attn_host(
            self._h, _hptr(q_new), _hptr(k_new), _hptr(v_new), _dptr(k_cache), _dptr(v_cache), _dptr(page_table),
            _hptr(seq_lens), _hptr(positions), _dptr(q_norm_w), _dptr(k_norm_w), float(rope_theta), float(eps),
            _hptr(out), _stream(stream)), "gqa_decode_attn_host")

    def attention_splitkv(self, q_new, k_new, v_new, k_cache, v_cache, page_table, seq_lens, positions, q_norm_w,
                          k_norm_w, rope_theta: float, eps: float, stream=None):
        _check(self._lib.gqa_attention_splitkv(
            self._h, _dptr(q_new), _dptr(k_new), _dptr(v_new), _dptr(k_cache), _dptr(v_cache), _dptr(page_table),
            _dptr(seq_lens), _dptr(positions), _dptr(q_norm_w), _dptr(k_norm_w), float(rope_theta), float(eps),
            _stream(stream)), "gqa_attention_splitkv")

    def combine(self, seq_lens, out, stream=None):
        _check(self._lib.gqa_combine(self._h, _dptr(seq_lens), _dptr(out), _stream(stream)), "gqa_combine")

    def read_q_rot(self) -> np.ndarray:
        d = self.desc
        out = np.zeros((d.batch, d.num_q_heads, d.head_dim), dtype=np.uint16)
        _check(self._lib.gqa_plan_read_q_rot(self._h, out.ctypes.data), "gqa_plan_read_q_rot")
        return out

    def device_errors(self, clear: bool = True) -> int:
        f = ctypes.c_uint32(0)
        _check(self._lib.gqa_plan_device_errors(self._h, ctypes.byref(f), int(bool(clear))), "gqa_plan_device_errors")
        return int(f.value)

    # ------------------------------------------------------------------ convenience
    def decode_attn_q4(self, q_new, k_new, v_new, k_idx, v_idx, k_scale, v_scale, page_table, seq_lens,
                       positions, q_norm_w, k_norm_w, rot_signs, codebook, rope_theta: float, eps: float, out,
                       stream=None):
        """The decode step over a 4-bit cache (gqa_decode_attn_q4, include/gqa_q4.h)."""
        _check(load().gqa_decode_attn_q4(
            self._h, _dptr(q_new), _dptr(k_new), _dptr(v_new), _dptr(k_idx), _dptr(v_idx), _dptr(k_scale),
            _dptr(v_scale), _dptr(page_table), _dptr(seq_lens), _dptr(positions), _dptr(q_norm_w), _dptr(k_norm_w),
            _dptr(rot_signs), _dptr(codebook), float(rope_theta), float(eps), _dptr(out), _stream(stream)),
            "gqa_decode_attn_q4")

    def run_q4(self, w, out, stream=None):
        """gqa_decode_attn_q4 on a 4-bit-cache workload (workloads.Q4Workload)."""
        self.decode_attn_q4(w.q_new, w.k_new, w.v_new, w.k_idx, w.v_idx, w.k_scale, w.v_scale, w.page_table,
                            w.seq_lens, w.positions, w.q_norm_w, w.k_norm_w, w.rot_signs, w.codebook, w.rope_theta,
                            w.eps, out, stream)

    def run(self, w, out, stream=None):
        """One decode step of a workloads.Workload already on this device."""
        self.decode_attn(w.q_new, w.k_new, w.v_new, w.k_cache, w.v_cache, w.page_table, w.seq_lens, w.positions,
                         w.q_norm_w, w.k_norm_w, w.rope_theta, w.eps, out, stream)

    def run_steps(self, w, out, stream=None, between=None):
        """The same step as its two launches; between(i) is called before (i = 0) and
        after (i = 1) the attention launch -- e.g. to record CUDA events around it."""
        if between:
            between(0)
        self.attention_splitkv(w.q_new, w.k_new, w.v_new, w.k_cache, w.v_cache, w.page_table, w.seq_lens,
                               w.positions, w.q_norm_w, w.k_norm_w, w.rope_theta, w.eps, stream)
        if between:
            between(1)
        self.combine(w.seq_lens, out, stream)
