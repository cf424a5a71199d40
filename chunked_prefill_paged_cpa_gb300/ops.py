"""Thin Python binding of libcpa (include/cpa.h): argument marshalling only.

The ``cpa_*`` functions mirror the C entry points one to one and return the
C status code.  ``kv_append`` / ``attention_forward`` are conveniences that
build the descriptor from torch tensors, call the C entry point on torch's
current stream and raise on a non-zero status.  Every step of the computation
runs in the library's CUDA kernels; there is no other implementation.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

CPA_OK, CPA_ERR_ARG, CPA_ERR_UNSUPPORTED, CPA_ERR_WORKSPACE, CPA_ERR_CUDA, CPA_ERR_DEVICE = (
    0, -1, -2, -3, -4, -5)
CPA_F32, CPA_BF16, CPA_F16 = 0, 1, 2
CPA_KV_SAME, CPA_KV_E4M3 = 0, 1

_lock = threading.Lock()
_lib = None


class CpaDesc(ctypes.Structure):
    _fields_ = [
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_pages", ctypes.c_int64),
        ("max_pages_per_seq", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("num_tokens", ctypes.c_int64),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("kv_dtype", ctypes.c_int32),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
    ]


class CpaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {cpa_status_string(status)} ({status})")
        self.status = status


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = False) -> ctypes.CDLL:
    """Load libcpa.so.  Raises if it is not built (no fallback exists)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB
        if not os.path.exists(path):
            if not build_if_missing:
                raise RuntimeError(
                    f"libcpa.so not built ({path}); run __graft_entry__.build() or "
                    "python -m chunked_prefill_paged_cpa_gb300.build")
            _build.build()
        lib = ctypes.CDLL(path)
        P, I32, F, Z = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        D = ctypes.POINTER(CpaDesc)
        lib.cpa_status_string.argtypes = [ctypes.c_int]
        lib.cpa_status_string.restype = ctypes.c_char_p
        lib.cpa_workspace_bytes.argtypes = [D, I32]
        lib.cpa_workspace_bytes.restype = Z
        lib.cpa_kv_append.argtypes = [P, P, P, P, P, D, P]
        lib.cpa_kv_append.restype = ctypes.c_int
        lib.cpa_attention_forward.argtypes = [P, P, P, P, P, P, I32, F, P, P, D]
        lib.cpa_attention_forward.restype = ctypes.c_int
        lib.cpa_append_attention_forward.argtypes = [P, P, P, P, P, P, P, P, P, I32, F, P, P, D]
        lib.cpa_append_attention_forward.restype = ctypes.c_int
        lib.cpa_window_attention_forward.argtypes = [P, P, P, P, P, P, I32, F, I32, I32, P, P, D]
        lib.cpa_window_attention_forward.restype = ctypes.c_int
        lib.cpa_append_window_attention_forward.argtypes = [P, P, P, P, P, P, P, P, P, I32, F, I32,
                                                            I32, P, P, D]
        lib.cpa_append_window_attention_forward.restype = ctypes.c_int
        lib.cpa_pages_workspace_bytes.argtypes = [ctypes.c_int64]
        lib.cpa_pages_workspace_bytes.restype = Z
        lib.cpa_copy_pages.argtypes = [P, P, P, I32, P, P, D, P]
        lib.cpa_copy_pages.restype = ctypes.c_int
        lib.cpa_fork_sequences.argtypes = [P, P, I32, P, P, I32, P, D, P]
        lib.cpa_fork_sequences.restype = ctypes.c_int
        lib.cpa_extend_sequences.argtypes = [P, P, I32, P, P, P, P, P, P, D, P]
        lib.cpa_extend_sequences.restype = ctypes.c_int
        lib.cpa_release_pages.argtypes = [P, I32, P, P, I32, I32, I32, P, D, P]
        lib.cpa_release_pages.restype = ctypes.c_int
        lib.cpa_compact_pages.argtypes = [P, I32, P, P, P, P, D, P]
        lib.cpa_compact_pages.restype = ctypes.c_int
        lib.cpa_attention_forward_noalloc.argtypes = [P, P, P, P, P, P, I32, F, P, P, D]
        lib.cpa_attention_forward_noalloc.restype = ctypes.c_int
        lib.cpa_read_device_status.argtypes = [D, P, ctypes.POINTER(I32)]
        lib.cpa_read_device_status.restype = ctypes.c_int
        lib.cpa_noalloc_scratch_bytes.argtypes = []
        lib.cpa_noalloc_scratch_bytes.restype = Z
        lib.cpa_noalloc_read_device_status.argtypes = [P, ctypes.POINTER(I32)]
        lib.cpa_noalloc_read_device_status.restype = ctypes.c_int
        _lib = lib
        return lib


# ---- one-to-one mirrors of the C ABI -------------------------------------

def cpa_status_string(status: int) -> str:
    return load().cpa_status_string(int(status)).decode()


def cpa_workspace_bytes(desc: CpaDesc, num_seqs: int) -> int:
    return int(load().cpa_workspace_bytes(ctypes.byref(desc), int(num_seqs)))


def cpa_kv_append(k, v, slot_mapping, k_cache, v_cache, desc: CpaDesc, stream) -> int:
    return int(load().cpa_kv_append(k, v, slot_mapping, k_cache, v_cache,
                                    ctypes.byref(desc), stream))


def cpa_attention_forward(q, k_cache, v_cache, block_table, query_start_loc, seq_lens,
                          num_seqs, scale, out, stream, desc: CpaDesc) -> int:
    return int(load().cpa_attention_forward(q, k_cache, v_cache, block_table,
                                            query_start_loc, seq_lens, int(num_seqs),
                                            float(scale), out, stream, ctypes.byref(desc)))


def cpa_append_attention_forward(q, k, v, slot_mapping, k_cache, v_cache, block_table,
                                 query_start_loc, seq_lens, num_seqs, scale, out, stream,
                                 desc: CpaDesc) -> int:
    return int(load().cpa_append_attention_forward(q, k, v, slot_mapping, k_cache, v_cache,
                                                   block_table, query_start_loc, seq_lens,
                                                   int(num_seqs), float(scale), out, stream,
                                                   ctypes.byref(desc)))


def cpa_window_attention_forward(q, k_cache, v_cache, block_table, query_start_loc, seq_lens,
                                 num_seqs, scale, window, sinks, out, stream,
                                 desc: CpaDesc) -> int:
    return int(load().cpa_window_attention_forward(q, k_cache, v_cache, block_table,
                                                   query_start_loc, seq_lens, int(num_seqs),
                                                   float(scale), int(window), int(sinks), out,
                                                   stream, ctypes.byref(desc)))


def cpa_append_window_attention_forward(q, k, v, slot_mapping, k_cache, v_cache, block_table,
                                        query_start_loc, seq_lens, num_seqs, scale, window, sinks,
                                        out, stream, desc: CpaDesc) -> int:
    return int(load().cpa_append_window_attention_forward(
        q, k, v, slot_mapping, k_cache, v_cache, block_table, query_start_loc, seq_lens,
        int(num_seqs), float(scale), int(window), int(sinks), out, stream, ctypes.byref(desc)))


def cpa_pages_workspace_bytes(num_pages: int) -> int:
    return int(load().cpa_pages_workspace_bytes(int(num_pages)))


def cpa_copy_pages(src, dst, num_pairs, max_pairs, k_cache, v_cache, desc: CpaDesc, stream) -> int:
    return int(load().cpa_copy_pages(src, dst, num_pairs, int(max_pairs), k_cache, v_cache,
                                     ctypes.byref(desc), stream))


def cpa_fork_sequences(parents, children, num_forks, block_table, seq_lens, num_rows, page_refs,
                       desc: CpaDesc, stream) -> int:
    return int(load().cpa_fork_sequences(parents, children, int(num_forks), block_table, seq_lens,
                                         int(num_rows), page_refs, ctypes.byref(desc), stream))


def cpa_extend_sequences(query_start_loc, seq_lens, num_seqs, block_table, page_refs,
                         slot_mapping, copy_src, copy_dst, counts, desc: CpaDesc, stream) -> int:
    return int(load().cpa_extend_sequences(query_start_loc, seq_lens, int(num_seqs), block_table,
                                           page_refs, slot_mapping, copy_src, copy_dst, counts,
                                           ctypes.byref(desc), stream))


def cpa_release_pages(rows, num_released, block_table, seq_lens, num_rows, window, sinks,
                      page_refs, desc: CpaDesc, stream) -> int:
    return int(load().cpa_release_pages(rows, int(num_released), block_table, seq_lens,
                                        int(num_rows), int(window), int(sinks), page_refs,
                                        ctypes.byref(desc), stream))


def cpa_compact_pages(block_table, num_rows, page_refs, copy_src, copy_dst, counts,
                      desc: CpaDesc, stream) -> int:
    return int(load().cpa_compact_pages(block_table, int(num_rows), page_refs, copy_src, copy_dst,
                                        counts, ctypes.byref(desc), stream))


def cpa_attention_forward_noalloc(q, k_cache, v_cache, block_table, query_start_loc,
                                  seq_lens, num_seqs, scale, out, stream,
                                  desc: CpaDesc) -> int:
    """Mirror of the C entry point for callers that cannot allocate device
    memory: the scratch is a fixed array inside the library and
    desc.workspace is ignored."""
    return int(load().cpa_attention_forward_noalloc(q, k_cache, v_cache, block_table,
                                                    query_start_loc, seq_lens, int(num_seqs),
                                                    float(scale), out, stream,
                                                    ctypes.byref(desc)))


def cpa_noalloc_scratch_bytes() -> int:
    """Size of the no-alloc entry point's built-in scratch array, as the
    library was compiled."""
    return int(load().cpa_noalloc_scratch_bytes())


def cpa_noalloc_read_device_status(stream) -> int:
    """Read and clear the status word of the no-alloc scratch array (waits
    for ``stream``); CPA_OK or CPA_ERR_DEVICE."""
    st = ctypes.c_int32(0)
    rc = load().cpa_noalloc_read_device_status(stream, ctypes.byref(st))
    if rc != CPA_OK:
        raise CpaError(rc, "cpa_noalloc_read_device_status")
    return int(st.value)


def cpa_read_device_status(desc: CpaDesc, stream) -> int:
    st = ctypes.c_int32(0)
    rc = load().cpa_read_device_status(ctypes.byref(desc), stream, ctypes.byref(st))
    if rc != CPA_OK:
        raise CpaError(rc, "cpa_read_device_status")
    return int(st.value)


# ---- torch conveniences ---------------------------------------------------

def _dtype_code(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return CPA_BF16
    if dtype == torch.float32:
        return CPA_F32
    if dtype == torch.float16:
        return CPA_F16
    raise TypeError(f"unsupported dtype {dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def make_desc(k_cache: torch.Tensor, num_q_heads: int, num_tokens: int,
              max_pages_per_seq: int, workspace: torch.Tensor | None = None,
              act_dtype: torch.dtype | None = None, k_scale: float = 1.0,
              v_scale: float = 1.0) -> CpaDesc:
    """Descriptor for a cache tensor: a uint8 cache holds E4M3 codes (its
    activations then have ``act_dtype``, bf16 by default, and the codes the
    per-tensor scales); any other cache holds the activation dtype."""
    num_pages, Hkv, page, D = k_cache.shape
    e4m3 = k_cache.dtype == torch.uint8
    dt = (act_dtype or torch.bfloat16) if e4m3 else k_cache.dtype
    return CpaDesc(int(num_q_heads), int(Hkv), int(D), int(page), int(num_pages),
                   int(max_pages_per_seq), _dtype_code(dt), int(num_tokens),
                   None if workspace is None else workspace.data_ptr(),
                   0 if workspace is None else workspace.numel() * workspace.element_size(),
                   CPA_KV_E4M3 if e4m3 else CPA_KV_SAME,
                   float(k_scale) if e4m3 else 0.0, float(v_scale) if e4m3 else 0.0)


def workspace_for(k_cache: torch.Tensor, num_q_heads: int, max_pages_per_seq: int,
                  num_seqs: int, num_tokens: int,
                  act_dtype: torch.dtype | None = None) -> torch.Tensor:
    """A zero-filled device workspace sized by cpa_workspace_bytes for steps of
    at most ``num_seqs`` sequences and ``num_tokens`` packed tokens on the
    current device (``act_dtype``: the queries' dtype for a uint8 E4M3 cache)."""
    desc = make_desc(k_cache, num_q_heads, num_tokens, max_pages_per_seq, act_dtype=act_dtype)
    n = cpa_workspace_bytes(desc, num_seqs)
    if n == 0:
        raise CpaError(CPA_ERR_ARG, "cpa_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=k_cache.device)


def kv_append(k, v, slot_mapping, k_cache, v_cache, workspace=None, stream=None,
              k_scale=1.0, v_scale=1.0) -> None:
    desc = make_desc(k_cache, 1, k.shape[0], 1, workspace, k.dtype, k_scale, v_scale)
    desc.num_q_heads = desc.num_kv_heads
    rc = cpa_kv_append(_ptr(k), _ptr(v), _ptr(slot_mapping), _ptr(k_cache), _ptr(v_cache),
                       desc, _stream(stream))
    if rc != CPA_OK:
        raise CpaError(rc, "cpa_kv_append")


def attention_forward(q, k_cache, v_cache, block_table, query_start_loc, seq_lens, scale,
                      workspace, out=None, stream=None, k_scale=1.0, v_scale=1.0) -> torch.Tensor:
    if out is None:
        out = torch.empty_like(q)
    desc = make_desc(k_cache, q.shape[1], q.shape[0], block_table.shape[1], workspace,
                     q.dtype, k_scale, v_scale)
    rc = cpa_attention_forward(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                               _ptr(query_start_loc), _ptr(seq_lens), seq_lens.shape[0],
                               scale, _ptr(out), _stream(stream), desc)
    if rc != CPA_OK:
        raise CpaError(rc, "cpa_attention_forward")
    return out


def append_attention_forward(q, k, v, slot_mapping, k_cache, v_cache, block_table,
                             query_start_loc, seq_lens, scale, workspace, out=None,
                             stream=None, k_scale=1.0, v_scale=1.0) -> torch.Tensor:
    """kv_append followed by attention_forward, as one C-ABI call (the append
    fused into the attention kernels where they take the shape)."""
    if out is None:
        out = torch.empty_like(q)
    desc = make_desc(k_cache, q.shape[1], q.shape[0], block_table.shape[1], workspace,
                     q.dtype, k_scale, v_scale)
    rc = cpa_append_attention_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(slot_mapping),
                                      _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
                                      _ptr(query_start_loc), _ptr(seq_lens), seq_lens.shape[0],
                                      scale, _ptr(out), _stream(stream), desc)
    if rc != CPA_OK:
        raise CpaError(rc, "cpa_append_attention_forward")
    return out


def _launch(where: str, fn, index: int, stream, args: tuple, desc: CpaDesc, desc_last: bool) -> None:
    """Calls C entry point ``fn`` on device ``index`` (made current for the
    call), on the stream given, else on torch's current stream of that device.
    ``args``: what comes before the stream and the descriptor."""
    if stream is None:
        st = torch._C._cuda_getCurrentRawStream(index)
    else:
        on = getattr(stream, "device", None)
        if on is not None and on.index != index:
            raise ValueError(f"the stream is on {on}, the tensors are on cuda:{index}")
        st = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    tail = (st, ctypes.byref(desc)) if desc_last else (ctypes.byref(desc), st)
    if torch._C._cuda_getDevice() == index:
        rc = fn(*args, *tail)
    else:
        with torch.cuda.device(index):
            rc = fn(*args, *tail)
    if rc != CPA_OK:
        raise CpaError(rc, where)


def _expect(name: str, t: torch.Tensor, dtype, shape: tuple, index: int) -> int:
    """The address of ``t``, a contiguous tensor of this dtype and shape on
    CUDA device ``index``; raises if it is something else: the library takes
    bare pointers.  (One condition on the way that every call takes: a step's
    ten tensors cost 5 us in all.)"""
    if (t.dtype is dtype and t.get_device() == index >= 0 and t.shape == shape
            and t.is_contiguous()):
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name} is {t.dtype}, expected {dtype}")
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name} is on {t.device}, expected "
                         f"{'a CUDA device' if index < 0 else f'cuda:{index}'}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} is not contiguous")


def _expect_any(name: str, t: torch.Tensor, dtype, dims: int, index: int):
    """The same for a tensor of any size: (address, shape)."""
    shape = t.shape
    if (t.dtype is dtype and t.get_device() == index >= 0 and len(shape) == dims
            and t.is_contiguous()):
        return t.data_ptr(), shape
    if len(shape) != dims:
        raise ValueError(f"{name} has shape {tuple(shape)}, expected {dims} dimensions")
    return _expect(name, t, dtype, shape, index), shape


def _i32(x) -> int:
    """A window or a number of sinks as the library takes it: what is larger
    means the same as the largest, and every negative is refused."""
    return min(max(int(x), -1), 2 ** 31 - 1)


_DTYPES = {torch.float32: CPA_F32, torch.bfloat16: CPA_BF16, torch.float16: CPA_F16}


def _cache_desc(k_cache, num_q_heads, num_tokens, max_pages, workspace, dtype, k_scale, v_scale,
                index):
    """Checked addresses of a workspace (or None) in a cache's descriptor."""
    num_pages, hkv, page, d = k_cache.shape
    ws = nb = 0
    if workspace is not None:
        ws, (nb,) = _expect_any("workspace", workspace, torch.uint8, 1, index)
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    if k_cache.dtype is torch.uint8:
        return CpaDesc(num_q_heads, hkv, d, page, num_pages, max_pages, code, num_tokens, ws or None,
                       nb, CPA_KV_E4M3, k_scale, v_scale)
    return CpaDesc(num_q_heads, hkv, d, page, num_pages, max_pages, code, num_tokens, ws or None, nb,
                   CPA_KV_SAME, 0.0, 0.0)


def _window_step(q, k_cache, v_cache, block_table, query_start_loc, seq_lens, workspace, out,
                 k_scale, v_scale):
    """Checks of the windowed calls' tensors: (out, device, addresses, descriptor)."""
    dt, index = q.dtype, k_cache.get_device()
    kdt = k_cache.dtype
    if kdt is not torch.uint8 and kdt is not dt:
        raise TypeError(f"q is {dt}, the caches are {kdt}")
    i32 = torch.int32
    kc, cache = _expect_any("k_cache", k_cache, kdt, 4, index)
    qa, qs = _expect_any("q", q, dt, 3, index)
    table, (seqs, cols) = _expect_any("block_table", block_table, i32, 2, index)
    tokens, heads, d = qs
    if d != cache[3]:
        raise ValueError(f"q has head_dim {d}, the caches have {cache[3]}")
    if out is None:
        out = torch.empty_like(q)
    at = (qa, kc, _expect("v_cache", v_cache, kdt, cache, index), table,
          _expect("query_start_loc", query_start_loc, i32, (seqs + 1,), index),
          _expect("seq_lens", seq_lens, i32, (seqs,), index), seqs)
    desc = _cache_desc(k_cache, heads, tokens, cols, workspace, dt, k_scale, v_scale, index)
    return out, index, at, _expect("out", out, dt, qs, index), desc


def window_attention_forward(q, k_cache, v_cache, block_table, query_start_loc, seq_lens, scale,
                             workspace, window, sinks=0, out=None, stream=None, k_scale=1.0,
                             v_scale=1.0) -> torch.Tensor:
    """Attention of the packed batch where the row at position x sees position
    j <= x when j < sinks or j > x - window.  Takes the workspace of
    ``workspace_for``; block_table entries of pages no row sees are not read."""
    out, index, at, to, desc = _window_step(q, k_cache, v_cache, block_table, query_start_loc,
                                            seq_lens, workspace, out, k_scale, v_scale)
    _launch("cpa_window_attention_forward", load().cpa_window_attention_forward, index, stream,
            (*at, float(scale), _i32(window), _i32(sinks), to), desc, True)
    return out


def append_window_attention_forward(q, k, v, slot_mapping, k_cache, v_cache, block_table,
                                    query_start_loc, seq_lens, scale, workspace, window, sinks=0,
                                    out=None, stream=None, k_scale=1.0,
                                    v_scale=1.0) -> torch.Tensor:
    """kv_append followed by window_attention_forward, as one C-ABI call."""
    out, index, at, to, desc = _window_step(q, k_cache, v_cache, block_table, query_start_loc,
                                            seq_lens, workspace, out, k_scale, v_scale)
    rows = (q.shape[0], k_cache.shape[1], k_cache.shape[3])
    new = (_expect("k", k, q.dtype, rows, index), _expect("v", v, q.dtype, rows, index),
           _expect("slot_mapping", slot_mapping, torch.int64, rows[:1], index))
    _launch("cpa_append_window_attention_forward", load().cpa_append_window_attention_forward, index,
            stream, (at[0], *new, *at[1:], float(scale), _i32(window), _i32(sinks), to), desc, True)
    return out


def pages_workspace_for(num_pages: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for the table operators of a pool of ``num_pages``."""
    n = cpa_pages_workspace_bytes(num_pages)
    if n == 0:
        raise CpaError(CPA_ERR_ARG, "cpa_pages_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


def _pool(block_table, page_refs, workspace):
    """Checks of the tensors every table operator takes: (device, rows,
    addresses of the table and the references, descriptor)."""
    index, i32 = page_refs.get_device(), torch.int32
    refs, (pages,) = _expect_any("page_refs", page_refs, i32, 1, index)
    table, (rows, cols) = _expect_any("block_table", block_table, i32, 2, index)
    ws, (nb,) = _expect_any("workspace", workspace, torch.uint8, 1, index)
    return index, rows, table, refs, CpaDesc(1, 1, 64, 16, pages, cols, CPA_BF16, 0, ws, nb,
                                             CPA_KV_SAME, 0.0, 0.0)


def _pairs(src, dst, least: int, index: int) -> tuple:
    a, (na,) = _expect_any("copy_src", src, torch.int32, 1, index)
    b, (nb,) = _expect_any("copy_dst", dst, torch.int32, 1, index)
    if na < least or nb < least:
        raise ValueError(f"copy_src and copy_dst need {least} entries, they have {na} and {nb}")
    return a, b


def copy_pages(src, dst, k_cache, v_cache, num_pairs=None, workspace=None, stream=None) -> None:
    """Copies pages ``src[i]`` of both caches to pages ``dst[i]``, for every i,
    or for i below ``num_pairs[0]`` (an int32 tensor on the device)."""
    index, kdt = k_cache.get_device(), k_cache.dtype
    kc, cache = _expect_any("k_cache", k_cache, kdt, 4, index)
    a, pairs = _expect_any("src", src, torch.int32, 1, index)
    n = None
    if num_pairs is not None:
        n, (count,) = _expect_any("num_pairs", num_pairs, torch.int32, 1, index)
        if count < 1:
            raise ValueError("num_pairs is empty")
    at = (a, _expect("dst", dst, torch.int32, pairs, index), n, pairs[0], kc,
          _expect("v_cache", v_cache, kdt, cache, index))
    desc = _cache_desc(k_cache, cache[1], 0, 1, workspace,
                       torch.bfloat16 if kdt is torch.uint8 else kdt, 1.0, 1.0, index)
    _launch("cpa_copy_pages", load().cpa_copy_pages, index, stream, at, desc, False)


def fork_sequences(parents, children, block_table, seq_lens, page_refs, workspace,
                   stream=None) -> None:
    """Row ``children[i]`` becomes a copy of row ``parents[i]`` that shares its pages."""
    index, rows, table, refs, desc = _pool(block_table, page_refs, workspace)
    a, n = _expect_any("parents", parents, torch.int32, 1, index)
    at = (a,
          _expect("children", children, torch.int32, n, index), n[0], table,
          _expect("seq_lens", seq_lens, torch.int32, (rows,), index), rows, refs)
    _launch("cpa_fork_sequences", load().cpa_fork_sequences, index, stream, at, desc, False)


def extend_sequences(query_start_loc, seq_lens, block_table, page_refs, slot_mapping, copy_src,
                     copy_dst, counts, workspace, stream=None) -> None:
    """Pages, slots and copies for a step's new tokens (``seq_lens`` counts
    them): fills ``slot_mapping``, the pairs' list and ``counts`` = (pairs, pages
    taken), the latter negative where the pool has too few."""
    index, rows, table, refs, desc = _pool(block_table, page_refs, workspace)
    slots, (desc.num_tokens,) = _expect_any("slot_mapping", slot_mapping, torch.int64, 1, index)
    at = (_expect("query_start_loc", query_start_loc, torch.int32, (rows + 1,), index),
          _expect("seq_lens", seq_lens, torch.int32, (rows,), index), rows, table, refs,
          slots, *_pairs(copy_src, copy_dst, rows, index),
          _expect("counts", counts, torch.int32, (2,), index))
    _launch("cpa_extend_sequences", load().cpa_extend_sequences, index, stream, at, desc, False)


def release_pages(rows, block_table, seq_lens, page_refs, workspace, window=0, sinks=0,
                  stream=None) -> None:
    """Gives back the pages of ``rows`` (None: all rows): every page, or, with a
    window, those that the queries to come do not see."""
    index, every, table, refs, desc = _pool(block_table, page_refs, workspace)
    n, which = every, None
    if rows is not None:
        which, (n,) = _expect_any("rows", rows, torch.int32, 1, index)
    at = (which, n, table, _expect("seq_lens", seq_lens, torch.int32, (every,), index), every,
          _i32(window), _i32(sinks), refs)
    _launch("cpa_release_pages", load().cpa_release_pages, index, stream, at, desc, False)


def compact_pages(block_table, page_refs, copy_src, copy_dst, counts, workspace,
                  stream=None) -> None:
    """Packs the pool's live pages to its front: ``counts`` = (pairs to copy, live pages)."""
    index, rows, table, refs, desc = _pool(block_table, page_refs, workspace)
    at = (table, rows, refs, *_pairs(copy_src, copy_dst, page_refs.shape[0] // 2, index),
          _expect("counts", counts, torch.int32, (2,), index))
    _launch("cpa_compact_pages", load().cpa_compact_pages, index, stream, at, desc, False)


def device_status(k_cache, num_q_heads, max_pages_per_seq, workspace, stream=None) -> int:
    desc = make_desc(k_cache, num_q_heads, 0, max_pages_per_seq, workspace)
    return cpa_read_device_status(desc, _stream(stream))
