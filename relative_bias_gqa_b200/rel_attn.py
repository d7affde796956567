"""ctypes binding of the C ABI in include/rel_attn.h.

Argument marshalling only: every step of the operation runs in the CUDA
library.  Importing this module loads ``librel_attn.so`` and raises
ImportError if it has not been built; there is no fallback path.
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

from .build import LIB_PATH

REL_ATTN_OK = 0
REL_ATTN_ERR_INVALID_ARG = -1
REL_ATTN_ERR_WORKSPACE_TOO_SMALL = -2
REL_ATTN_ERR_CUDA = -3
REL_ATTN_ERR_TIMEOUT = -4
REL_ATTN_ERR_BAD_SEQ = -5
REL_ATTN_ERR_NO_DEVICE = -6
REL_ATTN_ERR_NO_PAGES = -7

EXPORTED = (
    "rel_attn_decode", "rel_attn_partial", "rel_attn_combine", "rel_attn_workspace_bytes", "rel_attn_workspace_init",
    "rel_attn_read_status", "rel_attn_choose_splits", "rel_attn_bucket",
    "rel_attn_error_string", "rel_attn_version", "rel_attn_decode_static",
    "rel_attn_split_pages", "rel_attn_decode_e4m3", "rel_attn_partial_e4m3",
    "rel_attn_set_wait_limit", "rel_attn_kv_write", "rel_attn_prefill",
    "rel_attn_split_pages_e4m3", "rel_attn_sink_decode", "rel_attn_sink_decode_e4m3",
    "rel_attn_sink_prefill", "rel_attn_sink_prefill_e4m3", "rel_attn_sink_workspace_bytes",
    "rel_attn_sink_prefill_workspace_bytes", "rel_attn_pages_resize",
    "rel_attn_pages_fork", "rel_attn_pages_compact", "rel_attn_pages_workspace_bytes",
)


class RelAttnShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in (
        "batch", "q_tokens", "num_q_heads", "num_kv_heads", "head_dim",
        "page_size", "num_pages", "max_pages_per_seq", "num_buckets",
        "exact_buckets", "max_distance", "max_seq_len", "out_fp32")]


class RelAttnPages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("num_seqs", "max_pages_per_seq", "num_pages")] + \
               [(n, ctypes.c_void_p) for n in ("block_table", "seq_lens", "page_refs")]


class RelAttnPool(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("page_bytes", ctypes.c_size_t)]


class RelAttnError(RuntimeError):
    def __init__(self, code: int):
        self.code = code
        super().__init__(f"rel_attn error {code}: {error_string(code)}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m relative_bias_gqa_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    SP = ctypes.POINTER(RelAttnShape)
    lib.rel_attn_decode.argtypes = [SP, P, P, P, P, P, P, ctypes.c_int, ctypes.c_int,
                                    P, P, P, ctypes.c_size_t, P]
    lib.rel_attn_decode.restype = ctypes.c_int
    lib.rel_attn_partial.argtypes = lib.rel_attn_decode.argtypes
    lib.rel_attn_partial.restype = ctypes.c_int
    lib.rel_attn_combine.argtypes = [SP, ctypes.c_int, P, P, P, ctypes.c_size_t, P]
    lib.rel_attn_combine.restype = ctypes.c_int
    lib.rel_attn_decode_e4m3.argtypes = [SP, P, P, P, P, P, P, P, P, ctypes.c_int, ctypes.c_int,
                                         P, P, P, ctypes.c_size_t, P]
    lib.rel_attn_decode_e4m3.restype = ctypes.c_int
    lib.rel_attn_partial_e4m3.argtypes = lib.rel_attn_decode_e4m3.argtypes
    lib.rel_attn_partial_e4m3.restype = ctypes.c_int
    lib.rel_attn_decode_static.argtypes = [SP, P, P, P, P, P, P, ctypes.c_int, ctypes.c_int,
                                           P, P, P]
    lib.rel_attn_decode_static.restype = ctypes.c_int
    lib.rel_attn_workspace_bytes.argtypes = [SP, ctypes.c_int]
    lib.rel_attn_workspace_bytes.restype = ctypes.c_size_t
    lib.rel_attn_workspace_init.argtypes = [P, ctypes.c_size_t, P]
    lib.rel_attn_workspace_init.restype = ctypes.c_int
    lib.rel_attn_read_status.argtypes = [P, P]
    lib.rel_attn_read_status.restype = ctypes.c_int
    lib.rel_attn_choose_splits.argtypes = [SP, ctypes.c_int, ctypes.c_int]
    lib.rel_attn_choose_splits.restype = ctypes.c_int
    lib.rel_attn_bucket.argtypes = [SP, ctypes.c_int]
    lib.rel_attn_bucket.restype = ctypes.c_int
    lib.rel_attn_split_pages.argtypes = [SP, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                         ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
    lib.rel_attn_split_pages.restype = ctypes.c_int
    lib.rel_attn_split_pages_e4m3.argtypes = lib.rel_attn_split_pages.argtypes
    lib.rel_attn_split_pages_e4m3.restype = ctypes.c_int
    lib.rel_attn_prefill.argtypes = lib.rel_attn_decode.argtypes
    lib.rel_attn_prefill.restype = ctypes.c_int
    lib.rel_attn_kv_write.argtypes = [SP, P, P, P, P, P, P, P, P, P, P, P, P, P]
    lib.rel_attn_kv_write.restype = ctypes.c_int
    I = ctypes.c_int
    lib.rel_attn_sink_decode.argtypes = [SP, P, P, P, P, P, P, I, I, I, P, P, P, ctypes.c_size_t, P]
    lib.rel_attn_sink_decode.restype = I
    lib.rel_attn_sink_decode_e4m3.argtypes = [SP, P, P, P, P, P, P, P, P, I, I, I, P, P, P,
                                              ctypes.c_size_t, P]
    lib.rel_attn_sink_decode_e4m3.restype = I
    lib.rel_attn_sink_prefill.argtypes = [SP, P, P, P, P, P, P, I, I, P, P, P, ctypes.c_size_t, P]
    lib.rel_attn_sink_prefill.restype = I
    lib.rel_attn_sink_prefill_e4m3.argtypes = [SP, P, P, P, P, P, P, P, P, I, I, P, P, P,
                                               ctypes.c_size_t, P]
    lib.rel_attn_sink_prefill_e4m3.restype = I
    lib.rel_attn_sink_workspace_bytes.argtypes = [SP, I, I, I]
    lib.rel_attn_sink_workspace_bytes.restype = ctypes.c_size_t
    lib.rel_attn_sink_prefill_workspace_bytes.argtypes = [SP, I, I]
    lib.rel_attn_sink_prefill_workspace_bytes.restype = ctypes.c_size_t
    GP, PP = ctypes.POINTER(RelAttnPages), ctypes.POINTER(RelAttnPool)
    lib.rel_attn_pages_resize.argtypes = [GP, P, I, I, P, ctypes.c_size_t, P]
    lib.rel_attn_pages_resize.restype = I
    lib.rel_attn_pages_fork.argtypes = [GP, P, P, I, I, PP, I, P, ctypes.c_size_t, P]
    lib.rel_attn_pages_fork.restype = I
    lib.rel_attn_pages_compact.argtypes = [GP, PP, I, P, P, ctypes.c_size_t, P]
    lib.rel_attn_pages_compact.restype = I
    lib.rel_attn_pages_workspace_bytes.argtypes = [GP]
    lib.rel_attn_pages_workspace_bytes.restype = ctypes.c_size_t
    lib.rel_attn_set_wait_limit.argtypes = [ctypes.c_ulonglong]
    lib.rel_attn_set_wait_limit.restype = ctypes.c_int
    lib.rel_attn_error_string.argtypes = [ctypes.c_int]
    lib.rel_attn_error_string.restype = ctypes.c_char_p
    lib.rel_attn_version.argtypes = []
    lib.rel_attn_version.restype = ctypes.c_char_p
    return lib


lib = _load()


def error_string(code: int) -> str:
    return lib.rel_attn_error_string(code).decode()


def version() -> str:
    return lib.rel_attn_version().decode()


def make_shape(*, batch, q_tokens, num_q_heads, num_kv_heads, num_pages,
               max_pages_per_seq, num_buckets, head_dim=128, page_size=64,
               exact_buckets=1024, max_distance=1 << 20, max_seq_len=0,
               out_fp32=False) -> RelAttnShape:
    return RelAttnShape(batch, q_tokens, num_q_heads, num_kv_heads, head_dim,
                        page_size, num_pages, max_pages_per_seq, num_buckets,
                        exact_buckets, max_distance, max_seq_len, int(out_fp32))


def shape_of(q, k_cache, block_table, rel_table, *, max_seq_len=0, out_fp32=False,
             exact_buckets=1024, max_distance=1 << 20) -> RelAttnShape:
    B, T, Hq, D = q.shape
    num_pages, Hkv, P, dim = k_cache.shape
    if dim != D or rel_table.shape[-1] != D:
        raise ValueError(f"head dims differ: q {D}, k_cache {dim}, rel_table {rel_table.shape[-1]}")
    return make_shape(batch=B, q_tokens=T, num_q_heads=Hq, num_kv_heads=Hkv,
                      num_pages=num_pages, max_pages_per_seq=block_table.shape[1],
                      num_buckets=rel_table.shape[1], head_dim=D, page_size=P,
                      exact_buckets=exact_buckets, max_distance=max_distance,
                      max_seq_len=max_seq_len, out_fp32=out_fp32)


def _check_caches(k_cache, *others) -> None:
    """Caches that one table names: read and written with k_cache's extents."""
    for t in others:
        if t.shape != k_cache.shape:
            raise ValueError(f"caches differ: {tuple(k_cache.shape)} and {tuple(t.shape)}")


def rel_attn_workspace_bytes(shape: RelAttnShape, num_splits: int = 0) -> int:
    return int(lib.rel_attn_workspace_bytes(ctypes.byref(shape), num_splits))


def rel_attn_choose_splits(shape: RelAttnShape, window: int, sm_count: int = 0) -> int:
    r = lib.rel_attn_choose_splits(ctypes.byref(shape), window, sm_count)
    if r < 0:
        raise RelAttnError(r)
    return r


def rel_attn_bucket(shape: RelAttnShape, distance: int) -> int:
    return int(lib.rel_attn_bucket(ctypes.byref(shape), int(distance)))


def rel_attn_split_pages(shape: RelAttnShape, seq_len: int, window: int, num_splits: int,
                         split: int, e4m3: bool = False):
    """(first_page, end_page) of one split, as the partial kernel (the E4M3
    one with e4m3=True) walks it."""
    a, b = ctypes.c_int(), ctypes.c_int()
    fn = lib.rel_attn_split_pages_e4m3 if e4m3 else lib.rel_attn_split_pages
    rc = fn(ctypes.byref(shape), int(seq_len), int(window), int(num_splits),
            int(split), ctypes.byref(a), ctypes.byref(b))
    if rc != REL_ATTN_OK:
        raise RelAttnError(rc)
    return a.value, b.value


def rel_attn_set_wait_limit(limit_ns: int) -> None:
    """Bound of each device-side wait in later launches (0: the 2 s default)."""
    lib.rel_attn_set_wait_limit(int(limit_ns))


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


class Workspace:
    """Caller-owned device scratch for rel_attn_decode (status word + partials)."""

    def __init__(self, nbytes: int, device):
        self.nbytes = max(int(nbytes), 256)
        self.buf = torch.empty(self.nbytes, dtype=torch.uint8, device=device)
        rc = lib.rel_attn_workspace_init(ctypes.c_void_p(self.buf.data_ptr()),
                                         self.nbytes, ctypes.c_void_p(_stream_ptr(None)))
        if rc != REL_ATTN_OK:
            raise RelAttnError(rc)

    @classmethod
    def for_shape(cls, shape: RelAttnShape, num_splits: int, device) -> "Workspace":
        n = rel_attn_workspace_bytes(shape, num_splits)
        if n == 0:
            raise RelAttnError(REL_ATTN_ERR_INVALID_ARG)
        return cls(n, device)

    def read_status(self, stream=None) -> int:
        return int(lib.rel_attn_read_status(ctypes.c_void_p(self.buf.data_ptr()),
                                            ctypes.c_void_p(_stream_ptr(stream))))


def rel_attn_decode(q, k_cache, v_cache, block_table, seq_lens, rel_table,
                    window: int = 0, num_splits: int = 0, out=None, lse=None,
                    workspace: Optional[Workspace] = None, *, max_seq_len: int = 0,
                    out_fp32: bool = False, exact_buckets: int = 1024,
                    max_distance: int = 1 << 20, stream=None, with_lse: bool = True):
    """Relative-bias GQA decode attention on the current CUDA device.

    q bf16 [B, T, Hq, D]; k_cache / v_cache bf16 [num_pages, Hkv, P, D];
    block_table int32 [B, max_pages]; seq_lens int32 [B]; rel_table bf16
    [Hkv, NB, D] -- all contiguous CUDA tensors.  Returns (out, lse).
    Supported: D = 128, P = 64, Hq / Hkv in {4, 6, 8} with T <= 9 (T <= 8
    for 8); other shapes raise RelAttnError (REL_ATTN_ERR_INVALID_ARG).
    """
    for name, t, dt in (("q", q, torch.bfloat16), ("k_cache", k_cache, torch.bfloat16),
                        ("v_cache", v_cache, torch.bfloat16), ("rel_table", rel_table, torch.bfloat16),
                        ("block_table", block_table, torch.int32), ("seq_lens", seq_lens, torch.int32)):
        if not t.is_cuda or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor")
    _check_caches(k_cache, v_cache)
    shape = shape_of(q, k_cache, block_table, rel_table, max_seq_len=max_seq_len,
                     out_fp32=out_fp32, exact_buckets=exact_buckets,
                     max_distance=max_distance)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32 if out_fp32 else torch.bfloat16,
                          device=q.device)
    if lse is None and with_lse:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = Workspace.for_shape(shape, num_splits, q.device)
    rc = lib.rel_attn_decode(
        ctypes.byref(shape), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        block_table.data_ptr(), seq_lens.data_ptr(), rel_table.data_ptr(),
        int(window), int(num_splits), out.data_ptr(),
        lse.data_ptr() if lse is not None else None,
        workspace.buf.data_ptr(), workspace.nbytes, _stream_ptr(stream))
    if rc != REL_ATTN_OK:
        raise RelAttnError(rc)
    return out, lse


def rel_attn_decode_e4m3(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens, rel_table,
                         window: int = 0, num_splits: int = 0, out=None, lse=None,
                         workspace: Optional[Workspace] = None, *, max_seq_len: int = 0,
                         out_fp32: bool = False, exact_buckets: int = 1024,
                         max_distance: int = 1 << 20, stream=None, with_lse: bool = True):
    """rel_attn_decode over an E4M3 KV cache: k_codes / v_codes uint8 (or
    float8_e4m3fn) [num_pages, Hkv, P, D], k_scale / v_scale fp32 [Hkv]."""
    if k_codes.dtype == torch.float8_e4m3fn:
        k_codes = k_codes.view(torch.uint8)
    if v_codes.dtype == torch.float8_e4m3fn:
        v_codes = v_codes.view(torch.uint8)
    for name, t, dt in (("q", q, torch.bfloat16), ("k_codes", k_codes, torch.uint8),
                        ("v_codes", v_codes, torch.uint8), ("k_scale", k_scale, torch.float32),
                        ("v_scale", v_scale, torch.float32), ("rel_table", rel_table, torch.bfloat16),
                        ("block_table", block_table, torch.int32), ("seq_lens", seq_lens, torch.int32)):
        if not t.is_cuda or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor")
    _check_caches(k_codes, v_codes)
    shape = shape_of(q, k_codes, block_table, rel_table, max_seq_len=max_seq_len,
                     out_fp32=out_fp32, exact_buckets=exact_buckets, max_distance=max_distance)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32 if out_fp32 else torch.bfloat16,
                          device=q.device)
    if lse is None and with_lse:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = Workspace.for_shape(shape, num_splits, q.device)
    rc = lib.rel_attn_decode_e4m3(
        ctypes.byref(shape), q.data_ptr(), k_codes.data_ptr(), v_codes.data_ptr(),
        k_scale.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
        rel_table.data_ptr(), int(window), int(num_splits), out.data_ptr(),
        lse.data_ptr() if lse is not None else None,
        workspace.buf.data_ptr(), workspace.nbytes, _stream_ptr(stream))
    if rc != REL_ATTN_OK:
        raise RelAttnError(rc)
    return out, lse


def rel_attn_prefill(q, k_cache, v_cache, block_table, seq_lens, rel_table, window: int = 0,
                     num_splits: int = 0, out=None, lse=None, workspace: Optional[Workspace] = None,
                     *, max_seq_len: int = 0, out_fp32: bool = False, exact_buckets: int = 1024,
                     max_distance: int = 1 << 20, stream=None, with_lse: bool = True):
    """Attention for all C query tokens of each sequence (q [B, C, Hq, D],
    token t at position seq_len - C + t, causal); arguments as for
    rel_attn_decode.  Returns (out, lse)."""
    for name, t, dt in (("q", q, torch.bfloat16), ("k_cache", k_cache, torch.bfloat16),
                        ("v_cache", v_cache, torch.bfloat16), ("rel_table", rel_table, torch.bfloat16),
                        ("block_table", block_table, torch.int32), ("seq_lens", seq_lens, torch.int32)):
        if not t.is_cuda or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor")
    _check_caches(k_cache, v_cache)
    shape = shape_of(q, k_cache, block_table, rel_table, max_seq_len=max_seq_len,
                     out_fp32=out_fp32, exact_buckets=exact_buckets, max_distance=max_distance)
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32 if out_fp32 else torch.bfloat16,
                          device=q.device)
    if lse is None and with_lse:
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
    if workspace is None:
        n = prefill_workspace_bytes(shape, num_splits)
        workspace = Workspace(n, q.device)
    rc = lib.rel_attn_prefill(
        ctypes.byref(shape), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        block_table.data_ptr(), seq_lens.data_ptr(), rel_table.data_ptr(),
        int(window), int(num_splits), out.data_ptr(),
        lse.data_ptr() if lse is not None else None,
        workspace.buf.data_ptr(), workspace.nbytes, _stream_ptr(stream))
    if rc != REL_ATTN_OK:
        raise RelAttnError(rc)
    return out, lse


def prefill_workspace_bytes(shape: RelAttnShape, num_splits: int) -> int:
    """Workspace bytes rel_attn_prefill needs: the status word, plus, with
    more than one split, every row's partials (the layout of the decode
    workspace for B * C rows).  num_splits <= 0 assumes up to 256."""
    S = num_splits if num_splits > 0 else 256
    rows = shape.batch * shape.q_tokens * shape.num_q_heads
    if S == 1:
        return 256
    return 256 + (S * rows * 4 + 255) // 256 * 256 + S * rows * 128 * 4


def rel_attn_kv_write(k_new, v_new, conv_w, k_raw, v_raw, k_cache, v_cache, block_table,
                      seq_lens, k_scale=None, v_scale=None, workspace: Optional[Workspace] = None,
                      stream=None):
    """The KV-cache producer step (see include/rel_attn.h): short convolution
    of the T new tokens' K/V (k_new / v_new bf16 [B, T, Hkv, D], taps conv_w
    bf16 [2, Hkv, D, 4]), raw K/V into the sconv cache k_raw / v_raw, the
    convolved K/V into k_cache / v_cache (bf16, or uint8 / float8_e4m3fn
    E4M3 codes with k_scale / v_scale fp32 [Hkv]).  In place; returns None."""
    if k_cache.dtype == torch.float8_e4m3fn:
        k_cache = k_cache.view(torch.uint8)
    if v_cache.dtype == torch.float8_e4m3fn:
        v_cache = v_cache.view(torch.uint8)
    e4m3 = k_scale is not None
    cache_dt = torch.uint8 if e4m3 else torch.bfloat16
    checks = [("k_new", k_new, torch.bfloat16), ("v_new", v_new, torch.bfloat16),
              ("conv_w", conv_w, torch.bfloat16), ("k_raw", k_raw, torch.bfloat16),
              ("v_raw", v_raw, torch.bfloat16), ("k_cache", k_cache, cache_dt),
              ("v_cache", v_cache, cache_dt), ("block_table", block_table, torch.int32),
              ("seq_lens", seq_lens, torch.int32)]
    if e4m3:
        checks += [("k_scale", k_scale, torch.float32), ("v_scale", v_scale, torch.float32)]
    for name, t, dt in checks:
        if not t.is_cuda or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor")
    B, T, Hkv, D = k_new.shape
    if tuple(k_cache.shape[1::2]) != (Hkv, D) or v_new.shape != k_new.shape or tuple(conv_w.shape) != (2, Hkv, D, 4):
        raise ValueError("heads and head dims of k_new, v_new, conv_w and the caches differ")
    _check_caches(k_cache, v_cache, k_raw, v_raw)
    shape = make_shape(batch=B, q_tokens=T, num_q_heads=Hkv, num_kv_heads=Hkv,
                       num_pages=k_cache.shape[0], max_pages_per_seq=block_table.shape[1],
                       num_buckets=1, head_dim=D, page_size=k_cache.shape[2])
    rc = lib.rel_attn_kv_write(
        ctypes.byref(shape), k_new.data_ptr(), v_new.data_ptr(), conv_w.data_ptr(),
        k_raw.data_ptr(), v_raw.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        k_scale.data_ptr() if e4m3 else None, v_scale.data_ptr() if e4m3 else None,
        block_table.data_ptr(), seq_lens.data_ptr(),
        workspace.buf.data_ptr() if workspace is not None else None, _stream_ptr(stream))
    if rc != REL_ATTN_OK:
        raise RelAttnError(rc)


class Prepared:
    """A decode call with every argument marshalled once (shape struct, raw
    pointers, workspace), for callers that issue the same call repeatedly.
    ``decode()`` runs rel_attn_decode; ``partial()`` / ``combine()`` run the
    split-phase pair.  Tensors must stay alive and unmoved while in use."""

    def __init__(self, q, k_cache, v_cache, block_table, seq_lens, rel_table, window=0,
                 num_splits=0, *, out=None, lse=None, max_seq_len=0, out_fp32=False,
                 exact_buckets=1024, max_distance=1 << 20, stream=None, k_scale=None,
                 v_scale=None):
        _check_caches(k_cache, v_cache)
        self.shape = shape_of(q, k_cache, block_table, rel_table, max_seq_len=max_seq_len,
                              out_fp32=out_fp32, exact_buckets=exact_buckets,
                              max_distance=max_distance)
        if num_splits <= 0:
            num_splits = rel_attn_choose_splits(self.shape, window, 0)
        self.num_splits = num_splits
        self.out = out if out is not None else torch.empty(
            q.shape, dtype=torch.float32 if out_fp32 else torch.bfloat16, device=q.device)
        self.lse = lse if lse is not None else torch.empty(q.shape[:3], dtype=torch.float32,
                                                           device=q.device)
        self.workspace = Workspace.for_shape(self.shape, num_splits, q.device)
        self.window = int(window)
        self.stream = stream
        # an E4M3 KV cache (uint8 codes) comes with its per-KV-head scales
        self.e4m3 = k_scale is not None
        if self.e4m3 != (v_scale is not None):
            raise ValueError("k_scale and v_scale go together")
        self._keep = (q, k_cache, v_cache, block_table, seq_lens, rel_table, k_scale, v_scale)
        scales = (k_scale.data_ptr(), v_scale.data_ptr()) if self.e4m3 else ()
        self._args = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), *scales,
                      block_table.data_ptr(), seq_lens.data_ptr(), rel_table.data_ptr())

    def _common(self):
        return (ctypes.byref(self.shape), *self._args, self.window, self.num_splits,
                self.out.data_ptr(), self.lse.data_ptr(), self.workspace.buf.data_ptr(),
                self.workspace.nbytes, _stream_ptr(self.stream))

    def decode(self):
        rc = (lib.rel_attn_decode_e4m3 if self.e4m3 else lib.rel_attn_decode)(*self._common())
        if rc != REL_ATTN_OK:
            raise RelAttnError(rc)
        return self.out, self.lse

    def partial(self):
        rc = (lib.rel_attn_partial_e4m3 if self.e4m3 else lib.rel_attn_partial)(*self._common())
        if rc != REL_ATTN_OK:
            raise RelAttnError(rc)

    def combine(self):
        rc = lib.rel_attn_combine(ctypes.byref(self.shape), self.num_splits, self.out.data_ptr(),
                                  self.lse.data_ptr(), self.workspace.buf.data_ptr(),
                                  self.workspace.nbytes, _stream_ptr(self.stream))
        if rc != REL_ATTN_OK:
            raise RelAttnError(rc)


# ------------------------------------------------- sliding window with sinks
def _raw_stream(stream) -> int:
    """_stream_ptr without a Stream object for the current one (a short step's
    launch costs about as much on the host as on the device)."""
    if stream is not None:
        return int(stream.cuda_stream)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _on(stream):
    """Allocations and initialisations in the order of the stream that uses them."""
    return torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()


def _int32(name, value) -> int:
    value = int(value)
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{name} = {value} does not fit 32 bits")
    return value


def _check_device(device: int) -> None:
    if torch._C._cuda_getDevice() != device:
        raise RuntimeError(f"the tensors are on cuda:{device}, which is not the current device")


def _check_rows(name, t, like) -> None:
    """An int32 tensor of one dimension beside ``like``, which was checked."""
    if t.dtype is not torch.int32 or t.dim() != 1 or not t.is_contiguous() or t.device != like.device:
        raise ValueError(f"{name} must be a contiguous torch.int32 tensor of one dimension on {like.device}")


def _check_written(name, t, device, host=False) -> None:
    """Memory that kernels on ``device`` write: its own, or (``host``) mapped pinned host memory."""
    if t.device != device and not (host and t.device.type == "cpu" and t.is_pinned()):
        raise ValueError(f"{name} is on {t.device}, not on {device}" + (" or in pinned host memory" if host else ""))


def _codes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _check_tensors(checks):
    """Contiguous tensors of the given type, all on the current CUDA device."""
    for name, t, dt, shape in checks:
        if not t.is_cuda or t.dtype != dt or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor")
        if t.device.index != torch.cuda.current_device():
            raise ValueError(f"{name} is on {t.device}, not on the current device")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")


class SinkPrepared:
    """A sliding-window-with-sinks call (rel_attn_sink_decode, with ``prefill``
    rel_attn_sink_prefill; with k_scale and v_scale their E4M3 forms) with
    every argument checked and marshalled once, for repeated launches over the
    same buffers.  ``run()`` launches it on the current stream (or the one
    given) and returns (out, lse).  ``num_splits`` is a decode's: with
    ``prefill`` it is not used (the library splits by the number of query
    tiles, where the workspace has the room).  out and lse may be in pinned
    host memory.  Tensors must stay alive and unmoved."""

    def __init__(self, q, k_cache, v_cache, block_table, seq_lens, rel_table, window, num_sinks=0,
                 num_splits=0, *, prefill=False, out=None, lse=None, workspace=None, max_seq_len=0,
                 out_fp32=False, exact_buckets=1024, max_distance=1 << 20, stream=None,
                 k_scale=None, v_scale=None, with_lse=True):
        if (k_scale is None) != (v_scale is None):
            raise ValueError("k_scale and v_scale go together")
        e4m3 = k_scale is not None
        window, num_sinks, num_splits = _int32("window", window), _int32("num_sinks", num_sinks), _int32("num_splits", num_splits)
        k_cache, v_cache = _codes(k_cache), _codes(v_cache)
        if q.dim() != 4 or k_cache.dim() != 4 or rel_table.dim() != 3 or block_table.dim() != 2:
            raise ValueError("q and the caches have 4 dimensions, rel_table 3, block_table 2")
        B, T, Hq, D = q.shape
        Hkv = k_cache.shape[1]
        with _on(stream):
            if out is None:
                out = torch.empty(q.shape, dtype=torch.float32 if out_fp32 else torch.bfloat16, device=q.device)
            if lse is None and with_lse:
                lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device)
        cache = torch.uint8 if e4m3 else torch.bfloat16
        checks = [("q", q, torch.bfloat16, None), ("k_cache", k_cache, cache, None),
                  ("v_cache", v_cache, cache, k_cache.shape),
                  ("rel_table", rel_table, torch.bfloat16, (Hkv, rel_table.shape[1], D)),
                  ("block_table", block_table, torch.int32, (B, block_table.shape[1])),
                  ("seq_lens", seq_lens, torch.int32, (B,))]
        if e4m3:
            checks += [("k_scale", k_scale, torch.float32, (Hkv,)), ("v_scale", v_scale, torch.float32, (Hkv,))]
        _check_tensors(checks)
        # (out and lse may also be mapped pinned host memory)
        for name, t, dt, shape in (("out", out, torch.float32 if out_fp32 else torch.bfloat16, q.shape),
                                   ("lse", lse, torch.float32, q.shape[:3])):
            if t is not None:
                if t.dtype != dt or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
                    raise ValueError(f"{name} must be a contiguous {dt} tensor of shape {tuple(shape)}")
                _check_written(name, t, q.device, host=True)
        if workspace is not None:
            _check_written("workspace", workspace.buf, q.device)
        self.shape = shape_of(q, k_cache, block_table, rel_table, max_seq_len=max_seq_len, out_fp32=out_fp32,
                              exact_buckets=exact_buckets, max_distance=max_distance)
        if workspace is None:
            ref = ctypes.byref(self.shape)
            n = int(lib.rel_attn_sink_prefill_workspace_bytes(ref, window, num_sinks) if prefill else
                    lib.rel_attn_sink_workspace_bytes(ref, window, num_sinks, num_splits))
            if n == 0:
                raise RelAttnError(REL_ATTN_ERR_INVALID_ARG)
            with _on(stream):
                workspace = Workspace(n, q.device)
        self.out, self.lse, self.workspace = out, lse, workspace
        self.stream, self._device = stream, q.device.index
        self._keep = (q, k_cache, v_cache, block_table, seq_lens, rel_table, k_scale, v_scale)
        P, I = ctypes.c_void_p, ctypes.c_int
        scales = [P(k_scale.data_ptr()), P(v_scale.data_ptr())] if e4m3 else []
        self._fn = getattr(lib, ("rel_attn_sink_prefill" if prefill else "rel_attn_sink_decode") + ("_e4m3" if e4m3 else ""))
        self._args = [ctypes.byref(self.shape), P(q.data_ptr()), P(k_cache.data_ptr()), P(v_cache.data_ptr()),
                      *scales, P(block_table.data_ptr()), P(seq_lens.data_ptr()), P(rel_table.data_ptr()),
                      I(window), I(num_sinks), *([] if prefill else [I(num_splits)]),
                      P(out.data_ptr()), P(lse.data_ptr() if lse is not None else None),
                      P(workspace.buf.data_ptr()), ctypes.c_size_t(workspace.nbytes)]

    def run(self):
        _check_device(self._device)
        rc = self._fn(*self._args, _raw_stream(self.stream))
        if rc != REL_ATTN_OK:
            raise RelAttnError(rc)
        return self.out, self.lse


def rel_attn_sink_decode(q, k_cache, v_cache, block_table, seq_lens, rel_table, window, num_sinks=0,
                         num_splits=0, out=None, lse=None, workspace: Optional[Workspace] = None, **kw):
    """A decode or verify step (q bf16 [B, T, Hq, 128], T = 1..9) over a
    sliding window of ``window`` keys and the first ``num_sinks`` positions:
    token t at position p sees j <= p with j < num_sinks or p - j < window.
    Tensors as for rel_attn_decode; a row with seq_lens 0 is a free slot (out
    zeros, lse -inf).  Block-table entries that hold no visible key are never
    read.  Returns (out, lse); other keywords as for SinkPrepared."""
    return SinkPrepared(q, k_cache, v_cache, block_table, seq_lens, rel_table, window, num_sinks, num_splits,
                        out=out, lse=lse, workspace=workspace, **kw).run()


def rel_attn_sink_decode_e4m3(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens, rel_table, window,
                              num_sinks=0, num_splits=0, out=None, lse=None,
                              workspace: Optional[Workspace] = None, **kw):
    """rel_attn_sink_decode over an E4M3 cache: k_codes / v_codes uint8 (or
    float8_e4m3fn), k_scale / v_scale fp32 [Hkv]."""
    return SinkPrepared(q, k_codes, v_codes, block_table, seq_lens, rel_table, window, num_sinks, num_splits,
                        out=out, lse=lse, workspace=workspace, k_scale=k_scale, v_scale=v_scale, **kw).run()


def rel_attn_sink_prefill(q, k_cache, v_cache, block_table, seq_lens, rel_table, window, num_sinks=0,
                          out=None, lse=None, workspace: Optional[Workspace] = None, **kw):
    """The same attention for all C query tokens of each sequence (q bf16
    [B, C, Hq, 128], token t at position seq_len - C + t, causal)."""
    return SinkPrepared(q, k_cache, v_cache, block_table, seq_lens, rel_table, window, num_sinks, prefill=True,
                        out=out, lse=lse, workspace=workspace, **kw).run()


def rel_attn_sink_prefill_e4m3(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens, rel_table, window,
                               num_sinks=0, out=None, lse=None, workspace: Optional[Workspace] = None, **kw):
    """rel_attn_sink_prefill over an E4M3 cache."""
    return SinkPrepared(q, k_codes, v_codes, block_table, seq_lens, rel_table, window, num_sinks, prefill=True,
                        out=out, lse=lse, workspace=workspace, k_scale=k_scale, v_scale=v_scale, **kw).run()


# --------------------------------------------------------- pages of the cache
class Pages:
    """The pages of a cache: block_table int32 [rows, max_pages], seq_lens
    int32 [rows], page_refs int32 [num_pages] (references of each page, 0:
    free) and the pools whose pages they name (contiguous, [num_pages, ...]).
    The calls change them in place, on the current stream (or the one given);
    where the device finds an error they change nothing, and read_status()
    says which: REL_ATTN_ERR_NO_PAGES or REL_ATTN_ERR_BAD_SEQ.  Tensors must
    stay alive and unmoved."""

    def __init__(self, block_table, seq_lens, page_refs, pools=(), workspace: Optional[Workspace] = None,
                 stream=None):
        if block_table.dim() != 2:
            raise ValueError("block_table has 2 dimensions")
        rows, n = block_table.shape[0], page_refs.numel()
        if n == 0:
            raise ValueError("page_refs is empty: a pool has at least one page")
        _check_tensors([("block_table", block_table, torch.int32, None), ("seq_lens", seq_lens, torch.int32, (rows,)),
                        ("page_refs", page_refs, torch.int32, (n,))])
        pools = tuple(pools)
        for i, t in enumerate(pools):
            _check_tensors([(f"pools[{i}]", t, t.dtype, (n, *t.shape[1:]))])
        self.block_table, self.seq_lens, self.page_refs, self.pools = block_table, seq_lens, page_refs, pools
        self.stream, self._device, self._rows = stream, block_table.device.index, rows
        self._resize, self._fork, self._compact = lib.rel_attn_pages_resize, lib.rel_attn_pages_fork, lib.rel_attn_pages_compact
        self._c = RelAttnPages(rows, block_table.shape[1], n, block_table.data_ptr(), seq_lens.data_ptr(),
                               page_refs.data_ptr())
        self._pools = (RelAttnPool * max(1, len(pools)))(
            *[RelAttnPool(t.data_ptr(), t.numel() // n * t.element_size()) for t in pools])
        if workspace is None:
            need = int(lib.rel_attn_pages_workspace_bytes(ctypes.byref(self._c)))
            if need == 0:
                raise RelAttnError(REL_ATTN_ERR_INVALID_ARG)
            with _on(stream):
                workspace = Workspace(need, block_table.device)
        _check_written("workspace", workspace.buf, block_table.device)
        self.workspace = workspace
        self._book, self._count = ctypes.byref(self._c), ctypes.c_int(len(pools))
        self._ws = (ctypes.c_void_p(workspace.buf.data_ptr()), ctypes.c_size_t(workspace.nbytes))

    def resize(self, new_lens, window: int = 0, num_sinks: int = 0):
        """Every row to new_lens (int32 [rows]) positions: pages past them and
        pages that left the window (the first num_sinks positions stay) are
        given back, new positions get pages."""
        _check_device(self._device)
        _check_rows("new_lens", new_lens, self.block_table)
        if new_lens.shape[0] != self._rows:
            raise ValueError(f"new_lens has shape {tuple(new_lens.shape)}, not {tuple(self.seq_lens.shape)}")
        if not (-0x80000000 <= window <= 0x7FFFFFFF and -0x80000000 <= num_sinks <= 0x7FFFFFFF):
            raise ValueError("window and num_sinks fit 32 bits")
        rc = self._resize(self._book, new_lens.data_ptr(), window, num_sinks, *self._ws, _raw_stream(self.stream))
        if rc != REL_ATTN_OK:
            raise RelAttnError(rc)

    def fork(self, src_rows, dst_rows, copy_all: bool = False):
        """Rows dst_rows (free ones) continue rows src_rows (int32 [n] each):
        full pages are shared, the last one (copy_all: every one) copied."""
        _check_device(self._device)
        _check_rows("src_rows", src_rows, self.block_table)
        _check_rows("dst_rows", dst_rows, self.block_table)
        if src_rows.shape != dst_rows.shape:
            raise ValueError("src_rows and dst_rows have the same number of rows")
        rc = self._fork(self._book, src_rows.data_ptr(), dst_rows.data_ptr(), src_rows.shape[0], 1 if copy_all else 0,
                        self._pools, self._count, *self._ws, _raw_stream(self.stream))
        if rc != REL_ATTN_OK:
            raise RelAttnError(rc)

    def compact(self, num_live):
        """The live pages to the front of the pools; their number into
        num_live (int32 [1])."""
        _check_device(self._device)
        _check_rows("num_live", num_live, self.block_table)
        if num_live.shape[0] != 1:
            raise ValueError("num_live has one element")
        rc = self._compact(self._book, self._pools, self._count, num_live.data_ptr(), *self._ws, _raw_stream(self.stream))
        if rc != REL_ATTN_OK:
            raise RelAttnError(rc)

    def read_status(self, stream=None) -> int:
        """The device status since the last reading (see the class); after
        REL_ATTN_ERR_TIMEOUT the state may be partly changed, and the workspace
        is initialised anew."""
        stream = stream if stream is not None else self.stream
        status = self.workspace.read_status(stream)
        if status == REL_ATTN_ERR_TIMEOUT:
            rc = lib.rel_attn_workspace_init(*self._ws, _raw_stream(stream))
            if rc != REL_ATTN_OK:
                raise RelAttnError(rc)
        return status
