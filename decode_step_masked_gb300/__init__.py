"""Python binding of the GB300 masked multi-head attention decode step.

Argument marshalling only: every entry point of ``include/ftd.h`` is exposed
under the same name and forwards plain integers (device or host addresses)
and sizes to ``_build/libftd.so`` through ctypes.  All decode work runs in
the library's CUDA kernels; there is no CPU path here.  If the library has
not been built, ``load_library`` raises instead of falling back.

``DecodeStep`` is a convenience wrapper for callers holding torch tensors:
it reads ``data_ptr()`` and the current CUDA stream and calls the same ABI.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

from ._build import LIB, build_library  # noqa: F401

FTD_OK = 0
FTD_ERR_INVALID_ARG = 1
FTD_ERR_UNSUPPORTED = 2
FTD_ERR_OOM = 3
FTD_ERR_CUDA = 4
FTD_ERR_SEQ_OVERFLOW = 5
FTD_ERR_DEVICE_TIMEOUT = 6
FTD_ERR_BAD_PAGE = 7

FTD_F32, FTD_F16, FTD_BF16, FTD_I8 = 0, 1, 2, 3
FTD_KERNEL_AUTO, FTD_KERNEL_CUDA_CORE = 0, 1
FTD_ROPE_HALVES, FTD_ROPE_ADJACENT = 0, 1
FTD_ROPE_SECTIONS, FTD_ROPE_INTERLEAVED = 0, 1
DTYPES = {"f32": FTD_F32, "f16": FTD_F16, "bf16": FTD_BF16, "i8": FTD_I8}

# Symbols include/ftd.h declares; the loader checks each one is exported.
EXPORTS = ("ftd_init", "ftd_cache_ptrs", "ftd_decode_mha", "ftd_decode_mha_current", "ftd_decode_mha_paged",
           "ftd_decode_mha_host", "ftd_get_error", "ftd_destroy", "ftd_status_str", "ftd_last_error",
           "ftd_kernel_launches", "ftd_decode_mha_noalloc", "ftd_debug_stall_next",
           "ftd_debug_late_lengths", "ftd_debug_kernel", "ftd_decode_mha_proj", "ftd_set_rope", "ftd_rope_qkv", "ftd_enable_scores",
           "ftd_decode_mha_scored", "ftd_cache_evict", "ftd_cross_mha", "ftd_norm_rope_qkv", "ftd_build_tables",
           "ftd_enable_prefix", "ftd_decode_mha_prefix")


class FtdConfig(ctypes.Structure):
    _fields_ = [("max_batch", ctypes.c_int), ("n_q_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("max_len", ctypes.c_int), ("qkv_dtype", ctypes.c_int),
                ("cache_dtype", ctypes.c_int), ("softmax_scale", ctypes.c_float),
                ("out_dtype", ctypes.c_int), ("window", ctypes.c_int), ("page_size", ctypes.c_int),
                ("num_pages", ctypes.c_int), ("q_len", ctypes.c_int), ("kernel", ctypes.c_int),
                ("proj_dim", ctypes.c_int), ("wait_limit_us", ctypes.c_int)]


class FtdRopeConfig(ctypes.Structure):
    _fields_ = [("n_axes", ctypes.c_int), ("rotary_dim", ctypes.c_int), ("section", ctypes.c_int * 4),
                ("pairing", ctypes.c_int), ("order", ctypes.c_int), ("theta", ctypes.c_double),
                ("inv_freq", ctypes.POINTER(ctypes.c_double))]


class FtdError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{ftd_status_str(status)}: {message}")
        self.status = status


_lib: Optional[ctypes.CDLL] = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load the built library (``_build/libftd.so``) and declare its signatures."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or LIB
    if not os.path.exists(path):
        raise FileNotFoundError(
            f"{path} is missing: build it with decode_step_masked_gb300.build_library() "
            "(there is no fallback implementation)")
    lib = ctypes.CDLL(path)
    for name in EXPORTS:
        getattr(lib, name)  # AttributeError if a declared symbol is not exported
    P, I = ctypes.c_void_p, ctypes.c_int
    lib.ftd_init.argtypes = [ctypes.POINTER(FtdConfig), P, ctypes.POINTER(P)]
    lib.ftd_init.restype = I
    lib.ftd_cache_ptrs.argtypes = [P, ctypes.POINTER(P), ctypes.POINTER(P), ctypes.POINTER(P)]
    lib.ftd_cache_ptrs.restype = I
    for fn in (lib.ftd_decode_mha, lib.ftd_decode_mha_host):
        fn.argtypes = [P] * 11
        fn.restype = I
    lib.ftd_decode_mha_current.argtypes = [P] * 10
    lib.ftd_decode_mha_current.restype = I
    lib.ftd_decode_mha_paged.argtypes = [P] * 12
    lib.ftd_decode_mha_paged.restype = I
    lib.ftd_decode_mha_proj.argtypes = [P] * 13
    lib.ftd_decode_mha_proj.restype = I
    lib.ftd_get_error.argtypes = [P]
    lib.ftd_get_error.restype = I
    lib.ftd_destroy.argtypes = [P]
    lib.ftd_destroy.restype = None
    lib.ftd_status_str.argtypes = [I]
    lib.ftd_status_str.restype = ctypes.c_char_p
    lib.ftd_last_error.argtypes = []
    lib.ftd_last_error.restype = ctypes.c_char_p
    lib.ftd_kernel_launches.argtypes = []
    lib.ftd_kernel_launches.restype = ctypes.c_uint64
    lib.ftd_decode_mha_noalloc.argtypes = [ctypes.POINTER(FtdConfig)] + [P] * 11
    lib.ftd_decode_mha_noalloc.restype = I
    lib.ftd_debug_stall_next.argtypes = [P, I]
    lib.ftd_debug_stall_next.restype = I
    lib.ftd_set_rope.argtypes = [P, ctypes.POINTER(FtdRopeConfig)]
    lib.ftd_set_rope.restype = I
    lib.ftd_rope_qkv.argtypes = [P] * 4 + [ctypes.c_int64] * 2 + [P] * 2 + [ctypes.c_int64] + [P] * 4
    lib.ftd_rope_qkv.restype = I
    lib.ftd_norm_rope_qkv.argtypes = ([P] * 4 + [ctypes.c_int64] * 2 + [P] * 3 + [ctypes.c_float] * 2 + [P, ctypes.c_int64] +
                                      [P] * 8)
    lib.ftd_norm_rope_qkv.restype = I
    lib.ftd_build_tables.argtypes = [P] * 11 + [ctypes.c_int64, P]
    lib.ftd_build_tables.restype = I
    lib.ftd_enable_prefix.argtypes = [P, P]
    lib.ftd_enable_prefix.restype = I
    lib.ftd_decode_mha_prefix.argtypes = [P] * 14 + [ctypes.c_int64] + [P] * 3
    lib.ftd_decode_mha_prefix.restype = I
    lib.ftd_enable_scores.argtypes = [P, P]
    lib.ftd_enable_scores.restype = I
    lib.ftd_decode_mha_scored.argtypes = [P] * 16
    lib.ftd_decode_mha_scored.restype = I
    lib.ftd_cache_evict.argtypes = [P] * 12 + [I] * 3 + [P]
    lib.ftd_cache_evict.restype = I
    lib.ftd_cross_mha.argtypes = [P] * 9
    lib.ftd_cross_mha.restype = I
    lib.ftd_debug_kernel.argtypes = [P, I, ctypes.POINTER(I), ctypes.POINTER(I)]
    lib.ftd_debug_kernel.restype = I
    lib.ftd_debug_late_lengths.argtypes = [P, P, I, I, P]
    lib.ftd_debug_late_lengths.restype = I
    if path == LIB:
        _lib = lib
    return lib


# ------------------------------------------------------------ same-name ABI
def ftd_status_str(status: int) -> str:
    return load_library().ftd_status_str(int(status)).decode()


def ftd_last_error() -> str:
    return load_library().ftd_last_error().decode()


def ftd_kernel_launches() -> int:
    return int(load_library().ftd_kernel_launches())


def ftd_init(cfg: FtdConfig, stream: int = 0):
    """Returns (status, ctx handle as int or None)."""
    h = ctypes.c_void_p()
    st = load_library().ftd_init(ctypes.byref(cfg), ctypes.c_void_p(stream or None), ctypes.byref(h))
    return st, h.value


def ftd_cache_ptrs(ctx: int):
    k, v, s = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    st = load_library().ftd_cache_ptrs(ctypes.c_void_p(ctx), ctypes.byref(k), ctypes.byref(v), ctypes.byref(s))
    return st, k.value, v.value, s.value


def _ptrs(*xs):
    # Addresses go through as Python ints (or None): the argtypes declare them
    # c_void_p, and ctypes converts ints itself, without a wrapper object per
    # argument on the per-step path.
    return xs


def ftd_decode_mha(ctx, q, k_new, v_new, qkv_bias, k_cache, v_cache, seq_lens, scales, out, stream) -> int:
    return load_library().ftd_decode_mha(*_ptrs(ctx, q, k_new, v_new, qkv_bias, k_cache, v_cache, seq_lens,
                                                scales, out, stream))


def ftd_decode_mha_current(q, k_new, v_new, qkv_bias, k_cache, v_cache, seq_lens, scales, out, stream) -> int:
    return load_library().ftd_decode_mha_current(*_ptrs(q, k_new, v_new, qkv_bias, k_cache, v_cache, seq_lens,
                                                        scales, out, stream))


def ftd_decode_mha_paged(ctx, q, k_new, v_new, qkv_bias, k_pages, v_pages, block_table, seq_lens, scales, out,
                         stream) -> int:
    return load_library().ftd_decode_mha_paged(*_ptrs(ctx, q, k_new, v_new, qkv_bias, k_pages, v_pages,
                                                      block_table, seq_lens, scales, out, stream))


def ftd_decode_mha_proj(ctx, q, k_new, v_new, qkv_bias, k_cache, v_cache, seq_lens, scales, out, w_o, y,
                        stream) -> int:
    return load_library().ftd_decode_mha_proj(*_ptrs(ctx, q, k_new, v_new, qkv_bias, k_cache, v_cache, seq_lens,
                                                     scales, out, w_o, y, stream))


def ftd_set_rope(ctx, cfg: Optional[FtdRopeConfig]) -> int:
    return load_library().ftd_set_rope(ctx, ctypes.byref(cfg) if cfg is not None else None)


def ftd_rope_qkv(ctx, q, k, v, q_stride, kv_stride, qkv_bias, positions, n_tokens, q_out, k_out, v_out,
                 stream) -> int:
    return load_library().ftd_rope_qkv(ctx, q, k, v, q_stride, kv_stride, qkv_bias, positions, n_tokens, q_out, k_out,
                                       v_out, stream)


def ftd_norm_rope_qkv(ctx, q, k, v, q_stride, kv_stride, qkv_bias, q_weight, k_weight, eps, weight_offset, positions, n_tokens,
                      q_out, k_out, v_out, slots, k_cache, v_cache, scales, stream) -> int:
    return load_library().ftd_norm_rope_qkv(ctx, q, k, v, q_stride, kv_stride, qkv_bias, q_weight, k_weight, eps,
                                            weight_offset, positions, n_tokens, q_out, k_out, v_out, slots, k_cache,
                                            v_cache, scales, stream)


def ftd_build_tables(ctx, old_lens, new_lens, served, block_table, free_pages, n_free, n_free_out, offsets, slots, positions,
                     max_tokens, stream) -> int:
    return load_library().ftd_build_tables(ctx, old_lens, new_lens, served, block_table, free_pages, n_free, n_free_out,
                                           offsets, slots, positions, max_tokens, stream)


def ftd_enable_prefix(ctx, stream) -> int:
    return load_library().ftd_enable_prefix(ctx, stream)


def ftd_decode_mha_prefix(ctx, q, k_new, v_new, qkv_bias, k_cache, v_cache, block_table, seq_lens, scales, k_prefix, v_prefix,
                          prefix_scales, prefix_table, prefix_rows, prefix_lens, out, stream) -> int:
    return load_library().ftd_decode_mha_prefix(ctx, q, k_new, v_new, qkv_bias, k_cache, v_cache, block_table, seq_lens,
                                                scales, k_prefix, v_prefix, prefix_scales, prefix_table, prefix_rows,
                                                prefix_lens, out, stream)


def ftd_enable_scores(ctx, stream) -> int:
    return load_library().ftd_enable_scores(ctx, stream)


def ftd_decode_mha_scored(ctx, q, k_new, v_new, qkv_bias, k_cache, v_cache, block_table, seq_lens, scales, next_pos,
                          acc, acc_out, positions, out, stream) -> int:
    return load_library().ftd_decode_mha_scored(ctx, q, k_new, v_new, qkv_bias, k_cache, v_cache, block_table,
                                                seq_lens, scales, next_pos, acc, acc_out, positions, out, stream)


def ftd_cache_evict(ctx, k_cache, v_cache, scales, block_table, seq_lens, next_pos, acc, acc_out, positions,
                    positions_out, new_lens, budget, recent, sinks, stream) -> int:
    return load_library().ftd_cache_evict(ctx, k_cache, v_cache, scales, block_table, seq_lens, next_pos, acc, acc_out,
                                          positions, positions_out, new_lens, budget, recent, sinks, stream)


def ftd_cross_mha(ctx, q, q_bias, k_mem, v_mem, mem_lens, scales, out, stream) -> int:
    return load_library().ftd_cross_mha(ctx, q, q_bias, k_mem, v_mem, mem_lens, scales, out, stream)


def ftd_decode_mha_host(ctx, q, k_new, v_new, qkv_bias, k_cache, v_cache, seq_lens, scales, out,
                        stream) -> int:
    return load_library().ftd_decode_mha_host(*_ptrs(ctx, q, k_new, v_new, qkv_bias, k_cache, v_cache,
                                                     seq_lens, scales, out, stream))


def ftd_decode_mha_noalloc(cfg: FtdConfig, q, k_new, v_new, qkv_bias, k_cache, v_cache, seq_lens, scales, out,
                           device_err, stream) -> int:
    """The decode step without a context: scratch lives in the library's static device array."""
    return load_library().ftd_decode_mha_noalloc(ctypes.byref(cfg), *_ptrs(q, k_new, v_new, qkv_bias, k_cache,
                                                                           v_cache, seq_lens, scales, out,
                                                                           device_err, stream))


def ftd_debug_stall_next(ctx, calls: int) -> int:
    """Test hook: the next ``calls`` decode calls withhold one tile copy (bounded-wait error path)."""
    return load_library().ftd_debug_stall_next(ctypes.c_void_p(ctx), int(calls))


def ftd_debug_late_lengths(src, dst, n: int, delay_us: int, stream) -> int:
    """Test hook: a kernel that lets the next launch start at once and copies n lengths src -> dst late."""
    return load_library().ftd_debug_late_lengths(src, dst, int(n), int(delay_us), stream)


def ftd_debug_kernel(ctx, entry: int):
    """Test hook: (status, query rows of a block, on the tensor cores) for entry 0 the step, 1 scored, 2 cross."""
    rows, tc = ctypes.c_int(), ctypes.c_int()
    st = load_library().ftd_debug_kernel(ctypes.c_void_p(ctx or None), int(entry), ctypes.byref(rows), ctypes.byref(tc))
    return st, rows.value, bool(tc.value)


def ftd_get_error(ctx) -> int:
    return load_library().ftd_get_error(ctypes.c_void_p(ctx))


def ftd_destroy(ctx) -> None:
    load_library().ftd_destroy(ctypes.c_void_p(ctx or None))


def check(status: int) -> None:
    if status != FTD_OK:
        raise FtdError(status, ftd_last_error())


# ------------------------------------------------------- torch convenience
def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


_raw_stream = None


def _current_stream(device: int) -> int:
    """torch's current stream on a device, as an address (without a Stream object where torch has a way)."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    return _raw_stream(device)


def _expect(name, t, n, dtype=None, itemsize=0, dense=True, tail=()):
    """Raise where t does not begin with n elements of dtype (or of itemsize bytes), one after the other.  It may hold
    more, as a buffer kept for larger calls does, if its last dimensions are tail's."""
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements, {n} are needed")
    if (dtype is not None and t.dtype is not dtype) or (itemsize and t.element_size() != itemsize):
        raise ValueError(f"{name} is {t.dtype}, it has to be {dtype or f'a type of {itemsize} bytes'}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} has to be contiguous")
    if t.numel() > n and t.dim() > 1 and any(a != b for a, b in zip(reversed(t.shape), reversed(tail))):
        raise ValueError(f"{name} is laid out as {tuple(t.shape)}, its last dimensions have to be {tuple(tail)}")


def _row_stride(t, width: int, head_dim: int) -> int:
    """Elements from one token's row of ``width`` elements (heads flattened, or [heads, head_dim]) to the next; 0: dense."""
    if t.is_contiguous():
        return 0
    if t.dim() == 2 and t.shape[1] == width and t.stride(1) == 1:
        return t.stride(0)
    split = t.shape[-1] != width
    lead = t.dim() - (2 if split else 1)
    ok = lead >= 1 and t.stride(-1) == 1 and (not split or (t.shape[-1] == head_dim and t.stride(-2) == head_dim
                                                            and t.shape[-2] * head_dim == width))
    row, n = 0, 1  # the innermost token dimension's stride, and the tokens within the dimensions seen
    for i in reversed(range(lead if ok else 0)):
        if t.shape[i] == 1:
            continue
        row = row or t.stride(i)
        ok = ok and t.stride(i) == row * n
        n *= t.shape[i]
    if not ok:
        raise ValueError("rows of heads must be dense and a fixed number of elements apart")
    return row


class DecodeStep:
    """Owns one library context; calls take torch CUDA tensors (marshalling only)."""

    def __init__(self, max_batch, n_q_heads, n_kv_heads, head_dim, max_len, qkv_dtype="bf16",
                 cache_dtype="bf16", softmax_scale=0.0, stream: Optional[int] = None, out_dtype="f32",
                 window=0, page_size=0, num_pages=0, q_len=1, kernel=FTD_KERNEL_AUTO, wait_limit_us=0, proj_dim=0,
                 scored=False):
        import torch
        self.cfg = FtdConfig(max_batch, n_q_heads, n_kv_heads, head_dim, max_len, DTYPES[qkv_dtype],
                             DTYPES[cache_dtype], float(softmax_scale), DTYPES[out_dtype], int(window),
                             int(page_size), int(num_pages), int(q_len), int(kernel), int(proj_dim),
                             int(wait_limit_us))
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream
        st, ctx = ftd_init(self.cfg, s)
        check(st)
        self.ctx = ctx
        self.device = torch.cuda.current_device()
        self._widths = (n_q_heads * head_dim, n_kv_heads * head_dim, head_dim)
        self._qkv_bytes = 4 if qkv_dtype == "f32" else 2
        self._cache_bytes = {"f32": 4, "f16": 2, "bf16": 2, "i8": 1}[cache_dtype]
        self._out_bytes = 4 if out_dtype == "f32" else 2
        self._int32 = torch.int32
        self._axes = 0
        self._float32 = torch.float32
        # cache rows: elements of a plane
        self._rows = num_pages * n_kv_heads * page_size if page_size else max_batch * n_kv_heads * max_len
        self._plane_tail = (n_kv_heads, page_size or max_len)
        self._scales_tail = (num_pages if page_size else max_batch,) + self._plane_tail  # (V's plane lies right behind K's)
        n, eb, cb = max_batch * max(int(q_len), 1), self._qkv_bytes, self._cache_bytes
        # bytes of a step's q, new rows, output and caches, and of an element of each
        self._step_bytes = (n * n_q_heads * head_dim * eb, n * n_kv_heads * head_dim * eb, n * n_q_heads * head_dim * self._out_bytes,
                            self._rows * head_dim * cb, eb, self._out_bytes, cb)
        self._entries = max_batch * -(-max_len // page_size) if page_size else 0  # of a block table
        if scored:
            self.enable_scores(s)

    def cache_ptrs(self):
        st, k, v, s = ftd_cache_ptrs(self.ctx)
        check(st)
        return k, v, s

    def __call__(self, q, k_new, v_new, seq_lens, out, bias=None, k_cache=None, v_cache=None, scales=None,
                 stream: Optional[int] = None):
        import torch
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream
        if self.cfg.page_size:
            raise ValueError("a paged context takes paged(..., block_table, ...)")
        check(ftd_decode_mha(self.ctx, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(bias), _ptr(k_cache),
                             _ptr(v_cache), _ptr(seq_lens), _ptr(scales), _ptr(out), s))

    def proj(self, q, k_new, v_new, seq_lens, out, w_o, y, bias=None, k_cache=None, v_cache=None, scales=None,
             stream: Optional[int] = None):
        """The step followed by the output projection y = out . w_o^T (a context with proj_dim)."""
        import torch
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream
        check(ftd_decode_mha_proj(self.ctx, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(bias), _ptr(k_cache),
                                  _ptr(v_cache), _ptr(seq_lens), _ptr(scales), _ptr(out), _ptr(w_o), _ptr(y), s))

    def paged(self, q, k_new, v_new, block_table, seq_lens, out, bias=None, k_pages=None, v_pages=None,
              scales=None, stream: Optional[int] = None):
        import torch
        s = torch.cuda.current_stream().cuda_stream if stream is None else stream
        check(ftd_decode_mha_paged(self.ctx, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(bias), _ptr(k_pages),
                                   _ptr(v_pages), _ptr(block_table), _ptr(seq_lens), _ptr(scales), _ptr(out),
                                   s))

    def _check_planes(self, lens=(), ints=(), floats=(), table=None):
        """Raise where a length, a plane or the block table (None: absent) has another type or layout than the kernels
        take: int32 per slot, int32 and fp32 per cache row."""
        i32, f32, nb, nr = self._int32, self._float32, 4 * self.cfg.max_batch, 4 * self._rows
        for t in lens:
            if t is not None and (t.dtype is not i32 or t.nbytes != nb or not t.is_contiguous()):
                _expect("a list of lengths or next_pos", t, nb // 4, dtype=i32)
        for t in ints:
            if t is not None and (t.dtype is not i32 or t.nbytes != nr or not t.is_contiguous()):
                _expect("a positions plane", t, nr // 4, dtype=i32, tail=self._plane_tail)
        for t in floats:
            if t is not None and (t.dtype is not f32 or t.nbytes != nr or not t.is_contiguous()):
                _expect("a weights plane", t, nr // 4, dtype=f32, tail=self._plane_tail)
        if table is not None and self._entries and (table.dtype is not i32 or table.nbytes != 4 * self._entries
                                                    or not table.is_contiguous()):
            _expect("the block table", table, self._entries, dtype=i32, tail=(self._entries // self.cfg.max_batch,))

    def enable_scores(self, stream: Optional[int] = None):
        """Allocate what ``scored`` and ``evict`` need (``scored=True`` does it at construction)."""
        check(ftd_enable_scores(self.ctx, _current_stream(self.device) if stream is None else stream))

    def scored(self, q, k_new, v_new, seq_lens, next_pos, acc, positions, out, acc_out=None, bias=None, k_cache=None,
               v_cache=None, scales=None, block_table=None, stream: Optional[int] = None):
        """The step, which also adds every position's attention weight to ``acc`` (into ``acc_out`` when
        given); the new rows of ``positions`` (may be None, with next_pos) become next_pos, next_pos + 1, ..."""
        self._check_planes((seq_lens, next_pos), (positions,), (acc, acc_out), block_table)
        s = _current_stream(self.device) if stream is None else stream
        st = ftd_decode_mha_scored(self.ctx, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), _ptr(bias), _ptr(k_cache),
                                   _ptr(v_cache), _ptr(block_table), seq_lens.data_ptr(), _ptr(scales), _ptr(next_pos),
                                   acc.data_ptr(), _ptr(acc_out), _ptr(positions), out.data_ptr(), s)
        if st:
            check(st)

    def evict(self, acc, positions, seq_lens, next_pos, new_lens, budget, recent=0, sinks=0, acc_out=None,
              positions_out=None, k_cache=None, v_cache=None, scales=None, block_table=None,
              stream: Optional[int] = None):
        """Bring every slot down to ``budget`` rows per kv head by accumulated weight (``new_lens`` may be
        ``seq_lens``; planes change in place unless ``acc_out`` / ``positions_out`` are given)."""
        self._check_planes((seq_lens, next_pos, new_lens), (positions, positions_out), (acc, acc_out), block_table)
        s = _current_stream(self.device) if stream is None else stream
        st = ftd_cache_evict(self.ctx, _ptr(k_cache), _ptr(v_cache), _ptr(scales), _ptr(block_table),
                             seq_lens.data_ptr(), next_pos.data_ptr(), acc.data_ptr(), _ptr(acc_out),
                             positions.data_ptr(), _ptr(positions_out), new_lens.data_ptr(), int(budget), int(recent),
                             int(sinks), s)
        if st:
            check(st)

    def cross(self, q, mem_lens, out, q_bias=None, k_mem=None, v_mem=None, scales=None,
              stream: Optional[int] = None):
        """Cross attention of the slots' tokens to memories of ``mem_lens`` rows (None: the context's pool)."""
        self._check_planes((mem_lens,))
        s = _current_stream(self.device) if stream is None else stream
        st = ftd_cross_mha(self.ctx, q.data_ptr(), _ptr(q_bias), _ptr(k_mem), _ptr(v_mem), mem_lens.data_ptr(),
                           _ptr(scales), out.data_ptr(), s)
        if st:
            check(st)

    def set_rope(self, n_axes=1, sections=None, rotary_dim=0, theta=0.0, pairing="halves", order="sections",
                 inv_freq=None):
        """The rotary positions of ``rope``: sections holds the pairs of each axis, inv_freq (host floats)
        replaces theta^(-2i/R)."""
        cfg = FtdRopeConfig(n_axes=int(n_axes), rotary_dim=int(rotary_dim), theta=float(theta))
        sections = list(sections) if sections is not None else []
        if len(sections) > 4:
            raise ValueError("at most four axes")
        for a, n in enumerate(sections):
            cfg.section[a] = int(n)
        cfg.pairing = {"halves": FTD_ROPE_HALVES, "adjacent": FTD_ROPE_ADJACENT}[pairing]
        cfg.order = {"sections": FTD_ROPE_SECTIONS, "interleaved": FTD_ROPE_INTERLEAVED}[order]
        if inv_freq is not None:
            f = [float(x) for x in inv_freq]
            if len(f) != (int(rotary_dim) or self.cfg.head_dim) // 2:
                raise ValueError("inv_freq holds one value per pair")
            cfg.inv_freq = (ctypes.c_double * len(f))(*f)
        check(ftd_set_rope(self.ctx, cfg))
        self._axes = int(n_axes)

    def _check_rope(self, n, q, k, v, positions, q_out, k_out, v_out, bias):
        """Raise for what the pointers of a rope call cannot show."""
        qw, kw, d = self._widths
        eb = self._qkv_bytes
        if q.numel() != n * qw:
            raise ValueError(f"q holds {q.numel()} elements, no whole number of rows of {qw}")
        for name, t, width in (("q", q, qw), ("k", k, kw), ("v", v, kw)):
            if t is not None:
                _expect(name, t, n * width, itemsize=eb, dense=False)  # (_row_stride looks at the strides)
        for name, t, width in (("q_out", q_out, qw), ("k_out", k_out, kw), ("v_out", v_out, kw)):
            if t is not None:
                _expect(name, t, n * width, itemsize=eb, tail=(width,) if t.shape[-1] == width else (width // d, d))
        if bias is not None:
            _expect("bias", bias, qw + 2 * kw, itemsize=eb)
        if self._axes:  # (else the library says that set_rope comes first)
            _expect("positions", positions, n * self._axes, dtype=self._int32)
            if self._axes > 1 and positions.numel() > n * self._axes and positions.dim() > 1 and (
                    positions.numel() // positions.shape[0] != n):
                raise ValueError(f"positions is laid out as {tuple(positions.shape)}, an axis has {n} tokens")

    def rope(self, q, k, v, positions, q_out, k_out, v_out=None, bias=None, stream: Optional[int] = None):
        """Bias and rotary positions for the tokens of q, k (and v, which only takes the bias; None with
        v_out None): rows of heads a fixed stride apart, such as slices of a fused projection.  positions is
        int32 [n_axes, tokens]; the outputs are dense and may be their own dense inputs."""
        qw, kw, d = self._widths
        eb = self._qkv_bytes
        n = q.numel() // qw
        bq, bk = n * qw * eb, n * kw * eb
        # every size and type in one expression (a call for few tokens is bound by the host); _check_rope says
        # which it is
        if (q.nbytes != bq or k.nbytes != bk or q_out.nbytes != bq or k_out.nbytes != bk
                or positions.nbytes != 4 * n * self._axes or positions.dtype is not self._int32
                or not positions.is_contiguous() or not q_out.is_contiguous() or not k_out.is_contiguous()
                or (v is not None or v_out is not None)
                and (v is None or v_out is None or v.nbytes != bk or v_out.nbytes != bk or not v_out.is_contiguous())
                or bias is not None and (bias.nbytes != (qw + 2 * kw) * eb or not bias.is_contiguous())):
            self._check_rope(n, q, k, v, positions, q_out, k_out, v_out, bias)
        s = _current_stream(self.device) if stream is None else stream
        qs = 0 if q.is_contiguous() else _row_stride(q, qw, d)
        ks = 0 if k.is_contiguous() else _row_stride(k, kw, d)
        if v is not None and ((0 if v.is_contiguous() else _row_stride(v, kw, d)) or kw) != (ks or kw) and n > 1:
            raise ValueError("k and v must share one row stride")
        st = ftd_rope_qkv(self.ctx, q.data_ptr(), k.data_ptr(), None if v is None else v.data_ptr(), qs, ks,
                          None if bias is None else bias.data_ptr(), positions.data_ptr(), n, q_out.data_ptr(),
                          k_out.data_ptr(), None if v_out is None else v_out.data_ptr(), s)
        if st:
            check(st)

    def _check_norm_rope(self, n, q_weight, k_weight, slots, k_cache, v_cache, scales):
        """Raise for what the pointers of the norms and of a fill cannot show."""
        d, eb = self._widths[2], self._qkv_bytes
        for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
            if t is not None:
                _expect(name, t, d, itemsize=eb)
        if slots is not None:
            _expect("slots", slots, n, dtype=self._int32)
            for name, t in (("k_cache", k_cache), ("v_cache", v_cache)):
                if t is not None:
                    _expect(name, t, self._rows * d, itemsize=self._cache_bytes, tail=self._plane_tail + (d,))
            if scales is not None:
                _expect("scales", scales, 2 * self._rows, dtype=self._float32, tail=self._scales_tail)

    def norm_rope(self, q, k, v, positions, q_out, k_out=None, v_out=None, bias=None, q_weight=None, k_weight=None, eps=1e-6,
                  weight_offset=0.0, slots=None, k_cache=None, v_cache=None, scales=None, stream: Optional[int] = None):
        """``rope`` with norms of the query and key heads ahead of the rotation: x / sqrt(mean(x^2) + eps) *
        (weight + weight_offset), weights of head_dim elements (None: no norm).  With ``slots`` (int32 per
        token, as ``tables`` makes them; negative: none) keys and values go straight into the cache (None: the
        pool's), rounded or quantised as the step appends them, and k_out and v_out stay None."""
        qw, kw, d = self._widths
        eb = self._qkv_bytes
        n = q.numel() // qw
        bq, bk = n * qw * eb, n * kw * eb
        if (q.nbytes != bq or k.nbytes != bk or q_out.nbytes != bq or positions.nbytes != 4 * n * self._axes
                or positions.dtype is not self._int32 or not positions.is_contiguous() or not q_out.is_contiguous()
                or bias is not None and (bias.nbytes != (qw + 2 * kw) * eb or not bias.is_contiguous())
                or k_out is not None and (k_out.nbytes != bk or not k_out.is_contiguous())
                or v is not None and v.nbytes != bk or v_out is not None and (v_out.nbytes != bk or not v_out.is_contiguous())):
            self._check_rope(n, q, k, v, positions, q_out, k_out, v_out, bias)
        if (q_weight is not None and (q_weight.nbytes != d * eb or not q_weight.is_contiguous())
                or k_weight is not None and (k_weight.nbytes != d * eb or not k_weight.is_contiguous()) or slots is not None):
            self._check_norm_rope(n, q_weight, k_weight, slots, k_cache, v_cache, scales)
        s = _current_stream(self.device) if stream is None else stream
        qs = 0 if q.is_contiguous() else _row_stride(q, qw, d)
        ks = 0 if k.is_contiguous() else _row_stride(k, kw, d)
        if v is not None and ((0 if v.is_contiguous() else _row_stride(v, kw, d)) or kw) != (ks or kw) and n > 1:
            raise ValueError("k and v must share one row stride")
        st = ftd_norm_rope_qkv(self.ctx, q.data_ptr(), k.data_ptr(), _ptr(v), qs, ks, _ptr(bias), _ptr(q_weight),
                               _ptr(k_weight), eps, weight_offset, positions.data_ptr(), n, q_out.data_ptr(), _ptr(k_out),
                               _ptr(v_out), _ptr(slots), _ptr(k_cache), _ptr(v_cache), _ptr(scales), s)
        if st:
            check(st)

    def tables(self, old_lens, new_lens, served, block_table=None, free_pages=None, n_free=None, n_free_out=None, offsets=None,
               slots=None, positions=None, stream: Optional[int] = None):
        """Bring every slot from old_lens to new_lens cached rows: pages from and to the free list (a stack of
        n_free pages; paged contexts), ``served`` the lengths that were granted (may be either list), ``offsets``
        int32 [B + 1] of the new tokens packed slot by slot, and their ``slots`` and ``positions`` (int32, one length)."""
        self._check_planes((old_lens, new_lens, served), table=block_table)
        if free_pages is not None:
            _expect("free_pages", free_pages, self.cfg.num_pages, dtype=self._int32)
        for name, t, n in (("n_free", n_free, 1), ("n_free_out", n_free_out, 1), ("offsets", offsets, self.cfg.max_batch + 1),
                           ("slots", slots, 0), ("positions", positions, 0)):
            if t is not None:
                _expect(name, t, n, dtype=self._int32, tail=t.shape)
        if slots is not None and positions is not None and slots.numel() != positions.numel():
            raise ValueError(f"slots holds {slots.numel()} tokens, positions {positions.numel()}")
        n = slots.numel() if slots is not None else positions.numel() if positions is not None else 0
        s = _current_stream(self.device) if stream is None else stream
        st = ftd_build_tables(self.ctx, old_lens.data_ptr(), new_lens.data_ptr(), served.data_ptr(), _ptr(block_table),
                              _ptr(free_pages), _ptr(n_free), _ptr(n_free_out), _ptr(offsets), _ptr(slots), _ptr(positions),
                              n, s)
        if st:
            check(st)

    def enable_prefix(self, stream: Optional[int] = None):
        """Allocate what ``prefix`` needs."""
        check(ftd_enable_prefix(self.ctx, _current_stream(self.device) if stream is None else stream))

    def _check_step(self, q, k_new, v_new, out, bias, k_cache, v_cache, scales):
        """Raise where a tensor of a step holds too little, or another type or layout than the kernels take."""
        qw, kw, d = self._widths
        n, eb, cb = self.cfg.max_batch * max(self.cfg.q_len, 1), self._qkv_bytes, self._cache_bytes
        for name, t, size, eb, tail in (("q", q, n * qw, eb, None), ("k_new", k_new, n * kw, eb, None), ("v_new", v_new, n * kw, eb, None),
                                        ("out", out, n * qw, self._out_bytes, None), ("bias", bias, qw + 2 * kw, eb, None),
                                        ("k_cache", k_cache, self._rows * d, cb, self._plane_tail + (d,)),
                                        ("v_cache", v_cache, self._rows * d, cb, self._plane_tail + (d,)),
                                        ("scales", scales, 2 * self._rows, 4, self._scales_tail)):
            if t is not None and (t.nbytes != size * eb or t.itemsize != eb or not t.is_contiguous()):
                _expect(name, t, size, itemsize=eb, tail=t.shape if tail is None else tail)

    def _prefix_rows(self, k_prefix, v_prefix, prefix_scales, prefix_table):
        """Rows of the prefix by its tensors, which have to agree."""
        d, hkv = self._widths[2], self.cfg.n_kv_heads
        if self.cfg.page_size:
            if prefix_table is None:
                return 0
            _expect("prefix_table", prefix_table, 0, dtype=self._int32, tail=prefix_table.shape)
            return prefix_table.numel() * self.cfg.page_size
        if k_prefix is None or v_prefix is None:
            if k_prefix is not v_prefix:
                raise ValueError("k_prefix and v_prefix come together")
            return 0
        rows = k_prefix.numel() // (hkv * d)
        for name, t in (("k_prefix", k_prefix), ("v_prefix", v_prefix)):
            if t.numel() != rows * hkv * d or t.element_size() != self._cache_bytes or not t.is_contiguous() or (
                    t.dim() > 1 and (t.shape[-1] != d or t.dim() > 2 and t.shape[-2] != rows)):
                raise ValueError(f"{name} has to be a contiguous [{hkv}, rows, {d}] of the cache type, one shape for both")
        if prefix_scales is not None:
            _expect("prefix_scales", prefix_scales, 2 * hkv * rows, dtype=self._float32, tail=(hkv, rows))
        return rows

    def prefix(self, q, k_new, v_new, seq_lens, prefix_lens, out, k_prefix=None, v_prefix=None, prefix_scales=None,
               prefix_table=None, bias=None, k_cache=None, v_cache=None, scales=None, block_table=None,
               stream: Optional[int] = None):
        """The step of slots that share a prefix: slot b sees its first prefix_lens[b] rows and its own.  The prefix
        is [n_kv_heads, rows, head_dim] (INT8: and scales [2, n_kv_heads, rows]), or the pool's pages that
        ``prefix_table`` names.  After ``enable_prefix``."""
        self._check_planes((seq_lens, prefix_lens), table=block_table)
        bq, bk, bo, bc, eb, ob, cb = self._step_bytes
        if (q.nbytes != bq or q.itemsize != eb or not q.is_contiguous() or k_new.nbytes != bk or k_new.itemsize != eb
                or not k_new.is_contiguous() or v_new.nbytes != bk or v_new.itemsize != eb or not v_new.is_contiguous()
                or out.nbytes != bo or out.itemsize != ob or not out.is_contiguous()
                or k_cache is not None and (k_cache.nbytes != bc or k_cache.itemsize != cb or not k_cache.is_contiguous())
                or v_cache is not None and (v_cache.nbytes != bc or v_cache.itemsize != cb or not v_cache.is_contiguous())
                or bias is not None or scales is not None):
            self._check_step(q, k_new, v_new, out, bias, k_cache, v_cache, scales)
        rows = self._prefix_rows(k_prefix, v_prefix, prefix_scales, prefix_table)
        s = _current_stream(self.device) if stream is None else stream
        st = ftd_decode_mha_prefix(self.ctx, q.data_ptr(), k_new.data_ptr(), v_new.data_ptr(), _ptr(bias), _ptr(k_cache),
                                   _ptr(v_cache), _ptr(block_table), seq_lens.data_ptr(), _ptr(scales), _ptr(k_prefix),
                                   _ptr(v_prefix), _ptr(prefix_scales), _ptr(prefix_table), rows, prefix_lens.data_ptr(),
                                   out.data_ptr(), s)
        if st:
            check(st)

    def get_error(self) -> int:
        return ftd_get_error(self.ctx)

    def close(self):
        if getattr(self, "ctx", None):
            ftd_destroy(self.ctx)
            self.ctx = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
