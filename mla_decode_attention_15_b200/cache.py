"""Python binding of include/mla_cache.h (ctypes): rotary positions, the write of
new rows into the paged latent cache, decode attention over the cache in 8 bits,
and the fork, free, copy and compaction of pages.

Argument marshalling only, like ``binding``: every step runs in the CUDA kernels
of libmla_decode.so, and there is no fallback.
"""
from __future__ import annotations

import ctypes
import functools
import math
from typing import Optional, Tuple

import torch

from . import binding as bd
from .binding import MlaDecodeError, _check, _ptr, _require, _stream, mla_decode_dims

MLA_CACHE_BF16 = 0
MLA_CACHE_E4M3 = 1
MLA_DTYPE_BF16 = 0
MLA_DTYPE_FP32 = 1
MLA_ROPE_NONE = 0
MLA_ROPE_LINEAR = 1
MLA_ROPE_YARN = 2

MLA_STATUS_BAD_ROW = 0x20
MLA_STATUS_NO_FREE_PAGE = 0x40
MLA_STATUS_BAD_REF_COUNT = 0x80

FORK_MAX = 1024

CACHE_EXPORTED = (
    "mla_rope_init",
    "mla_rope_apply",
    "mla_cache_append",
    "mla_cache_fork_workspace_bytes",
    "mla_cache_fork",
    "mla_cache_free",
    "mla_cache_copy_pages",
    "mla_cache_compact_workspace_bytes",
    "mla_cache_compact",
    "mla_cache_version",
    "mla_decode_q8_schedule_bytes",
    "mla_decode_q8_workspace_bytes",
    "mla_decode_q8_get_schedule",
    "mla_decode_q8_get_schedule_host",
    "mla_decode_q8_fwd",
    "mla_decode_q8_combine",
)


class mla_rope_config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("theta", "factor", "beta_fast", "beta_slow", "amplitude")] + \
               [(n, ctypes.c_int32) for n in ("original_max_position", "scaling", "interleaved", "reserved")]


class mla_rope_table(ctypes.Structure):
    _fields_ = [("turns", ctypes.c_double * 32), ("amplitude", ctypes.c_float), ("interleaved", ctypes.c_int32)]


class mla_rope_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tokens", "num_heads", "width", "offset")] + \
               [(n, ctypes.c_int64) for n in ("x_token_stride", "x_head_stride", "out_token_stride", "out_head_stride")] + \
               [(n, ctypes.c_int32) for n in ("dtype", "transpose")]


class mla_cache_dims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "batch", "max_blocks_per_seq", "num_blocks", "page_size", "row_width", "dtype")]


_lib = None


def lib() -> ctypes.CDLL:
    """libmla_decode.so with the signatures of mla_cache.h set."""
    global _lib
    if _lib is None:
        L = bd.lib()
        vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        P, C = ctypes.POINTER(mla_decode_dims), ctypes.POINTER(mla_cache_dims)
        size, rc = ctypes.c_size_t, ctypes.c_int
        for name, res, args in (
                ("mla_rope_init", rc, [ctypes.POINTER(mla_rope_config), ctypes.POINTER(mla_rope_table)]),
                ("mla_rope_apply", rc, [ctypes.POINTER(mla_rope_dims), ctypes.POINTER(mla_rope_table), vp, vp, vp, vp]),
                ("mla_cache_append", rc, [C, i32, vp, i64, vp, i64, vp, ctypes.POINTER(mla_rope_table), vp, vp, vp, vp, vp, vp]),
                ("mla_cache_fork_workspace_bytes", size, [i32]),
                ("mla_cache_fork", rc, [C, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]),
                ("mla_cache_free", rc, [C, i32, vp, vp, vp, vp, vp, vp]),
                ("mla_cache_copy_pages", rc, [C, i32, vp, vp, vp, vp, vp, vp]),
                ("mla_cache_compact_workspace_bytes", size, [C]),
                ("mla_cache_compact", rc, [C, vp, vp, vp, vp, vp, vp, vp, vp]),
                ("mla_cache_version", rc, []),
                ("mla_decode_q8_schedule_bytes", size, [P]),
                ("mla_decode_q8_workspace_bytes", size, [P]),
                ("mla_decode_q8_get_schedule", rc, [P, vp, vp, vp]),
                ("mla_decode_q8_get_schedule_host", rc, [P, vp, vp]),
                ("mla_decode_q8_fwd", rc, [P, vp, vp, vp, vp, vp, vp, vp, ctypes.c_float, vp, vp, vp]),
                ("mla_decode_q8_combine", rc, [P, vp, vp, vp, vp, vp])):
            f = getattr(L, name)
            f.restype, f.argtypes = res, args
        _lib = L
    return _lib


def mla_cache_version() -> int:
    return int(lib().mla_cache_version())


# Small calls are bound by the host, so the checks below build no text and no tuples
# unless they fail, and structures that only hold sizes are made once per size.
_BF16, _F32, _E4M3, _I32 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _fail(msg: str, *args) -> None:
    raise ValueError(msg % args if args else msg)


def _i32(t: torch.Tensor, shape, what: str, device) -> None:
    if t.dtype is not _I32 or t.shape != shape or not t.is_contiguous():
        _fail("%s must be contiguous int32 %s", what, list(shape))
    if t.device != device:
        _fail("%s must be on %s", what, device)


def _launch_stream(device: torch.device, stream) -> int:
    """The stream's handle.  The library launches on the current device, so the
    tensors and the stream must be of that device."""
    if device.type != "cuda":
        _fail("tensors must be on a CUDA device")
    if device.index != torch.cuda.current_device():
        _fail("tensors must be on the current CUDA device")
    if stream is None:
        return _raw_stream(device.index) if _raw_stream is not None else torch.cuda.current_stream(device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        if stream.device != device:
            _fail("stream must be of the current CUDA device")
        return stream.cuda_stream
    return int(stream)


def _empty(shape, dtype, device, stream, what: str) -> torch.Tensor:
    """Memory for a launch on ``stream``, from that stream's pool: the current
    stream's may still be in use by work that is queued there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        _fail("a raw stream handle needs %s of the caller's", what)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _status(status: Optional[torch.Tensor], device) -> Optional[int]:
    if status is None:
        return None
    if status.dtype is not _I32 or status.numel() < 1 or not status.is_contiguous() or status.device != device:
        _fail("status must be int32 on %s", device)
    return status.data_ptr()


@functools.lru_cache(maxsize=1024)
def _cache_dims(batch: int, max_blocks: int, num_blocks: int, dtype: int):
    return ctypes.byref(mla_cache_dims(batch, max_blocks, num_blocks, bd.PAGE_SIZE, bd.D_QK, dtype))


@functools.lru_cache(maxsize=1024)
def _rope_dims(*sizes):
    return ctypes.byref(mla_rope_dims(*sizes))


# ---------------------------------------------------------------- rotary positions
def make_rope(theta: float = 10000.0, interleaved: bool = True, scaling: str = "none", factor: float = 1.0,
              original_max_position: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
              amplitude: float = 1.0) -> mla_rope_table:
    """Rotary table of the 64 RoPE columns (mla_rope_init): angular frequencies
    theta^(-2i/64), divided by ``factor`` (scaling "linear"), or blended
    between both by wavelength ("yarn"); ``amplitude`` multiplies the rotated
    values.  Host memory; keep it for as long as the model lives."""
    kinds = {"none": MLA_ROPE_NONE, "linear": MLA_ROPE_LINEAR, "yarn": MLA_ROPE_YARN}
    _require(scaling in kinds, "scaling must be one of %s" % sorted(kinds))
    cfg = mla_rope_config(float(theta), float(factor), float(beta_fast), float(beta_slow), float(amplitude),
                          int(original_max_position), kinds[scaling], int(bool(interleaved)), 0)
    table = mla_rope_table()
    _check(lib().mla_rope_init(ctypes.byref(cfg), ctypes.byref(table)), "mla_rope_init")
    return table


def rope_apply(x: torch.Tensor, positions: torch.Tensor, rope: mla_rope_table, offset: int = 0,
               out: Optional[torch.Tensor] = None, transpose: bool = False, stream=None) -> torch.Tensor:
    """x [T, h, W] (or [T, W]) bf16 or fp32 with its columns [offset, offset + 64)
    rotated for positions [T] (int32); the other columns pass through.  Rows
    may be strided (multiples of 8 values); ``out=x`` rotates in place.
    ``transpose`` applies the transposed map: the gradient of x from that of
    the result.  Without ``out`` the result belongs to ``stream`` (a torch.cuda.Stream)."""
    shape, dtype, device = x.shape, x.dtype, x.device
    if len(shape) not in (2, 3):
        _fail("x must be [T, h, W] or [T, W]")
    if dtype is not _BF16 and dtype is not _F32:
        _fail("x must be bf16 or fp32")
    if out is None:
        out = _empty(shape, dtype, device, stream, "out")
    elif out.shape != shape or out.dtype is not dtype or out.device != device:
        _fail("out must have the shape, type and device of x")
    T, W = shape[0], shape[-1]
    h = shape[1] if len(shape) == 3 else 1
    _i32(positions, (T,), "positions", device)
    if T == 0 or h == 0:
        return out
    xs, os_ = x.stride(), out.stride()
    if xs[-1] != 1 or os_[-1] != 1:
        _fail("the columns of x and out must be contiguous")
    stream = _launch_stream(device, stream)
    # (a dimension of one row has no stride of its own)
    xh, oh = (xs[1], os_[1]) if h > 1 else (W, W)
    d = _rope_dims(T, h, W, int(offset), xs[0] if T > 1 else h * xh, xh, os_[0] if T > 1 else h * oh, oh,
                   MLA_DTYPE_BF16 if dtype is _BF16 else MLA_DTYPE_FP32, int(bool(transpose)))
    rc = lib().mla_rope_apply(d, ctypes.byref(rope), x.data_ptr(), positions.data_ptr(), out.data_ptr(), stream)
    if rc:
        _check(rc, "mla_rope_apply")
    return out


# ---------------------------------------------------------------- the cache
def _pool_dims(kv_cache: torch.Tensor, kv_scales: Optional[torch.Tensor], batch: int, max_blocks: int):
    """The dims of a pool and its table, and the scales' address."""
    shape, q8 = kv_cache.shape, kv_cache.dtype is _E4M3
    nb = shape[0]
    if not (q8 or kv_cache.dtype is _BF16) or shape != (nb, bd.PAGE_SIZE, 1, bd.D_QK) or not kv_cache.is_contiguous():
        _fail("kv_cache must be contiguous bf16 or float8_e4m3fn [num_blocks, 64, 1, 576]")
    if not q8:
        if kv_scales is not None:
            _fail("a bf16 cache has no scales")
        return _cache_dims(batch, max_blocks, nb, MLA_CACHE_BF16), None
    if kv_scales is None or kv_scales.dtype is not _F32 or kv_scales.shape != (nb, 1) or not kv_scales.is_contiguous() or \
            kv_scales.device != kv_cache.device:
        _fail("kv_scales must be contiguous fp32 [num_blocks, 1] beside an 8-bit cache")
    return _cache_dims(batch, max_blocks, nb, MLA_CACHE_E4M3), kv_scales.data_ptr()


def _books(block_table, cache_seqlens, ref_counts, nb, device) -> Tuple[int, int]:
    shape = block_table.shape
    if len(shape) != 2:
        _fail("block_table must be int32 [B, max_blocks_per_seq]")
    _i32(block_table, shape, "block_table", device)
    _i32(cache_seqlens, shape[:1], "cache_seqlens", device)
    if ref_counts is not None:
        _i32(ref_counts, (nb,), "ref_counts", device)
    return shape[0], shape[1]


def cache_append(c_kv: torch.Tensor, k_pe: torch.Tensor, new_offsets: torch.Tensor, block_table: torch.Tensor,
                 cache_seqlens: torch.Tensor, kv_cache: torch.Tensor, kv_scales: Optional[torch.Tensor] = None,
                 rope: Optional[mla_rope_table] = None, status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Writes new rows into the cache (mla_cache_append).  c_kv [T, 512] and
    k_pe [T, 64] bf16 (their rows may be strided, as the two parts of one
    projection are), new_offsets [B + 1] int32: rows new_offsets[b] ..
    new_offsets[b + 1] are the last positions of request b, whose
    cache_seqlens counts them already.  With ``rope`` the keys are rotated for
    their positions.  An 8-bit cache's page scales follow its rows."""
    device = kv_cache.device
    T = c_kv.shape[0]
    B, width = _books(block_table, cache_seqlens, None, 0, device)
    d, scales = _pool_dims(kv_cache, kv_scales, B, width)
    cs, ps = c_kv.stride(), k_pe.stride()
    if c_kv.dtype is not _BF16 or c_kv.shape != (T, bd.D_V) or (cs[1] != 1 and T) or c_kv.device != device:
        _fail("c_kv must be bf16 [T, 512] on %s", device)
    if k_pe.dtype is not _BF16 or k_pe.shape != (T, bd.D_QK - bd.D_V) or (ps[1] != 1 and T) or k_pe.device != device:
        _fail("k_pe must be bf16 [T, 64] on %s, as many rows as c_kv", device)
    _i32(new_offsets, (B + 1,), "new_offsets", device)
    status = _status(status, device)
    if T == 0:
        return
    stream = _launch_stream(device, stream)
    rc = lib().mla_cache_append(d, T, c_kv.data_ptr(), cs[0] if T > 1 else bd.D_V, k_pe.data_ptr(),
                                ps[0] if T > 1 else bd.D_QK - bd.D_V, new_offsets.data_ptr(),
                                None if rope is None else ctypes.byref(rope), block_table.data_ptr(),
                                cache_seqlens.data_ptr(), kv_cache.data_ptr(), scales, status, stream)
    if rc:
        _check(rc, "mla_cache_append")


def cache_fork(parents: torch.Tensor, children: torch.Tensor, block_table: torch.Tensor, cache_seqlens: torch.Tensor,
               ref_counts: torch.Tensor, kv_cache: torch.Tensor, kv_scales: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Makes the empty rows ``children`` copies of ``parents`` (mla_cache_fork): full
    pages are shared and counted, a last page that is not full is copied
    into the lowest free page."""
    device, n = kv_cache.device, parents.numel()
    B, width = _books(block_table, cache_seqlens, ref_counts, kv_cache.shape[0], device)
    d, scales = _pool_dims(kv_cache, kv_scales, B, width)
    _i32(parents, (n,), "parents", device)
    _i32(children, (n,), "children", device)
    status = _status(status, device)
    if n == 0:
        return
    raw = _launch_stream(device, stream)
    workspace = _workspace(workspace, 12 * n, device, stream)
    rc = lib().mla_cache_fork(d, n, parents.data_ptr(), children.data_ptr(), block_table.data_ptr(),
                              cache_seqlens.data_ptr(), ref_counts.data_ptr(), kv_cache.data_ptr(), scales,
                              workspace.data_ptr(), status, raw)
    if rc:
        _check(rc, "mla_cache_fork")


def cache_free(rows: torch.Tensor, block_table: torch.Tensor, cache_seqlens: torch.Tensor, ref_counts: torch.Tensor,
               status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gives up the pages of ``rows`` and empties them (mla_cache_free)."""
    device, n = block_table.device, rows.numel()
    nb = ref_counts.numel()
    B, width = _books(block_table, cache_seqlens, ref_counts, nb, device)
    _i32(rows, (n,), "rows", device)
    status = _status(status, device)
    if n == 0:
        return
    stream = _launch_stream(device, stream)
    rc = lib().mla_cache_free(_cache_dims(B, width, nb, MLA_CACHE_BF16), n, rows.data_ptr(), block_table.data_ptr(),
                              cache_seqlens.data_ptr(), ref_counts.data_ptr(), status, stream)
    if rc:
        _check(rc, "mla_cache_free")


def cache_copy_pages(src: torch.Tensor, dst: torch.Tensor, kv_cache: torch.Tensor, kv_scales: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Page dst[i] of the pool = page src[i], with its scale (mla_cache_copy_pages)."""
    device, n = kv_cache.device, src.numel()
    d, scales = _pool_dims(kv_cache, kv_scales, 1, 1)
    _i32(src, (n,), "src", device)
    _i32(dst, (n,), "dst", device)
    status = _status(status, device)
    if n == 0:
        return
    stream = _launch_stream(device, stream)
    rc = lib().mla_cache_copy_pages(d, n, src.data_ptr(), dst.data_ptr(), kv_cache.data_ptr(), scales, status, stream)
    if rc:
        _check(rc, "mla_cache_copy_pages")


def _workspace(workspace, need: int, device, stream) -> torch.Tensor:
    if workspace is None:
        workspace = _empty(need, torch.uint8, device, stream, "a workspace")
    elif workspace.dtype is not torch.uint8 or workspace.numel() < need or not workspace.is_contiguous() or \
            workspace.device != device:
        _fail("workspace must be %d bytes (uint8) on %s", need, device)
    return workspace


def cache_compact_workspace(num_blocks: int, device) -> torch.Tensor:
    """A workspace for cache_compact on a pool of num_blocks pages; its first
    int32 is the number of pages in use after a call."""
    n = int(lib().mla_cache_compact_workspace_bytes(_cache_dims(1, 1, int(num_blocks), MLA_CACHE_BF16)))
    if n == 0:
        raise MlaDecodeError(bd.MLA_ERR_INVALID_ARG, "cache_compact_workspace")
    return torch.empty(n, dtype=torch.uint8, device=device)


def cache_compact(block_table: torch.Tensor, cache_seqlens: torch.Tensor, ref_counts: torch.Tensor, kv_cache: torch.Tensor,
                  kv_scales: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Moves the pages in use to the front of the pool (mla_cache_compact)."""
    device, nb = kv_cache.device, kv_cache.shape[0]
    B, width = _books(block_table, cache_seqlens, ref_counts, nb, device)
    d, scales = _pool_dims(kv_cache, kv_scales, B, width)
    status = _status(status, device)
    raw = _launch_stream(device, stream)
    workspace = _workspace(workspace, 16 + 8 * nb, device, stream)
    rc = lib().mla_cache_compact(d, block_table.data_ptr(), cache_seqlens.data_ptr(), ref_counts.data_ptr(),
                                 kv_cache.data_ptr(), scales, workspace.data_ptr(), status, raw)
    if rc:
        _check(rc, "mla_cache_compact")


# ---------------------------------------------------------------- decode over the 8-bit cache
def mla_decode_q8_schedule_bytes(dims: mla_decode_dims) -> int:
    return int(lib().mla_decode_q8_schedule_bytes(ctypes.byref(dims)))


def mla_decode_q8_workspace_bytes(dims: mla_decode_dims) -> int:
    return int(lib().mla_decode_q8_workspace_bytes(ctypes.byref(dims)))


def mla_decode_q8_get_schedule(dims, cache_seqlens, schedule, stream=None) -> None:
    _check(lib().mla_decode_q8_get_schedule(ctypes.byref(dims), _ptr(cache_seqlens), _ptr(schedule), _stream(stream)),
           "mla_decode_q8_get_schedule")


def mla_decode_q8_get_schedule_host(dims, cache_seqlens, schedule) -> None:
    """Host version; ``cache_seqlens`` (int32) and ``schedule`` are CPU tensors."""
    _check(lib().mla_decode_q8_get_schedule_host(ctypes.byref(dims), _ptr(cache_seqlens), _ptr(schedule)),
           "mla_decode_q8_get_schedule_host")


def mla_decode_q8_fwd(dims, schedule, workspace, q, kv_cache, kv_scales, block_table, cache_seqlens, softmax_scale: float,
                      out, lse, stream=None) -> None:
    _check(lib().mla_decode_q8_fwd(ctypes.byref(dims), _ptr(schedule), _ptr(workspace), _ptr(q), _ptr(kv_cache),
                                   _ptr(kv_scales), _ptr(block_table), _ptr(cache_seqlens), float(softmax_scale), _ptr(out),
                                   _ptr(lse), _stream(stream)), "mla_decode_q8_fwd")


def mla_decode_q8_combine(dims, schedule, workspace, out, lse, stream=None) -> None:
    _check(lib().mla_decode_q8_combine(ctypes.byref(dims), _ptr(schedule), _ptr(workspace), _ptr(out), _ptr(lse),
                                       _stream(stream)), "mla_decode_q8_combine")


class Q8Decoder:
    """Schedule and workspace buffers for one shape of decode batch over the
    8-bit cache; same use as MlaDecoder, with the page scales beside the cache."""

    def __init__(self, batch: int, s_q: int, num_heads: int, num_blocks: int, max_blocks_per_seq: int,
                 causal: bool = False, num_sms: int = 0, device: Optional[torch.device] = None, fp32_out: bool = False,
                 inline_plan: bool = False):
        self.device = torch.device(device or "cuda")
        if num_sms == 0:
            num_sms = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.dims = bd.make_dims(batch, s_q, num_heads, num_blocks, max_blocks_per_seq, causal, num_sms,
                                 (bd.MLA_FLAG_FP32_OUT if fp32_out else 0) |
                                 (bd.MLA_FLAG_INLINE_PLAN if inline_plan else 0))
        sb, wb = mla_decode_q8_schedule_bytes(self.dims), mla_decode_q8_workspace_bytes(self.dims)
        if sb == 0 or wb == 0:
            raise MlaDecodeError(bd.MLA_ERR_INVALID_ARG, "Q8Decoder dims")
        self.schedule = torch.empty(sb, dtype=torch.uint8, device=self.device)
        self.workspace = torch.empty(wb, dtype=torch.uint8, device=self.device)
        self.out = torch.empty(batch, s_q, num_heads, bd.D_V, dtype=torch.float32 if fp32_out else torch.bfloat16,
                               device=self.device)
        self.lse = torch.empty(batch, num_heads, s_q, dtype=torch.float32, device=self.device)
        self._schedule, self._workspace = self.schedule.data_ptr(), self.workspace.data_ptr()
        self._out, self._lse = self.out.data_ptr(), self.lse.data_ptr()
        self._q_shape = torch.Size((batch, s_q, num_heads, bd.D_QK))
        self._kv_shape = torch.Size((num_blocks, bd.PAGE_SIZE, 1, bd.D_QK))
        self._scales_shape = torch.Size((num_blocks, 1))
        self._bt_shape = torch.Size((batch, max_blocks_per_seq))

    def check_inputs(self, q, kv_cache, kv_scales, block_table, cache_seqlens) -> None:
        device = self.out.device
        if q.dtype is not _BF16 or q.shape != self._q_shape or not q.is_contiguous() or q.device != device:
            _fail("q must be contiguous bf16 %s on %s", list(self._q_shape), device)
        if kv_cache.dtype is not _E4M3 or kv_cache.shape != self._kv_shape or not kv_cache.is_contiguous() or \
                kv_cache.device != device:
            _fail("kv_cache must be contiguous float8_e4m3fn %s on %s", list(self._kv_shape), device)
        if kv_scales.dtype is not _F32 or kv_scales.shape != self._scales_shape or not kv_scales.is_contiguous() or \
                kv_scales.device != device:
            _fail("kv_scales must be contiguous fp32 %s on %s", list(self._scales_shape), device)
        _i32(block_table, self._bt_shape, "block_table", device)
        _i32(cache_seqlens, self._bt_shape[:1], "cache_seqlens", device)

    def plan(self, cache_seqlens: torch.Tensor, stream=None) -> None:
        _i32(cache_seqlens, self._bt_shape[:1], "cache_seqlens", self.out.device)
        mla_decode_q8_get_schedule(self.dims, cache_seqlens, self.schedule, _launch_stream(self.out.device, stream))

    def __call__(self, q, kv_cache, kv_scales, block_table, cache_seqlens, softmax_scale: float, stream=None,
                 check: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
        if check:
            self.check_inputs(q, kv_cache, kv_scales, block_table, cache_seqlens)
        rc = lib().mla_decode_q8_fwd(ctypes.byref(self.dims), self._schedule, self._workspace, q.data_ptr(),
                                     kv_cache.data_ptr(), kv_scales.data_ptr(), block_table.data_ptr(),
                                     cache_seqlens.data_ptr(), softmax_scale, self._out, self._lse,
                                     _launch_stream(self.out.device, stream))
        if rc:
            _check(rc, "mla_decode_q8_fwd")
        return self.out, self.lse

    def status(self) -> int:
        return bd.mla_decode_get_status(self.schedule)


# ---------------------------------------------------------------- one layer's step
def absorbed_mla_step(q_in: torch.Tensor, c_kv: torch.Tensor, k_pe: torch.Tensor, positions: torch.Tensor,
                      new_offsets: torch.Tensor, w_uk: torch.Tensor, w_uv: torch.Tensor, rope: mla_rope_table,
                      block_table: torch.Tensor, cache_seqlens: torch.Tensor, kv_cache: torch.Tensor,
                      kv_scales: Optional[torch.Tensor], softmax_scale: float, decoder,
                      status: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One absorbed-MLA decode step for one layer, from the projections' outputs:
    the queries' RoPE part is rotated, the new rows are written into the cache,
    and ``absorbed_mla_decode`` follows over the cache as it then is.

    q_in [B, s_q, h, 192] (each head's 128-wide part, then its RoPE part), c_kv
    [B * s_q, 512] and k_pe [B * s_q, 64]: the new tokens' rows, request by request;
    positions [B * s_q] int32: theirs in their requests; new_offsets [B + 1] int32: 0,
    s_q, 2 s_q, ...; cache_seqlens counts the new rows.  ``decoder`` is a planned
    MlaDecoder for a bf16 cache (kv_scales None), or a Q8Decoder.  Returns (out
    [B, s_q, h, 128] bf16, lse [B, h, s_q])."""
    if isinstance(stream, torch.cuda.Stream):
        # (what the step allocates then belongs to that stream)
        with torch.cuda.stream(stream):
            return absorbed_mla_step(q_in, c_kv, k_pe, positions, new_offsets, w_uk, w_uv, rope, block_table, cache_seqlens,
                                     kv_cache, kv_scales, softmax_scale, decoder, status)
    if stream is not None:
        _fail("stream must be a torch.cuda.Stream")
    if q_in.dim() != 4:
        _fail("q_in must be [B, s_q, h, 192]")
    B, s_q, h, width = q_in.shape
    # What a later part would refuse is refused here, before rows are written into the cache.
    d, device = decoder.dims, kv_cache.device
    if isinstance(decoder, Q8Decoder) != (kv_scales is not None):
        _fail("an 8-bit cache and its scales go with a Q8Decoder, a bf16 cache with an MlaDecoder")
    if (B, s_q, h, width) != (d.batch, d.s_q, d.num_heads, bd.ABSORB_D_NOPE + bd.ABSORB_D_ROPE):
        _fail("q_in must be [B, s_q, h, 192] of the decoder's sizes")
    if kv_cache.shape[0] != d.num_blocks or block_table.shape != (B, d.max_blocks_per_seq) or decoder.out.device != device:
        _fail("kv_cache and block_table must have the decoder's sizes and device")
    if decoder.out.dtype is not _BF16:
        _fail("the decoder's output must be bf16")
    if q_in.dtype is not _BF16:
        _fail("q_in must be bf16")
    bd._bf16_on(w_uk, (h, bd.ABSORB_D_NOPE, bd.ABSORB_D_LATENT), "w_uk", device)
    bd._bf16_on(w_uv, (h, bd.ABSORB_D_LATENT, bd.ABSORB_D_V_HEAD), "w_uv", device)
    if not math.isfinite(softmax_scale):
        _fail("softmax_scale must be finite")
    q = rope_apply(q_in.reshape(B * s_q, h, width), positions, rope, offset=bd.ABSORB_D_NOPE).view(q_in.shape)
    cache_append(c_kv, k_pe, new_offsets, block_table, cache_seqlens, kv_cache, kv_scales, rope, status)
    q_lat = bd.absorb_q(q, w_uk)
    if kv_scales is None:
        o_lat, lse = decoder(q_lat, kv_cache, block_table, cache_seqlens, softmax_scale)
    else:
        o_lat, lse = decoder(q_lat, kv_cache, kv_scales, block_table, cache_seqlens, softmax_scale)
    return bd.absorb_o(o_lat, w_uv), lse
