"""Python binding of include/mla_cache.h (ctypes): rotary positions, the write of
new rows into the paged latent cache, decode attention over the cache in 8 bits,
and the fork, free, copy and compaction of pages.

Argument marshalling only, like ``binding``: every step runs in the CUDA kernels
of libmla_decode.so, and there is no fallback.
"""
from __future__ import annotations

import ctypes
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


def _i32(t: torch.Tensor, shape, what: str, device) -> None:
    _require(t.dtype == torch.int32 and t.is_contiguous() and tuple(t.shape) == tuple(shape),
             "%s must be contiguous int32 %s" % (what, list(shape)))
    _require(t.device == device, "%s must be on %s" % (what, device))


def _on_current(device: torch.device, stream) -> None:
    """The library launches on the current device; a stream carries its own."""
    dev = stream.device if isinstance(stream, torch.cuda.Stream) else None
    _require(device.type == "cuda", "tensors must be on a CUDA device")
    _require(device.index == torch.cuda.current_device() and (dev is None or dev == device),
             "tensors and stream must be of the current CUDA device")


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
    the result."""
    _require(x.dim() in (2, 3), "x must be [T, h, W] or [T, W]")
    _require(x.dtype in (torch.bfloat16, torch.float32), "x must be bf16 or fp32")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _require(out.shape == x.shape and out.dtype == x.dtype and out.device == x.device,
             "out must have the shape, type and device of x")
    T, W = x.shape[0], x.shape[-1]
    h = x.shape[1] if x.dim() == 3 else 1
    _i32(positions, (T,), "positions", x.device)
    if T == 0 or h == 0:
        return out
    _require(x.stride(-1) == 1 and out.stride(-1) == 1, "the columns of x and out must be contiguous")
    _on_current(x.device, stream)

    def strides(t):  # (a dimension of one row has no stride of its own)
        hs = t.stride(1) if t.dim() == 3 and h > 1 else W
        return (t.stride(0) if T > 1 else h * hs), hs

    d = mla_rope_dims(T, h, W, int(offset), *strides(x), *strides(out),
                      MLA_DTYPE_BF16 if x.dtype == torch.bfloat16 else MLA_DTYPE_FP32, int(bool(transpose)))
    _check(lib().mla_rope_apply(ctypes.byref(d), ctypes.byref(rope), _ptr(x), _ptr(positions), _ptr(out), _stream(stream)),
           "mla_rope_apply")
    return out


# ---------------------------------------------------------------- the cache
def _pool_dims(kv_cache: torch.Tensor, kv_scales: Optional[torch.Tensor], batch: int, max_blocks: int) -> mla_cache_dims:
    nb = kv_cache.shape[0]
    q8 = kv_cache.dtype == torch.float8_e4m3fn
    _require((q8 or kv_cache.dtype == torch.bfloat16) and kv_cache.is_contiguous() and
             tuple(kv_cache.shape) == (nb, bd.PAGE_SIZE, 1, bd.D_QK),
             "kv_cache must be contiguous bf16 or float8_e4m3fn [num_blocks, 64, 1, 576]")
    if q8:
        _require(kv_scales is not None and kv_scales.dtype == torch.float32 and kv_scales.is_contiguous() and
                 tuple(kv_scales.shape) == (nb, 1) and kv_scales.device == kv_cache.device,
                 "kv_scales must be contiguous fp32 [num_blocks, 1] beside an 8-bit cache")
    else:
        _require(kv_scales is None, "a bf16 cache has no scales")
    return mla_cache_dims(int(batch), int(max_blocks), int(nb), bd.PAGE_SIZE, bd.D_QK,
                          MLA_CACHE_E4M3 if q8 else MLA_CACHE_BF16)


def _books(block_table, cache_seqlens, ref_counts, nb, device) -> None:
    _require(block_table.dim() == 2, "block_table must be int32 [B, max_blocks_per_seq]")
    _i32(block_table, block_table.shape, "block_table", device)
    _i32(cache_seqlens, (block_table.shape[0],), "cache_seqlens", device)
    if ref_counts is not None:
        _i32(ref_counts, (nb,), "ref_counts", device)


def _status(status: Optional[torch.Tensor], device) -> None:
    if status is not None:
        _require(status.dtype == torch.int32 and status.numel() >= 1 and status.is_contiguous() and status.device == device,
                 "status must be int32 on %s" % device)


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
    _books(block_table, cache_seqlens, None, 0, device)
    d = _pool_dims(kv_cache, kv_scales, block_table.shape[0], block_table.shape[1])
    for t, w, what in ((c_kv, bd.D_V, "c_kv"), (k_pe, bd.D_QK - bd.D_V, "k_pe")):
        _require(t.dtype == torch.bfloat16 and t.dim() == 2 and tuple(t.shape) == (T, w) and
                 (t.stride(1) == 1 or t.numel() == 0) and t.device == device, "%s must be bf16 [T, %d] on %s" % (what, w, device))
    _i32(new_offsets, (block_table.shape[0] + 1,), "new_offsets", device)
    _status(status, device)
    if T == 0:
        return
    _on_current(device, stream)
    _check(lib().mla_cache_append(ctypes.byref(d), T, _ptr(c_kv), c_kv.stride(0) if T > 1 else bd.D_V, _ptr(k_pe),
                                  k_pe.stride(0) if T > 1 else bd.D_QK - bd.D_V, _ptr(new_offsets),
                                  None if rope is None else ctypes.byref(rope), _ptr(block_table), _ptr(cache_seqlens),
                                  _ptr(kv_cache), _ptr(kv_scales), _ptr(status), _stream(stream)), "mla_cache_append")


def cache_fork(parents: torch.Tensor, children: torch.Tensor, block_table: torch.Tensor, cache_seqlens: torch.Tensor,
               ref_counts: torch.Tensor, kv_cache: torch.Tensor, kv_scales: Optional[torch.Tensor] = None,
               status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Makes the empty rows ``children`` copies of ``parents`` (mla_cache_fork): full
    pages are shared and counted, a last page that is not full is copied
    into the lowest free page."""
    device, n = kv_cache.device, parents.numel()
    _books(block_table, cache_seqlens, ref_counts, kv_cache.shape[0], device)
    d = _pool_dims(kv_cache, kv_scales, block_table.shape[0], block_table.shape[1])
    _i32(parents, (n,), "parents", device)
    _i32(children, (n,), "children", device)
    _status(status, device)
    if n == 0:
        return
    _on_current(device, stream)
    workspace = _workspace(workspace, int(lib().mla_cache_fork_workspace_bytes(n)), device, stream)
    _check(lib().mla_cache_fork(ctypes.byref(d), n, _ptr(parents), _ptr(children), _ptr(block_table), _ptr(cache_seqlens),
                                _ptr(ref_counts), _ptr(kv_cache), _ptr(kv_scales), _ptr(workspace), _ptr(status),
                                _stream(stream)), "mla_cache_fork")


def cache_free(rows: torch.Tensor, block_table: torch.Tensor, cache_seqlens: torch.Tensor, ref_counts: torch.Tensor,
               status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Gives up the pages of ``rows`` and empties them (mla_cache_free)."""
    device, n = block_table.device, rows.numel()
    nb = ref_counts.numel()
    _books(block_table, cache_seqlens, ref_counts, nb, device)
    _i32(rows, (n,), "rows", device)
    _status(status, device)
    if n == 0:
        return
    _on_current(device, stream)
    d = mla_cache_dims(block_table.shape[0], block_table.shape[1], nb, bd.PAGE_SIZE, bd.D_QK, MLA_CACHE_BF16)
    _check(lib().mla_cache_free(ctypes.byref(d), n, _ptr(rows), _ptr(block_table), _ptr(cache_seqlens), _ptr(ref_counts),
                                _ptr(status), _stream(stream)), "mla_cache_free")


def cache_copy_pages(src: torch.Tensor, dst: torch.Tensor, kv_cache: torch.Tensor, kv_scales: Optional[torch.Tensor] = None,
                     status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Page dst[i] of the pool = page src[i], with its scale (mla_cache_copy_pages)."""
    device, n = kv_cache.device, src.numel()
    d = _pool_dims(kv_cache, kv_scales, 1, 1)
    _i32(src, (n,), "src", device)
    _i32(dst, (n,), "dst", device)
    _status(status, device)
    if n == 0:
        return
    _on_current(device, stream)
    _check(lib().mla_cache_copy_pages(ctypes.byref(d), n, _ptr(src), _ptr(dst), _ptr(kv_cache), _ptr(kv_scales),
                                      _ptr(status), _stream(stream)), "mla_cache_copy_pages")


def _workspace(workspace, need: int, device, stream) -> torch.Tensor:
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        if isinstance(stream, torch.cuda.Stream):
            workspace.record_stream(stream)  # it is dropped before the stream has run
        else:
            _require(stream is None, "a raw stream handle needs a workspace of the caller's")
    _require(workspace.dtype == torch.uint8 and workspace.is_contiguous() and workspace.numel() >= need and
             workspace.device == device, "workspace must be %d bytes (uint8) on %s" % (need, device))
    return workspace


def cache_compact_workspace(num_blocks: int, device) -> torch.Tensor:
    """A workspace for cache_compact on a pool of num_blocks pages; its first
    int32 is the number of pages in use after a call."""
    d = mla_cache_dims(1, 1, int(num_blocks), bd.PAGE_SIZE, bd.D_QK, MLA_CACHE_BF16)
    n = int(lib().mla_cache_compact_workspace_bytes(ctypes.byref(d)))
    if n == 0:
        raise MlaDecodeError(bd.MLA_ERR_INVALID_ARG, "cache_compact_workspace")
    return torch.empty(n, dtype=torch.uint8, device=device)


def cache_compact(block_table: torch.Tensor, cache_seqlens: torch.Tensor, ref_counts: torch.Tensor, kv_cache: torch.Tensor,
                  kv_scales: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  status: Optional[torch.Tensor] = None, stream=None) -> None:
    """Moves the pages in use to the front of the pool (mla_cache_compact)."""
    device, nb = kv_cache.device, kv_cache.shape[0]
    _books(block_table, cache_seqlens, ref_counts, nb, device)
    d = _pool_dims(kv_cache, kv_scales, block_table.shape[0], block_table.shape[1])
    _status(status, device)
    _on_current(device, stream)
    workspace = _workspace(workspace, int(lib().mla_cache_compact_workspace_bytes(ctypes.byref(d))), device, stream)
    _check(lib().mla_cache_compact(ctypes.byref(d), _ptr(block_table), _ptr(cache_seqlens), _ptr(ref_counts), _ptr(kv_cache),
                                   _ptr(kv_scales), _ptr(workspace), _ptr(status), _stream(stream)), "mla_cache_compact")


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

    def check_inputs(self, q, kv_cache, kv_scales, block_table, cache_seqlens) -> None:
        d = self.dims
        _require(q.dtype == torch.bfloat16 and q.is_contiguous() and
                 tuple(q.shape) == (d.batch, d.s_q, d.num_heads, bd.D_QK), "q must be bf16 [B, s_q, h, 576]")
        _require(kv_cache.dtype == torch.float8_e4m3fn and kv_cache.is_contiguous() and
                 tuple(kv_cache.shape) == (d.num_blocks, bd.PAGE_SIZE, 1, bd.D_QK),
                 "kv_cache must be float8_e4m3fn [num_blocks, 64, 1, 576]")
        _require(kv_scales.dtype == torch.float32 and kv_scales.is_contiguous() and
                 tuple(kv_scales.shape) == (d.num_blocks, 1), "kv_scales must be fp32 [num_blocks, 1]")
        _require(block_table.dtype == torch.int32 and block_table.is_contiguous() and
                 tuple(block_table.shape) == (d.batch, d.max_blocks_per_seq),
                 "block_table must be int32 [B, max_blocks_per_seq]")
        _require(cache_seqlens.dtype == torch.int32 and cache_seqlens.is_contiguous() and
                 tuple(cache_seqlens.shape) == (d.batch,), "cache_seqlens must be int32 [B]")
        for t in (q, kv_cache, kv_scales, block_table, cache_seqlens):
            _require(t.device == self.out.device, "all tensors must be on %s" % self.out.device)

    def plan(self, cache_seqlens: torch.Tensor, stream=None) -> None:
        mla_decode_q8_get_schedule(self.dims, cache_seqlens, self.schedule, stream)

    def __call__(self, q, kv_cache, kv_scales, block_table, cache_seqlens, softmax_scale: float, stream=None,
                 check: bool = True) -> Tuple[torch.Tensor, torch.Tensor]:
        if check:
            self.check_inputs(q, kv_cache, kv_scales, block_table, cache_seqlens)
        mla_decode_q8_fwd(self.dims, self.schedule, self.workspace, q, kv_cache, kv_scales, block_table, cache_seqlens,
                          softmax_scale, self.out, self.lse, stream)
        return self.out, self.lse

    def status(self) -> int:
        return bd.mla_decode_get_status(self.schedule)
