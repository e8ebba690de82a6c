"""Boundary of include/mla_cache.h, CPU only: every declared function is exported and
bound, bad arguments are refused before the device is touched, and the rotary
table's numbers.  The fp64 oracle of the cache's operators is pinned here too."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import helpers
from mla_decode_attention_15_b200 import _build, binding as bd, cache as ca
from oracle import cache as oc

OK, BAD, UNSUP = bd.MLA_OK, bd.MLA_ERR_INVALID_ARG, bd.MLA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return ca.lib()


def test_header_symbols_are_exported_and_bound(lib):
    text = open(os.path.join(helpers.ROOT, "include", "mla_cache.h")).read()
    names = set(re.findall(r"^(?:int|size_t)\s+(mla_\w+)\s*\(", text, re.M))
    assert names == set(ca.CACHE_EXPORTED)
    dyn = subprocess.run(["nm", "-D", "--defined-only", _build.LIB], capture_output=True, text=True).stdout
    for n in names:
        assert (" T " + n) in dyn, n
    assert ca.mla_cache_version() == 1


# ------------------------------------------------------------------ rotary table
def _cfg(**kw):
    base = dict(theta=10000.0, factor=4.0, beta_fast=32.0, beta_slow=1.0, amplitude=1.0, original_max_position=4096,
                scaling=ca.MLA_ROPE_YARN, interleaved=1, reserved=0)
    base.update(kw)
    return ca.mla_rope_config(**base)


@pytest.mark.parametrize("change", [dict(theta=1.0), dict(theta=math.inf), dict(theta=math.nan), dict(factor=0.0),
                                    dict(factor=math.nan), dict(beta_fast=0.0), dict(beta_slow=-1.0), dict(amplitude=math.inf),
                                    dict(original_max_position=0), dict(scaling=3), dict(scaling=-1), dict(interleaved=2),
                                    dict(reserved=1)])
def test_rope_init_refusals(lib, change):
    t = ca.mla_rope_table()
    assert lib.mla_rope_init(ctypes.byref(_cfg(**change)), ctypes.byref(t)) == BAD
    assert lib.mla_rope_init(None, ctypes.byref(t)) == BAD
    assert lib.mla_rope_init(ctypes.byref(_cfg()), None) == BAD


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=8.0), dict(scaling="yarn", factor=40.0),
                                dict(scaling="yarn", factor=4.0, original_max_position=32768, theta=1e6),
                                dict(scaling="yarn", factor=2.0, original_max_position=8)])
def test_rope_table_frequencies(lib, kw):
    got = np.array(list(ca.make_rope(**kw).turns)) * 2 * math.pi
    np.testing.assert_allclose(got, oc.frequencies(**kw), rtol=1e-14)


def test_make_rope_names_its_scalings(lib):
    with pytest.raises(ValueError):
        ca.make_rope(scaling="ntk")


# ------------------------------------------------------------------ refusals
def _rope_rc(lib, ptrs=(0x1000, 0x2000, 0x3000), **kw):
    base = dict(tokens=4, num_heads=2, width=192, offset=128, x_token_stride=384, x_head_stride=192, out_token_stride=384,
                out_head_stride=192, dtype=0, transpose=0)
    base.update(kw)
    d = ca.mla_rope_dims(**base)
    t = ca.make_rope()
    return lib.mla_rope_apply(ctypes.byref(d), ctypes.byref(t), *ptrs, None)


@pytest.mark.parametrize("kw,code", [
    (dict(tokens=-1), BAD), (dict(num_heads=0), BAD), (dict(num_heads=65536), BAD), (dict(width=2056), BAD), (dict(width=56), BAD), (dict(width=196), BAD), (dict(offset=4), BAD),
    (dict(offset=136), BAD), (dict(offset=-8), BAD), (dict(width=65544), BAD), (dict(transpose=2), BAD), (dict(dtype=2), UNSUP),
    (dict(x_token_stride=385), BAD), (dict(x_head_stride=-192), BAD),
    (dict(out_head_stride=184), BAD), (dict(out_token_stride=376), BAD), (dict(out_token_stride=0), BAD)])
def test_rope_apply_refusals(lib, kw, code):
    assert _rope_rc(lib, **kw) == code


def test_rope_apply_pointers(lib):
    for i in range(3):
        p = [0x1000, 0x2000, 0x3000]
        p[i] = None
        assert _rope_rc(lib, tuple(p)) == BAD
        p[i] = 0x4002
        assert _rope_rc(lib, tuple(p)) == BAD
    assert _rope_rc(lib, (0x1000, 0x2000, 0x1000), x_token_stride=0) == BAD  # in place with other strides
    assert _rope_rc(lib, (None, None, None), tokens=0) == OK
    assert lib.mla_rope_apply(None, None, None, None, None, None) == BAD


def _cache_dims(**kw):
    base = dict(batch=2, max_blocks_per_seq=4, num_blocks=8, page_size=64, row_width=576, dtype=ca.MLA_CACHE_E4M3)
    base.update(kw)
    return ca.mla_cache_dims(**base)


BAD_DIMS = [(dict(batch=0), BAD), (dict(max_blocks_per_seq=0), BAD), (dict(num_blocks=0), BAD), (dict(page_size=32), UNSUP),
            (dict(row_width=512), UNSUP), (dict(dtype=2), UNSUP), (dict(batch=1 << 20, max_blocks_per_seq=1 << 12), UNSUP),
            (dict(max_blocks_per_seq=1 << 26), UNSUP)]


def _calls(lib):
    """name -> (function of (dims, pointers) -> rc, number of pointers, those that need 16 bytes, that may be NULL)"""
    def append(d, p):
        return lib.mla_cache_append(d, 3, p[0], 512, p[1], 64, p[2], None, p[3], p[4], p[5], p[6], p[7], None)

    def fork(d, p):
        return lib.mla_cache_fork(d, 2, *p, None)

    def free(d, p):
        return lib.mla_cache_free(d, 2, *p, None)

    def copy(d, p):
        return lib.mla_cache_copy_pages(d, 2, *p, None)

    def compact(d, p):
        return lib.mla_cache_compact(d, *p, None)

    return dict(append=(append, 8, (0, 1, 5, 6), (7,)), fork=(fork, 9, (5, 6, 7), (8,)), free=(free, 5, (), (4,)),
                copy=(copy, 5, (2, 3), (4,)), compact=(compact, 7, (3, 4, 5), (6,)))


@pytest.mark.parametrize("name", ["append", "fork", "free", "copy", "compact"])
def test_cache_call_refusals(lib, name):
    fn, n, wide, opt = _calls(lib)[name]
    ptrs = [0x10000 * (i + 1) for i in range(n)]
    for kw, code in BAD_DIMS:
        assert fn(ctypes.byref(_cache_dims(**kw)), ptrs) == code, kw
    assert fn(None, ptrs) == BAD
    d = ctypes.byref(_cache_dims())
    for i in range(n):
        p = list(ptrs)
        if i not in opt:
            p[i] = None
            assert fn(d, p) == BAD, i
        p[i] = 0x90002
        assert fn(d, p) == BAD, i
        if i in wide:
            p[i] = 0x90008
            assert fn(d, p) == BAD, i
    if name != "free":  # a bf16 pool has no scales
        assert fn(ctypes.byref(_cache_dims(dtype=ca.MLA_CACHE_BF16)), ptrs) == BAD


def test_cache_counts_and_strides(lib):
    d, P = ctypes.byref(_cache_dims()), [0x10000 * (i + 1) for i in range(9)]
    for n in (0, -1, ca.FORK_MAX + 1):
        assert lib.mla_cache_fork(d, n, *P, None) == BAD
        assert lib.mla_cache_fork_workspace_bytes(n) == 0
    assert lib.mla_cache_fork_workspace_bytes(ca.FORK_MAX) >= 12 * ca.FORK_MAX
    assert lib.mla_cache_free(d, 0, *P[:5], None) == BAD
    assert lib.mla_cache_copy_pages(d, -1, *P[:5], None) == BAD
    assert lib.mla_cache_copy_pages(d, 0, None, None, *P[:2], None, None) == OK
    for cs, ps, T in ((504, 64, 3), (516, 64, 3), (512, 56, 3), (512, 68, 3), (512, 64, -1)):
        assert lib.mla_cache_append(d, T, P[0], cs, P[1], ps, P[2], None, P[3], P[4], P[5], P[6], None, None) == BAD
    assert lib.mla_cache_append(d, 0, None, 512, None, 64, P[2], None, P[3], P[4], P[5], P[6], None, None) == OK
    assert lib.mla_cache_compact_workspace_bytes(ctypes.byref(_cache_dims(num_blocks=0))) == 0
    # (what the Python wrappers allocate)
    assert lib.mla_cache_compact_workspace_bytes(d) == 16 + 8 * 8
    assert [lib.mla_cache_fork_workspace_bytes(n) for n in (1, 7, 1024)] == [12, 84, 12288]


def _q8_rc(lib, d, p):
    return lib.mla_decode_q8_fwd(ctypes.byref(d), *p[:7], ctypes.c_float(0.07), p[7], p[8], None)


def _dd(**kw):
    base = dict(batch=4, s_q=1, num_heads=16, num_blocks=100, max_blocks_per_seq=10, causal=False, num_sms=148)
    base.update(kw)
    return bd.make_dims(**base)


def test_q8_decode_refusals(lib):
    P = [0x10000 * (i + 1) for i in range(9)]
    d = _dd()
    for i in range(9):
        for bad in (None, 0x90008):
            p = list(P)
            p[i] = bad
            assert _q8_rc(lib, d, p) == BAD, (i, bad)
    for kw, code in [(dict(batch=0), BAD), (dict(s_q=3), UNSUP), (dict(num_heads=257), UNSUP), (dict(num_heads=129, s_q=2), UNSUP),
                     (dict(flags=0x100), BAD), (dict(num_blocks=0), BAD)]:
        assert _q8_rc(lib, _dd(**kw), P) == code, kw
        assert ca.mla_decode_q8_schedule_bytes(_dd(**kw)) == 0 and ca.mla_decode_q8_workspace_bytes(_dd(**kw)) == 0
        assert lib.mla_decode_q8_get_schedule(ctypes.byref(_dd(**kw)), P[0], P[1], None) == code
        assert lib.mla_decode_q8_combine(ctypes.byref(_dd(**kw)), *P[:4], None) == code
    assert lib.mla_decode_q8_fwd(ctypes.byref(d), *P[:7], ctypes.c_float(math.nan), *P[7:], None) == BAD


def test_q8_sizes(lib):
    # 16 columns: one group of 16; 17 .. 32: one of 32; more: groups of 32 that share ranges of pages
    assert ca.mla_decode_q8_workspace_bytes(_dd()) == 2 * 148 * 16 * 513 * 4
    assert ca.mla_decode_q8_workspace_bytes(_dd(num_heads=17)) == 2 * 148 * 32 * 513 * 4
    assert ca.mla_decode_q8_workspace_bytes(_dd(num_heads=128, s_q=2)) == 2 * 18 * 8 * 32 * 513 * 4
    assert ca.mla_decode_q8_workspace_bytes(_dd(num_heads=128, s_q=2, num_sms=4)) == 2 * 4 * 32 * 513 * 4


@pytest.mark.parametrize("h,s_q,G,share", [(16, 1, 148, 1), (128, 2, 18, 8), (33, 2, 49, 3)])
def test_q8_host_plan_covers_every_page_once(lib, h, s_q, G, share):
    lens = torch.tensor([1, 64, 65, 5000, 0, 640], dtype=torch.int32)
    d = _dd(batch=6, num_heads=h, s_q=s_q, max_blocks_per_seq=80)
    buf = torch.zeros(ca.mla_decode_q8_schedule_bytes(d), dtype=torch.uint8)
    ca.mla_decode_q8_get_schedule_host(d, lens, buf)
    hdr, meta, bginfo, prefix = helpers.read_plan(buf.numpy(), G, 6)
    assert hdr[1] == G and hdr[12] == share and hdr[11] == 6
    seen = {}
    for items in helpers.walk_plan(meta, bginfo, lens, 1, 80):
        for bg, p0, p1, unsplit, slot in items:
            for j in range(p0, p1):
                assert seen.setdefault((bg, j), slot) == slot
    assert len(seen) == sum((int(n) + 63) // 64 for n in lens)


@pytest.mark.parametrize("G", [1, 2, 7, 32, 148])
def test_q8_host_plan_of_ragged_batches(lib, G):
    """Ranges that fall inside an item's overhead are empty and belong to no split."""
    g = torch.Generator().manual_seed(G)
    for trial in range(40):
        B = int(torch.randint(1, 60, (1,), generator=g))
        lens = torch.randint(0, (65, 300, 5120)[trial % 3], (B,), generator=g, dtype=torch.int32)
        d = _dd(batch=B, num_heads=16, max_blocks_per_seq=80, num_sms=G)
        buf = torch.zeros(ca.mla_decode_q8_schedule_bytes(d), dtype=torch.uint8)
        ca.mla_decode_q8_get_schedule_host(d, lens, buf)
        hdr, meta, bginfo, prefix = helpers.read_plan(buf.numpy(), G, B)
        pieces, seen = {}, set()
        for items in helpers.walk_plan(meta, bginfo, lens, 1, 80):
            for bg, p0, p1, unsplit, slot in items:
                if p1 > p0:
                    pieces.setdefault(bg, []).append((p0, p1, slot))
                    assert unsplit or slot not in seen and 0 <= slot < 2 * G
                    seen |= set() if unsplit else {slot}
        for b, n in enumerate(lens.tolist()):
            got = sorted(pieces.get(b, []))
            assert [x for p0, p1, _ in got for x in range(p0, p1)] == list(range((n + 63) // 64))
            assert int(bginfo[b][1]) == len(got)
            s0 = int(bginfo[b][0])
            if len(got) > 1:   # the slots the combine kernel reads
                assert [s for _, _, s in got] == [s0] + [2 * ((s0 >> 1) + i) for i in range(1, len(got))]


def test_python_wrappers_check_shapes(lib):
    kv = torch.zeros(4, 64, 1, 576, dtype=torch.float8_e4m3fn)
    sc = torch.ones(4, 1)
    bt, sl = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    off, refs = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    c, k = torch.zeros(3, 512, dtype=torch.bfloat16), torch.zeros(3, 64, dtype=torch.bfloat16)
    rows = torch.zeros(1, dtype=torch.int32)
    for call in (lambda: ca.cache_append(c.float(), k, off, bt, sl, kv, sc), lambda: ca.cache_append(c, k, off, bt, sl, kv),
                 lambda: ca.cache_append(c, k[:2], off, bt, sl, kv, sc), lambda: ca.cache_append(c, k, off[:2], bt, sl, kv, sc),
                 lambda: ca.cache_append(c, k, off, bt, sl, kv.view(torch.uint8), sc),
                 lambda: ca.cache_append(c, k, off, bt, sl, torch.zeros(4, 64, 1, 576, dtype=torch.bfloat16), sc),
                 lambda: ca.cache_append(c, k, off, bt, sl, kv, sc),                      # CPU tensors
                 lambda: ca.cache_fork(rows, rows, bt, sl, refs[:3], kv, sc), lambda: ca.cache_fork(rows, rows.long(), bt, sl, refs, kv, sc),
                 lambda: ca.cache_free(rows, bt, sl[:1], refs), lambda: ca.cache_compact(bt, sl, refs, kv),
                 lambda: ca.cache_copy_pages(rows, off, kv, sc),
                 lambda: ca.rope_apply(torch.zeros(2, 2, 192), off, ca.make_rope()),
                 lambda: ca.rope_apply(torch.zeros(3, 2, 192, dtype=torch.float16), off, ca.make_rope())):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the oracle
def test_oracle_e4m3_and_scales():
    v = np.concatenate([np.random.RandomState(0).randn(4096) * 30, [0, 448, -448, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 17, 0.0634765625]])
    want = torch.from_numpy(v).float().to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(oc.e4m3(v.astype(np.float32)), want)
    assert oc.scale_of(448.0) == 1 and oc.scale_of(448.5) == 2 and oc.scale_of(224.0) == 0.5 and oc.scale_of(224.1) == 1
    assert oc.scale_of(0.0) == 2.0 ** -100 and oc.scale_of(3e38) == 2.0 ** 119
    assert np.isnan(oc.e4m3(np.array([np.inf, -np.inf, np.nan]))).all()


def test_oracle_rotation_keeps_lengths_and_offsets():
    x = np.random.RandomState(1).randn(4, 64)
    for inter in (True, False):
        y = oc.rotate(x, [0, 1, 70000, 2 ** 31 - 1], interleaved=inter)
        np.testing.assert_allclose(y[0], x[0])
        np.testing.assert_allclose((y ** 2).sum(1), (x ** 2).sum(1))
        np.testing.assert_allclose(oc.rotate(y, [0, 1, 70000, 2 ** 31 - 1], interleaved=inter, transpose=True), x, atol=1e-12)
    # the score of two rotated rows depends on their distance alone
    a, b = np.random.RandomState(2).randn(2, 1, 64)
    s = [float((oc.rotate(a, [p + 5]) * oc.rotate(b, [p])).sum()) for p in (0, 3, 1000)]
    np.testing.assert_allclose(s, s[0], rtol=1e-9)


@pytest.mark.parametrize("kw", [dict(amplitude=1e39), dict(amplitude=-1e300), dict(scaling="linear", factor=1e-308),
                                dict(scaling="linear", factor=5e-324), dict(scaling="yarn", factor=1e-305)])
def test_rope_tables_that_hold_no_numbers_are_refused(lib, kw):
    """An amplitude that is infinite in fp32, and frequencies by which an angle would be."""
    with pytest.raises(bd.MlaDecodeError):
        ca.make_rope(**kw)
    ca.make_rope(amplitude=3e38)
    ca.make_rope(scaling="linear", factor=1e-200)
