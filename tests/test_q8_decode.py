"""Decode attention over the 8-bit cache against the fp64 oracle.

An e4m3 value times a power of two is a bf16 value, so the C oracle reads the same
cache, widened.  Tolerance of one fp32 output value, from the arithmetic (M: the
weights' mean of |v|; n visible tokens; R: the largest page scale):
  - a weight is rounded to fp16's 11 bits, half a step 2^-12, or cut off below 2^-22
    of the largest weight times R * 448 at most:      2^-12 M + 2^-22 n R 448 w_max
  - a score is off by dz (fp32 sums of 2 x 576 exact products, and the query's remainder:
    half of e4m3's last subnormal place is 2^-10, a sixteenth of it in the second term,
    over a largest magnitude of at least 224: below 2^-21 of that):    2 dz M
  - exponentials, sums, merge of splits and the division in fp32:    2^-18 M
A bf16 output adds one rounding, half of its eps."""
import ctypes

import numpy as np
import pytest
import torch

import helpers
import oracle
from mla_decode_attention_15_b200 import _build, binding as bd, cache as ca

pytestmark = pytest.mark.gpu
SCALE = 192 ** -0.5


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    _build.build()
    oracle.build()
    return torch.device("cuda:0")


def build(lens, s_q, h, seed, sigma=1.0, spread=0, peaked=False, spare=3):
    """CPU tensors; page scales vary by 2^spread around the values' own."""
    g = torch.Generator().manual_seed(seed)
    pages = [(n + 63) // 64 for n in lens]
    nb, width = sum(pages) + spare, max(max(pages), 1)
    x = torch.randn(nb, 64, 576, generator=g) * sigma * torch.exp2(torch.randint(-spread, spread + 1, (nb, 1, 1), generator=g).float())
    if peaked:
        x[torch.rand(nb, 64, generator=g) < 0.02] *= 8
    e = torch.ceil(torch.log2(x.abs().amax((1, 2)) / 448))
    scales = torch.exp2(e)[:, None].contiguous()
    kv = (x / scales[:, :, None]).to(torch.float8_e4m3fn)[:, :, None].contiguous()
    ids = torch.randperm(nb, generator=g).int()
    bt = torch.full((len(lens), width), -1, dtype=torch.int32)
    k = 0
    for b, p in enumerate(pages):
        bt[b, :p] = ids[k:k + p]
        k += p
    q = (torch.randn(len(lens), s_q, h, 576, generator=g) * sigma).bfloat16()
    return dict(q=q, kv=kv, scales=scales, bt=bt, lens=torch.tensor(lens, dtype=torch.int32))


def wide(d):
    return (d["kv"].float() * d["scales"][:, :, None, None]).bfloat16()


def reference(d, causal):
    return oracle.mla_oracle_fwd(d["q"], wide(d), d["bt"], d["lens"], SCALE, causal=causal)


def bounds(d, causal):
    """[rows, 512] bound on an fp32 output and [rows] bound on a score, rows as the oracle's."""
    B, s_q, h, _ = d["q"].shape
    tol, dzs = np.zeros((B * s_q * h, 512)), np.zeros(B * s_q * h)
    kv = wide(d)
    for b in range(B):
        L = int(d["lens"][b])
        ids = d["bt"][b, :(L + 63) // 64].long()
        k = kv[ids].double().reshape(-1, 576)[:L]
        R = float(d["scales"][ids].max()) if len(ids) else 0.0
        for s in range(s_q):
            n = L - s_q + 1 + s if causal and s_q > 1 else L
            r = slice((b * s_q + s) * h, (b * s_q + s + 1) * h)
            if n <= 0:
                continue
            q, kk = d["q"][b, s].double(), k[:n]
            w = torch.softmax(q @ kk.T * SCALE, -1)
            dz = SCALE * (1152 * 2.0 ** -24 * (q.abs() @ kk.abs().T).amax(-1) +
                          2.0 ** -21 * q.abs().amax(-1) * kk.abs().sum(-1).max())
            M = w @ kk[:, :512].abs()
            dzs[r] = dz.numpy()
            tol[r] = ((2.0 ** -12 + 2.0 ** -18 + 2 * dz)[:, None] * M +
                      (2.0 ** -22 * n * R * 448 * w.amax(-1))[:, None]).numpy()
    return tol, dzs


def run(d, dev, causal=False, inline=False, num_sms=0, fp32=False, dec=None):
    g = {k: v.to(dev) for k, v in d.items()}
    B, s_q, h, _ = d["q"].shape
    dec = dec or ca.Q8Decoder(B, s_q, h, d["kv"].shape[0], d["bt"].shape[1], causal, num_sms, dev, fp32, inline)
    dec.plan(g["lens"])
    dec.out.fill_(float("nan"))
    dec.lse.fill_(float("nan"))
    dec.workspace.fill_(0xff)
    out, lse = dec(g["q"], g["kv"], g["scales"], g["bt"], g["lens"], SCALE)
    torch.cuda.synchronize()
    assert dec.status() == 0
    return out.cpu().clone(), lse.cpu().clone()


def check(d, out, lse, causal):
    ref, rl = reference(d, causal)
    B, s_q, h, _ = d["q"].shape
    tol, dz = bounds(d, causal)
    if out.dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    err = np.abs(out.double().numpy().reshape(-1, 512) - ref)
    assert (err <= tol).all(), (np.nanmax(err / np.maximum(tol, 1e-300)), np.argwhere(~(err <= tol))[0])
    got = lse.double().numpy().transpose(0, 2, 1).reshape(-1)
    assert np.array_equal(np.isneginf(got), np.isneginf(rl))
    fin = np.isfinite(rl)
    assert (np.abs(got[fin] - rl[fin]) <= dz[fin] + 2.0 ** -20 + 2.0 ** -21 * np.abs(rl[fin])).all()


EDGE = [1, 2, 63, 64, 65, 127, 128, 129, 191, 192, 0, 700]


@pytest.mark.parametrize("inline", [False, True])
@pytest.mark.parametrize("h,s_q", [(1, 1), (16, 1), (16, 2), (5, 2), (17, 1), (40, 2), (128, 1), (128, 2)])
def test_parity_edge_lengths(dev, h, s_q, inline):
    causal = s_q > 1
    d = build([n if n == 0 else max(n, s_q) for n in EDGE], s_q, h, seed=h + s_q)
    out, lse = run(d, dev, causal, inline)
    check(d, out, lse, causal)
    out, lse = run(d, dev, causal, inline, fp32=True)
    check(d, out, lse, causal)


@pytest.mark.parametrize("num_sms", [1, 2, 7, 148])
@pytest.mark.parametrize("h", [16, 33])
def test_parity_any_number_of_ranges(dev, num_sms, h):
    d = build([1500, 64, 3001, 1, 260], 2, h, seed=num_sms, peaked=True)
    out, lse = run(d, dev, True, num_sms % 2 == 0, num_sms, fp32=True)
    check(d, out, lse, True)


@pytest.mark.parametrize("B,h", [(3100, 16), (3100, 20), (24600, 2)])
def test_large_batches(dev, B, h):
    """More requests than the plan's small scratch holds, and than the decode kernel plans itself."""
    g = torch.Generator().manual_seed(B + h)
    lens = torch.randint(0, 200, (B,), generator=g).tolist()
    lens[0], lens[-1] = 1500, 131
    pages = [(n + 63) // 64 for n in lens]
    d = build([64 * 30], 1, 1, seed=B)  # a pool of 33 pages that all requests share
    d["q"] = torch.randn(B, 1, h, 576, generator=g).bfloat16()
    d["lens"] = torch.tensor(lens, dtype=torch.int32)
    d["bt"] = torch.randint(0, d["kv"].shape[0], (B, max(pages)), generator=g, dtype=torch.int64).to(torch.int32)
    out, lse = run(d, dev, False, True)
    pick = [0, B - 1] + torch.randperm(B, generator=g)[:200].tolist()
    part = dict(d, q=d["q"][pick], lens=d["lens"][pick], bt=d["bt"][pick])
    check(part, out[pick], lse[pick], False)
    a = run(d, dev, False, False)
    assert torch.equal(a[0], out) and torch.equal(a[1], lse)


def test_not_causal_and_shorter_than_s_q(dev):
    d = build([1, 2, 70, 0], 2, 16, seed=3)
    for causal in (True, False):  # length 1: the first query token sees nothing when causal
        out, lse = run(d, dev, causal, True, fp32=True)
        check(d, out, lse, causal)
        if causal:
            assert bool(torch.isneginf(lse[0, :, 0]).all()) and not out[0, 0].any()


@pytest.mark.parametrize("spread", [1, 4, 12])
def test_pages_of_different_scale(dev, spread):
    """Pages whose scales differ by up to 2^24: the reference scale grows along the sequence."""
    d = build([1000, 3000, 64], 1, 16, seed=spread, spread=spread, sigma=2.0 ** -spread)
    out, lse = run(d, dev, False, True, num_sms=3, fp32=True)
    check(d, out, lse, False)


def test_zero_pages_beside_others(dev):
    """Pages of zeros, written with the least scale, and with scale 0: their tokens count in
    the sum of the weights."""
    d = build([640, 640], 1, 16, seed=8)
    z = d["bt"][:, [0, 3, 9]].flatten().long()
    d["kv"].view(torch.uint8)[z] = 0
    d["scales"][z] = 2.0 ** -100
    out, lse = run(d, dev, False, True, num_sms=2, fp32=True)
    check(d, out, lse, False)
    d["scales"][z[:3]] = 0.0
    out2, lse2 = run(d, dev, False, True, num_sms=2, fp32=True)
    check(d, out2, lse2, False)


@pytest.mark.parametrize("inline", [False, True])
def test_rows_behind_the_length_may_hold_anything(dev, inline):
    """NaN bytes in unused rows, unused pages and their scales' pages: no effect, to the bit."""
    lens = [1, 65, 127, 130, 300]
    d = build(lens, 2, 16, seed=12)
    want = run(d, dev, True, inline, num_sms=4)
    used = torch.zeros(d["kv"].shape[0], 64, dtype=torch.bool)
    for b, n in enumerate(lens):
        for t in range(n):
            used[int(d["bt"][b, t // 64]), t % 64] = True
    raw = d["kv"].view(torch.uint8)
    raw[~used] = 0x7f
    d["scales"][~used.any(1)] = float("nan")
    got = run(d, dev, True, inline, num_sms=4)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    raw[~used] = 0xff
    got = run(d, dev, True, inline, num_sms=1)
    check(d, *got, True)


def test_queries_of_any_size(dev):
    """Rows of queries from tiny to large, zero rows, and rows that are not finite: only those fail."""
    d = build([500, 900], 1, 16, seed=14)
    d["q"][0] *= torch.exp2(torch.arange(-40, 8, 3).float())[:, None].bfloat16()
    d["q"][1, 0, 3] = 0
    out, lse = run(d, dev, False, True, fp32=True)
    check(d, out, lse, False)
    bad = {k: v.clone() for k, v in d.items()}
    bad["q"][1, 0, 5, 9], bad["q"][0, 0, 2, 575] = float("inf"), float("nan")
    o2, l2 = run(bad, dev, False, True, fp32=True)
    keep = torch.ones(2, 1, 16, dtype=torch.bool)
    keep[1, 0, 5] = keep[0, 0, 2] = False
    assert torch.equal(o2[keep], out[keep]) and torch.isnan(o2[~keep]).all()
    assert torch.isnan(l2[1, 5, 0]) and torch.isnan(l2[0, 2, 0])


def test_scores_that_rise_along_the_sequence(dev):
    """Every page holds a larger score than the one before: the reference moves at each step."""
    d = build([64 * 14], 1, 32, seed=15)
    k = d["kv"].float()
    k[d["bt"][0].long()] *= 0.05
    for j in range(14):
        k[int(d["bt"][0, j]), 5, 0] = d["q"][0, 0].float().mean(0) / d["q"][0, 0].float().mean(0).abs().max() * (10 + 30 * j)
    d["kv"] = k.clamp(-448, 448).to(torch.float8_e4m3fn)
    for sms in (1, 3):
        out, lse = run(d, dev, False, True, sms, fp32=True)
        check(d, out, lse, False)


@pytest.mark.parametrize("scale", [1e30, 1e34, -1e30])
def test_scores_of_any_size(dev, scale):
    """Scores near the ends of fp32: one token takes all the weight, and scores far below zero are
    still scores.  The weight 1 is exact, so the row comes out exactly but for the division."""
    d = build([3, 200, 64], 1, 16, seed=24)
    d["q"] = -d["q"].abs()
    d["kv"] = d["kv"].float().abs().to(torch.float8_e4m3fn)
    g = {k: v.to(dev) for k, v in d.items()}
    dec = ca.Q8Decoder(3, 1, 16, d["kv"].shape[0], d["bt"].shape[1], False, 2, dev, fp32_out=True, inline_plan=True)
    dec.plan(g["lens"])
    out, lse = dec(g["q"], g["kv"], g["scales"], g["bt"], g["lens"], scale)
    torch.cuda.synchronize()
    assert dec.status() == 0 and bool(torch.isfinite(lse).all())
    kv = wide(d).double()
    for b, L in enumerate([3, 200, 64]):
        k = kv[d["bt"][b, :(L + 63) // 64].long()].reshape(-1, 576)[:L]
        z = d["q"][b, 0].double() @ k.T * scale
        best, at = z.max(-1)
        assert bool(((lse[b, :, 0].cpu().double() - best).abs() <= 2.0 ** -13 * best.abs()).all())
        ref = k[at, :512]
        assert bool(((out[b, 0].cpu().double() - ref).abs() <= 2.0 ** -20 * ref.abs()).all())


def test_same_bits_again_and_on_another_stream(dev):
    d = build([5000, 3, 4097, 64], 2, 16, seed=16)
    a = run(d, dev, True, True)
    g = {k: v.to(dev) for k, v in d.items()}
    dec = ca.Q8Decoder(4, 2, 16, d["kv"].shape[0], d["bt"].shape[1], True, 0, dev, inline_plan=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dec.plan(g["lens"], s)
    for _ in range(3):
        out, lse = dec(g["q"], g["kv"], g["scales"], g["bt"], g["lens"], SCALE, stream=s)
    s.synchronize()
    assert dec.status() == 0 and torch.equal(out.cpu(), a[0]) and torch.equal(lse.cpu(), a[1])
    # two decoders on two streams at once, each with its own buffers
    dec2 = ca.Q8Decoder(4, 2, 16, d["kv"].shape[0], d["bt"].shape[1], True, 0, dev)
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    dec2.plan(g["lens"], s2)
    for _ in range(5):
        dec(g["q"], g["kv"], g["scales"], g["bt"], g["lens"], SCALE, stream=s)
        dec2(g["q"], g["kv"], g["scales"], g["bt"], g["lens"], SCALE, stream=s2)
    torch.cuda.synchronize()
    for x in (dec, dec2):
        assert x.status() == 0 and torch.equal(x.out.cpu(), a[0]) and torch.equal(x.lse.cpu(), a[1])


def test_separate_combine_and_graph(dev):
    d = build([3000, 100], 1, 16, seed=17)
    a = run(d, dev, False, False)
    g = {k: v.to(dev) for k, v in d.items()}
    dims = bd.make_dims(2, 1, 16, d["kv"].shape[0], d["bt"].shape[1], False, 148, bd.MLA_FLAG_NO_COMBINE)
    sched = torch.zeros(ca.mla_decode_q8_schedule_bytes(dims), dtype=torch.uint8, device=dev)
    ws = torch.zeros(ca.mla_decode_q8_workspace_bytes(dims), dtype=torch.uint8, device=dev)
    out, lse = torch.empty_like(a[0], device=dev), torch.empty_like(a[1], device=dev)

    def step():
        ca.mla_decode_q8_get_schedule(dims, g["lens"], sched)
        ca.mla_decode_q8_fwd(dims, sched, ws, g["q"], g["kv"], g["scales"], g["bt"], g["lens"], SCALE, out, lse)
        ca.mla_decode_q8_combine(dims, sched, ws, out, lse)

    step()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), a[0]) and torch.equal(lse.cpu(), a[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    d2 = build([2990, 101], 1, 16, seed=18)  # the same buffers, other data
    b = run(d2, dev, False, False)
    for k in d:
        g[k].copy_(d2[k])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), b[0]) and torch.equal(lse.cpu(), b[1])


def test_faults_are_reported(dev):
    d = build([300, 70], 1, 16, seed=19)
    for inline in (False, True):
        g = {k: v.to(dev) for k, v in d.items()}
        dec = ca.Q8Decoder(2, 1, 16, d["kv"].shape[0], d["bt"].shape[1], False, 2, dev, inline_plan=inline)
        for entry in (-1, d["kv"].shape[0]):
            bt = g["bt"].clone()
            bt[0, 2] = entry
            dec.plan(g["lens"])
            dec(g["q"], g["kv"], g["scales"], bt, g["lens"], SCALE)
            torch.cuda.synchronize()
            assert dec.status() == bd.MLA_STATUS_BAD_BLOCK_TABLE
        lens = torch.tensor([300, 64 * d["bt"].shape[1] + 1], dtype=torch.int32, device=dev)
        bt = torch.zeros_like(g["bt"])
        dec.plan(lens)
        dec(g["q"], g["kv"], g["scales"], bt, lens, SCALE)
        torch.cuda.synchronize()
        assert dec.status() == bd.MLA_STATUS_BAD_SEQLEN
    # a plan of the bf16 kernels, and an unwritten one
    dims = bd.make_dims(2, 1, 40, d["kv"].shape[0], d["bt"].shape[1], False, 148)
    q = torch.zeros(2, 1, 40, 576, dtype=torch.bfloat16, device=dev)
    sched = torch.zeros(1 << 16, dtype=torch.uint8, device=dev)
    ws = torch.zeros(ca.mla_decode_q8_workspace_bytes(dims), dtype=torch.uint8, device=dev)
    out, lse = torch.zeros(2, 1, 40, 512, dtype=torch.bfloat16, device=dev), torch.zeros(2, 40, 1, device=dev)
    bd.mla_decode_get_schedule(dims, g["lens"], sched)
    ca.mla_decode_q8_fwd(dims, sched, ws, q, g["kv"], g["scales"], g["bt"], g["lens"], SCALE, out, lse)
    torch.cuda.synchronize()
    assert bd.mla_decode_get_status(sched) == bd.MLA_STATUS_BAD_SCHEDULE and not out.any()


@pytest.mark.parametrize("h", [16, 32])
def test_wait_runs_out(dev, h):
    """The first pages are never loaded: the wait on them ends after its limit, the call
    reports it, and the device goes on."""
    d = build([300], 1, h, seed=20)
    g = {k: v.to(dev) for k, v in d.items()}
    dims = bd.make_dims(1, 1, h, d["kv"].shape[0], d["bt"].shape[1], False, 2, bd.MLA_FLAG_TEST_STALL)
    dec = ca.Q8Decoder(1, 1, h, d["kv"].shape[0], d["bt"].shape[1], False, 2, dev)
    dec.dims = dims
    dec.plan(g["lens"])
    dec(g["q"], g["kv"], g["scales"], g["bt"], g["lens"], SCALE)
    torch.cuda.synchronize()
    assert dec.status() == bd.MLA_STATUS_TIMEOUT
    out, lse = run(d, dev, False, False)
    check(d, out, lse, False)


def test_far_into_a_large_pool(dev):
    """Byte offsets past 2^32: the pages of the end of a 4.3 GB pool."""
    d = build([700, 64], 1, 16, seed=22)
    nb, n = 117_000, d["kv"].shape[0]
    kv = torch.empty(nb, 64, 1, 576, dtype=torch.float8_e4m3fn, device=dev)
    scales = torch.ones(nb, 1, device=dev)
    kv[-n:].copy_(d["kv"])
    scales[-n:] = d["scales"].to(dev)
    bt = torch.where(d["bt"] >= 0, d["bt"] + (nb - n), d["bt"])
    dec = ca.Q8Decoder(2, 1, 16, nb, bt.shape[1], False, 0, dev, fp32_out=True, inline_plan=True)
    lens = d["lens"].to(dev)
    dec.plan(lens)
    out, lse = dec(d["q"].to(dev), kv, scales, bt.to(dev), lens, SCALE)
    torch.cuda.synchronize()
    assert dec.status() == 0
    check(d, out.cpu(), lse.cpu(), False)


def test_long_context(dev):
    """One request of 60,000 tokens over every SM, against fp64 on the GPU."""
    g = torch.Generator(device=dev).manual_seed(1)
    L = 60_001
    nb = (L + 63) // 64
    kv = (torch.randn(nb, 64, 1, 576, generator=g, device=dev) * 64).clamp(-448, 448).to(torch.float8_e4m3fn)
    scales = torch.full((nb, 1), 2.0 ** -6, device=dev)
    bt = torch.randperm(nb, generator=torch.Generator().manual_seed(2)).int()[None].to(dev)
    lens = torch.tensor([L], dtype=torch.int32, device=dev)
    q = torch.randn(1, 1, 16, 576, generator=g, device=dev).bfloat16()
    dec = ca.Q8Decoder(1, 1, 16, nb, nb, False, 0, dev, fp32_out=True, inline_plan=True)
    dec.plan(lens)
    out, lse = dec(q, kv, scales, bt, lens, SCALE)
    k = (kv.double() * 2.0 ** -6)[bt[0].long()].view(-1, 576)[:L]
    z = q[0, 0].double() @ k.T * SCALE
    w = torch.softmax(z, -1)
    ref, M = w @ k[:, :512], w @ k[:, :512].abs()
    tol = (2.0 ** -12 + 2.0 ** -18 + 1e-4) * M + 2.0 ** -22 * L * 7 * w.amax(-1)[:, None]
    assert dec.status() == 0 and bool(((out[0, 0].double() - ref).abs() <= tol).all())
    assert float((lse[0, :, 0].double() - torch.logsumexp(z, -1)).abs().max()) <= 2e-5


def test_append_fork_decode_compact_together(dev):
    """The operators as a program uses them: prompts are written with their positions,
    one is forked, both go on by a token each, a request ends, the pool is
    packed; every decode is checked against the oracle on the cache as it is."""
    g = torch.Generator().manual_seed(30)
    B, h, nb = 5, 16, 40
    rope = ca.make_rope(scaling="yarn", factor=40.0)
    kv = torch.full((nb, 64, 1, 576), 0x7f, dtype=torch.uint8).view(torch.float8_e4m3fn).to(dev)  # nobody's pages: NaN
    scales = torch.zeros(nb, 1, device=dev)
    refs = torch.zeros(nb, dtype=torch.int32)
    bt = torch.full((B, 8), -1, dtype=torch.int32)
    new = [100, 64, 0, 200, 0]
    ids, k = torch.randperm(nb, generator=g).int(), 0
    for b, n in enumerate(new):
        p = (n + 63) // 64
        bt[b, :p] = ids[k:k + p]
        refs[ids[k:k + p].long()] = 1
        k += p
    bt, refs, lens = bt.to(dev), refs.to(dev), torch.tensor(new, dtype=torch.int32, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    dec = ca.Q8Decoder(B, 1, h, nb, 8, False, 0, dev, inline_plan=True)
    dec.plan(lens)

    def rows(n):
        return torch.randn(n, 576, generator=g).bfloat16().to(dev)

    def put(counts):
        r = rows(sum(counts))
        off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=dev)
        ca.cache_append(r[:, :512], r[:, 512:], off, bt, lens, kv, scales, rope=rope, status=status)

    def attend():
        x = torch.randn(B, h, 576, generator=g).bfloat16().to(dev)
        pos = torch.clamp(lens - 1, min=0)
        q = ca.rope_apply(x, pos, rope, offset=512)[:, None].contiguous()
        out, lse = dec(q, kv, scales, bt, lens, SCALE)
        torch.cuda.synchronize()
        assert dec.status() == 0 and int(status) == 0
        d = dict(q=q.cpu(), kv=kv.cpu(), scales=scales.cpu(), bt=bt.cpu(), lens=lens.cpu())
        live = torch.zeros(nb, 64, dtype=torch.bool)
        for b in range(B):
            for t in range(int(d["lens"][b])):
                live[int(d["bt"][b, t // 64]), t % 64] = True
        d["kv"].view(torch.uint8)[~live] = 0  # (the oracle takes no NaN)
        check(d, out.cpu(), lse.cpu(), False)
        return out.clone()

    put(new)
    attend()
    ca.cache_fork(torch.tensor([0], dtype=torch.int32, device=dev), torch.tensor([2], dtype=torch.int32, device=dev), bt, lens, refs,
                  kv, scales, status=status)
    lens[[0, 2]] += 1
    put([1, 0, 1, 0, 0])
    out = attend()
    assert not torch.equal(out[0], out[2])
    ca.cache_free(torch.tensor([3], dtype=torch.int32, device=dev), bt, lens, refs, status=status)
    before = refs.cpu()
    ca.cache_compact(bt, lens, refs, kv, scales, status=status)
    assert int((refs > 0).sum()) == int((before > 0).sum()) and not refs[int((before > 0).sum()):].any()
    attend()


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("inline", [True, False])
@pytest.mark.parametrize("s_q,h", [(1, 16), (2, 128)])
def test_absorbed_step_is_its_parts(dev, s_q, h, inline, q8):
    """A layer's step: the same bits as its parts called one by one with the device drained between
    them, three steps in a row on one stream, into caches of either form; the new rows
    are the ones the decode sees."""
    B, nb, steps = 4, 24, 3
    g = torch.Generator().manual_seed(40 + h)
    r = lambda *s: (torch.randn(*s, generator=g)).bfloat16().to(dev)  # noqa: E731
    rope = ca.make_rope(scaling="yarn", factor=40.0)
    w_uk, w_uv = r(h, 128, 512) / 11, r(h, 512, 128) / 22
    lens0 = [0, 63, 64, 200]
    bt = torch.randperm(nb, generator=g).int().view(B, 6).contiguous().to(dev)
    off = (torch.arange(B + 1, dtype=torch.int32) * s_q).to(dev)
    pools = []
    for _ in range(2):
        d = build([64], 1, 1, seed=41, spare=nb - 1)
        kv = (d["kv"] if q8 else wide(d)).to(dev)
        pools.append((kv, d["scales"].to(dev) if q8 else None))
    ins = [(r(B, s_q, h, 192), r(B * s_q, 576)) for _ in range(steps)]
    make = (lambda: ca.Q8Decoder(B, s_q, h, nb, 6, s_q > 1, 0, dev, inline_plan=inline)) if q8 else \
        (lambda: bd.MlaDecoder(B, s_q, h, nb, 6, s_q > 1, 0, dev, inline_plan=inline))
    a, b = make(), make()
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    lens = [torch.tensor([n + s_q * (i + 1) for n in lens0], dtype=torch.int32, device=dev) for i in range(steps)]
    pos = [(x[:, None] - s_q + torch.arange(s_q, device=dev, dtype=torch.int32)).flatten().contiguous() for x in lens]
    torch.cuda.synchronize()
    got = []
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for i, (q, kv) in enumerate(ins):
        a.plan(lens[i], stream)
        out, lse = ca.absorbed_mla_step(q, kv[:, :512], kv[:, 512:], pos[i], off, w_uk, w_uv, rope, bt, lens[i], *pools[0], SCALE, a,
                                        status, stream)
        with torch.cuda.stream(stream):
            got.append((out, lse.clone()))
    stream.synchronize()
    assert a.status() == 0 and int(status) == 0
    for i, (q, kv) in enumerate(ins):
        b.plan(lens[i])
        torch.cuda.synchronize()
        qr = ca.rope_apply(q.view(B * s_q, h, 192), pos[i], rope, offset=128).view(q.shape)
        torch.cuda.synchronize()
        ca.cache_append(kv[:, :512], kv[:, 512:], off, bt, lens[i], *pools[1], rope=rope)
        torch.cuda.synchronize()
        ql = bd.absorb_q(qr, w_uk)
        torch.cuda.synchronize()
        o, lse = b(ql, *(x for x in pools[1] if x is not None), bt, lens[i], SCALE)
        torch.cuda.synchronize()
        assert torch.equal(lse, got[i][1])
        assert torch.equal(bd.absorb_o(o, w_uv), got[i][0])
    assert torch.equal(pools[0][0].view(torch.uint8), pools[1][0].view(torch.uint8))
    d = dict(q=ql.cpu(), bt=bt.cpu(), lens=lens[-1].cpu())
    pool = wide(dict(kv=pools[1][0].cpu(), scales=pools[1][1].cpu())) if q8 else pools[1][0].cpu()
    ref, rl = oracle.mla_oracle_fwd(d["q"], pool, d["bt"], d["lens"], SCALE, causal=s_q > 1)
    helpers.compare(o, lse, ref, rl)


def test_plan_checks_the_lengths(dev):
    dec = ca.Q8Decoder(4, 1, 16, 8, 2, device=dev)
    ok = torch.ones(4, dtype=torch.int32, device=dev)
    dec.plan(ok)
    for bad in (ok[:3], ok.long(), ok.cpu(), torch.ones(8, dtype=torch.int32, device=dev)[::2]):
        with pytest.raises(ValueError):
            dec.plan(bad)
    torch.cuda.synchronize()
    assert dec.status() == 0


# ------------------------------------------------------------------ scales far apart
def exact(d, scale=SCALE, causal=False):
    """fp64 attention over the cache's own values, any scales: (out [rows, 512], lse [rows], a bound on an
    fp32 output, a bound on lse).  Per token t with weight w_t, page scale s_t and score error e_t:
      - its weight is rounded by 2^-12 of itself, or its product with s_t is cut off below 2^-22 of the largest
        product w s of the row; a value is at most 448 s
      - exponentials, sums, merge of splits and the division in fp32:  2^-18 M
      - e_t moves the row by e_t w_t (|v_t| + |out|): fp32 sums of the products, the query's remainder,
        and z + log2 s, its difference to the reference and the base's 4, each rounded in fp32 (in
        units of log2: 2^-24 of at most 2 (|z| + |log2 s|) + 4, four times)"""
    B, s_q, h, _ = d["q"].shape
    out, tol = torch.zeros(B, s_q, h, 512, dtype=torch.float64), torch.zeros(B, s_q, h, 512, dtype=torch.float64)
    lse, ltol = torch.full((B, s_q, h), -float("inf"), dtype=torch.float64), torch.zeros(B, s_q, h, dtype=torch.float64)
    for b in range(B):
        L = int(d["lens"][b])
        ids = d["bt"][b, :(L + 63) // 64].long()
        s = d["scales"][ids].double().repeat_interleave(64, 0)[:L, 0]
        k = d["kv"][ids].double().reshape(-1, 576)[:L] * s[:, None]
        for i in range(s_q):
            n = L - s_q + 1 + i if causal and s_q > 1 else L
            if n <= 0:
                continue
            q, kk, v = d["q"][b, i].double(), k[:n], k[:n, :512].abs()
            z = q @ kk.T * scale
            w = torch.softmax(z, -1)
            lse[b, i], out[b, i] = torch.logsumexp(z, -1), w @ kk[:, :512]
            e = abs(scale) * (1152 * 2.0 ** -24 * (q.abs() @ kk.abs().T) + 2.0 ** -21 * q.abs().amax(-1)[:, None] * kk.abs().sum(-1))
            e = e + 2.0 ** -21 * (z.abs() * 1.5 + torch.log2(s[:n]).abs() + 4)
            we = w * e
            tol[b, i] = ((2.0 ** -12 + 2.0 ** -18) * w + we) @ v + we.sum(-1)[:, None] * out[b, i].abs() + \
                (2.0 ** -22 * n * 448 * (w * s[:n]).amax(-1))[:, None] + 2.0 ** -148
            ltol[b, i] = we.sum(-1) + 2.0 ** -20 + 2.0 ** -21 * lse[b, i].abs()
    return out, lse, tol, ltol


def check64(d, out, lse, scale=SCALE, causal=False):
    ref, rl, tol, ltol = exact(d, scale, causal)
    err = (out.double() - ref).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), (~(err <= tol)).nonzero()[0].tolist())
    got = lse.double().transpose(1, 2)
    assert bool(((got == rl) | ((got - rl).abs() <= ltol)).all())


def far_page(d, pages, scale):
    """These pages (of the pool) get a scale, large latent values where no query looks, and a last
    column that brings their scores far below the others'."""
    d["q"][..., :32] = 0
    d["q"][..., 575] = 4
    g = torch.Generator().manual_seed(99)
    for p in pages:
        v = torch.zeros(64, 1, 576)
        v[..., :32] = torch.randint(-448, 449, (64, 1, 32), generator=g)
        v[..., 575] = -448
        d["kv"][p], d["scales"][p] = v.to(torch.float8_e4m3fn), scale


@pytest.mark.parametrize("h", [16, 32])
@pytest.mark.parametrize("where", [[0], [5], [3, 8]])
@pytest.mark.parametrize("k", [8, 14, 20, 30, 90])
def test_a_page_of_a_large_scale_without_weight(dev, h, where, k):
    """It takes nothing from the weights of the others, wherever it lies."""
    d = build([1000, 700], 1, h, seed=50 + k)
    far_page(d, [int(d["bt"][b, j]) for b in range(2) for j in where], 2.0 ** k)
    for sms in (1, 3):
        out, lse = run(d, dev, False, True, sms, fp32=True)
        check64(d, out, lse)


@pytest.mark.parametrize("h", [16, 32])
@pytest.mark.parametrize("e", [-140, -120, -101, -100, -98, -40, 60, 100, 119])
def test_scales_of_any_size(dev, h, e):
    """One or two scales for all pages, with queries that bring the scores back to size (up to
    2^60; beside larger scales they are 0: every token weighs the same)."""
    d = build([300, 65, 1], 1, h, seed=60)
    g = torch.Generator().manual_seed(61)
    d["scales"] = torch.exp2(torch.randint(0, 2, d["scales"].shape, generator=g).double() + e).float()
    d["kv"] = (torch.randn(d["kv"].shape, generator=g) * 32).to(torch.float8_e4m3fn)
    d["q"] = (d["q"].double() * (2.0 ** min(-5 - e, 120) if e <= 60 else 0.0)).bfloat16()
    for sms in (1, 2):
        out, lse = run(d, dev, False, True, sms, fp32=True)
        check64(d, out, lse)


@pytest.mark.parametrize("h", [16, 32])
@pytest.mark.parametrize("low", [-60, -100, -110])
@pytest.mark.parametrize("first", [True, False])
def test_weight_on_pages_of_a_small_scale(dev, h, low, first):
    """Nearly all the weight on pages far smaller than the rest, before, between and behind them: the
    sum of the weights is theirs, whatever the others' values are worth."""
    d = build([900], 1, h, seed=70)
    ids = d["bt"][0].long()
    small = ids[0::3] if first else ids[1::3]
    d["q"][..., :575] *= 2.0 ** -4
    d["q"][..., 575] = 16
    d["kv"][ids, :, :, 575] = torch.tensor(-40.0).to(torch.float8_e4m3fn)  # -46 of score, and some 10 around it
    d["kv"][small] = torch.randn(len(small), 64, 1, 576, generator=torch.Generator().manual_seed(3)).to(torch.float8_e4m3fn)
    d["scales"][ids] = 1.0
    d["scales"][small] = 2.0 ** low
    for sms in (1, 2):
        out, lse = run(d, dev, False, True, sms, fp32=True)
        check64(d, out, lse)


@pytest.mark.parametrize("h", [16, 32])
@pytest.mark.parametrize("exponent,rise,q", [(20, 5, 1), (22, 5, 1), (23, 5, 1), (24, 6, 2), (26, 8, 8), (27, 16, 8)])
def test_large_scores_that_rise_a_little(dev, h, exponent, rise, q):
    """Scores of a size at which fp32 has no room for a reference and a margin in one number.  Each is
    exact: softmax_scale is ln 2, so scores are in units of log2, and q k = 2^exponent + rise i."""
    n = 4
    d = build([128 * n], 1, h, seed=80)
    d["q"] = torch.zeros(d["q"].shape, dtype=torch.bfloat16)
    d["q"][..., 574], d["q"][..., 575] = 2.0 ** (exponent - 8), q
    kv = torch.randn(d["kv"].shape, generator=torch.Generator().manual_seed(4)) * 8
    kv[..., 512:] = 0
    kv[..., 574] = 128  # half of the score of the tokens that rise
    for i in range(n):
        row = kv[int(d["bt"][0, 2 * i]), 7 * i, 0]
        row[574], row[575] = 256, rise * i // q
    d["kv"], d["scales"] = kv.to(torch.float8_e4m3fn), torch.ones_like(d["scales"])
    k = d["kv"][d["bt"][0].long()].double().reshape(-1, 576)
    z = d["q"][0, 0].double() @ k.T
    assert sorted(z[0].tolist())[-n:] == [2.0 ** exponent + rise * i for i in range(n)]
    w = torch.softmax(z * np.log(2), -1)
    g = {x: y.to(dev) for x, y in d.items()}
    dec = ca.Q8Decoder(1, 1, h, d["kv"].shape[0], d["bt"].shape[1], False, 1, dev, fp32_out=True, inline_plan=True)
    dec.plan(g["lens"])
    out, _ = dec(g["q"], g["kv"], g["scales"], g["bt"], g["lens"], float(np.log(2)))
    torch.cuda.synchronize()
    assert dec.status() == 0
    err = (out[0, 0].cpu().double() - w @ k[:, :512]).abs()
    tol = (2.0 ** -12 + 2.0 ** -18) * (w @ k[:, :512].abs()) + 2.0 ** -22 * len(k) * 448 * w.amax(-1)[:, None]
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("q8", [True, False])
def test_absorbed_step_refuses_before_it_writes(dev, q8):
    """A call that any of its parts would refuse leaves the cache as it was."""
    B, h, nb = 2, 16, 8
    d = build([64], 1, 1, seed=45, spare=nb - 1)
    kv, scales = (d["kv"] if q8 else wide(d)).to(dev), d["scales"].to(dev) if q8 else None
    r = lambda *s: torch.randn(*s, device=dev).bfloat16()  # noqa: E731
    make = lambda cls, *a, **k: cls(B, 1, h, nb, 4, False, 0, dev, *a, **k)  # noqa: E731
    mine, other = (ca.Q8Decoder, bd.MlaDecoder) if q8 else (bd.MlaDecoder, ca.Q8Decoder)
    dec = make(mine, inline_plan=True)
    lens = torch.tensor([70, 3], dtype=torch.int32, device=dev)
    dec.plan(lens)
    good = dict(q_in=r(B, 1, h, 192), c_kv=r(B, 512), k_pe=r(B, 64), positions=lens - 1,
                new_offsets=torch.arange(B + 1, dtype=torch.int32, device=dev), w_uk=r(h, 128, 512), w_uv=r(h, 512, 128), rope=ca.make_rope(),
                block_table=torch.arange(nb, dtype=torch.int32, device=dev).view(B, 4), cache_seqlens=lens, kv_cache=kv,
                kv_scales=scales, softmax_scale=SCALE, decoder=dec)
    before, sc = kv.clone(), None if scales is None else scales.clone()
    bad = [dict(w_uk=good["w_uk"][:, :64].contiguous()), dict(w_uk=good["w_uk"].float()), dict(w_uv=good["w_uv"][:8]), dict(w_uv=good["w_uk"]),
           dict(w_uv=good["w_uv"].cpu()), dict(softmax_scale=float("inf")), dict(softmax_scale=float("nan")), dict(decoder=make(other)),
           dict(decoder=make(mine, fp32_out=True)), dict(decoder=mine(B, 1, h, nb + 1, 4, False, 0, dev)),
           dict(decoder=mine(B, 1, h, nb, 5, False, 0, dev)), dict(decoder=mine(B, 1, h + 1, nb, 4, False, 0, dev)),
           dict(q_in=good["q_in"][:1]), dict(q_in=r(B, 1, h, 256)), dict(q_in=good["q_in"].float())]
    for change in bad:
        with pytest.raises((ValueError, bd.MlaDecodeError)):
            ca.absorbed_mla_step(**dict(good, **change))
    torch.cuda.synchronize()
    assert torch.equal(kv.view(torch.uint8), before.view(torch.uint8)) and (sc is None or torch.equal(scales, sc))
    ca.absorbed_mla_step(**good)
    torch.cuda.synchronize()
    assert dec.status() == 0 and not torch.equal(kv.view(torch.uint8), before.view(torch.uint8))
