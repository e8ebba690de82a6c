"""The operators around a paged latent cache: rotary positions, the write of new
rows (bf16, or e4m3 with one scale per page), attention over the 8-bit cache, and
the fork, free and compaction of its pages.

``run`` computes each in its plain form (elementary torch operations in 32 bits, 64
for angles) or, with ``own``, by the framework's calls.  The shapes are those of
the absorbed-MLA decode: rows of 576 (512 latent + 64 RoPE), pages of 64 tokens,
16 or 128 heads, one or two new tokens per request.
"""
import math

import torch

own = False

PAGE, D_QK, D_V, D_ROPE, D_IN, ROPE_AT = 64, 576, 512, 64, 192, 128
SCALE = 192 ** -0.5
E4M3 = torch.float8_e4m3fn
E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -100, 119  # exponents of a page scale
YARN = dict(theta=10000.0, scaling="yarn", factor=40.0, original_max_position=4096, beta_fast=32.0, beta_slow=1.0,
            amplitude=1.0)
PLAIN_ROPE = dict(theta=10000.0, scaling="none", factor=1.0, original_max_position=4096, beta_fast=32.0, beta_slow=1.0,
                  amplitude=1.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the RoPE part of one decode step's queries: 16 requests x 16 heads, far positions
        dict(name="rope_decode_t16_h16", op="rope", tokens=16, heads=16, layout="interleaved", scaling="yarn",
             transpose=False, dtype="bf16", top=65536),
        # a prompt's queries for 128 heads, half layout, the gradient's direction
        dict(name="rope_prompt_grad_t4099_h128", op="rope", tokens=4099, heads=128, layout="half", scaling="none",
             transpose=True, dtype="bf16", top=16384),
        # one new row for each of 128 running requests, 8-bit cache: pages that already hold rows
        dict(name="append_decode_e4m3_b128", op="append", batch=128, new_lo=1, new_hi=1, ctx_lo=63, ctx_hi=4096,
             dtype="e4m3", layout="interleaved", scaling="yarn"),
        # prompts and chunks of prompts of every length into the 8-bit cache
        dict(name="append_prompt_e4m3_b16", op="append", batch=16, new_lo=17, new_hi=4099, ctx_lo=0, ctx_hi=900,
             dtype="e4m3", layout="interleaved", scaling="yarn"),
        # attention: the smallest decode step, where latency counts
        dict(name="attend_b1_l1024_h16", op="attend", batch=1, s_q=1, heads=16, lo=1024, hi=1024, sigma=1.0, peaked=False),
        # two-token decode over ragged contexts with a few dominant rows
        dict(name="attend_b16_sq2_1k16k_h16", op="attend", batch=16, s_q=2, heads=16, lo=1025, hi=16383, sigma=1.0,
             peaked=True),
        # the long-context decode of the headline benchmark
        dict(name="attend_b16_l65536_h16", op="attend", batch=16, s_q=1, heads=16, lo=65536, hi=65536, sigma=1.0,
             peaked=False),
        # two-token decode with every head on one GPU: bound by arithmetic
        dict(name="attend_b32_sq2_8k32k_h128", op="attend", batch=32, s_q=2, heads=128, lo=8192, hi=32768, sigma=0.5,
             peaked=False),
        # parallel sampling: every prompt forks three continuations
        dict(name="fork_e4m3_p8_x3", op="fork", parents=8, times=3, lo=100, hi=5000, dtype="e4m3"),
        dict(name="fork_bf16_p64_x3", op="fork", parents=64, times=3, lo=1000, hi=9000, dtype="bf16"),
        # requests that ended leave holes: free them, then pack the pool
        dict(name="compact_e4m3_b64", op="compact", batch=64, ended=24, lo=1000, hi=20000, dtype="e4m3"),
        dict(name="compact_bf16_b16", op="compact", batch=16, ended=9, lo=64, hi=4096, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "fork", "compact"])
    layout, scaling = rng.choice(["interleaved", "half"]), rng.choice(["none", "yarn"])
    if op == "rope":
        tokens = _log(rng, 1, 4099)
        return dict(op=op, tokens=tokens, heads=_log(rng, 1, 128), layout=layout, scaling=scaling,
                    transpose=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "fp32"]) if tokens < 2000 else "bf16",
                    top=_log(rng, 4096, 1 << 20))
    if op == "append":
        batch = _log(rng, 1, 128)
        hi = _log(rng, 1, max(1, 32000 // batch))
        return dict(op=op, batch=batch, new_lo=rng.randint(1, hi), new_hi=hi, ctx_lo=rng.randint(0, 64),
                    ctx_hi=_log(rng, 64, 4096), dtype=rng.choice(["e4m3", "e4m3", "bf16"]), layout=layout, scaling=scaling)
    if op == "attend":
        s_q, batch, heads = rng.choice([1, 1, 2]), _log(rng, 1, 48), _log(rng, 1, 128)
        hi = _log(rng, 2, min(65536, (1 << 20) // batch, 160_000_000 // (batch * heads * s_q)))
        return dict(op=op, batch=batch, s_q=s_q, heads=heads, lo=rng.randint(min(2, hi), hi), hi=hi,
                    sigma=rng.choice([0.5, 1.0]), peaked=rng.random() < 0.3)
    if op == "fork":
        parents = _log(rng, 1, 64)
        return dict(op=op, parents=parents, times=rng.randint(1, 3), lo=rng.randint(1, 100), hi=_log(rng, 101, 9000),
                    dtype=rng.choice(["e4m3", "bf16"]))
    batch = _log(rng, 2, 64)
    return dict(op=op, batch=batch, ended=rng.randint(1, batch - 1), lo=rng.randint(1, 1000), hi=_log(rng, 1001, 10000),
                dtype=rng.choice(["e4m3", "bf16"]))


# ------------------------------------------------------------------ inputs
def _spread(lo, hi, n):
    """n whole numbers from lo to hi in even steps: a case has the same total for every seed."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]


def _pages(n):
    return -(-n // PAGE)


def _exp_of(amax):
    """The least e with amax <= 448 * 2^e, within the exponents a scale may have."""
    m, e = torch.frexp(amax / E4M3_MAX)
    e = torch.where(m == 0.5, e - 1, e)
    return torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(MIN_EXP, MAX_EXP)


def _pow2(e):
    return torch.ldexp(torch.ones((), device=e.device), e)


class _Rand:
    """Draws of one seed: the GPU's generator for values, the CPU's for bookkeeping."""

    def __init__(self, seed):
        self.host = torch.Generator().manual_seed(seed)
        self.gpu = torch.Generator(device="cuda").manual_seed(seed)

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.gpu, device="cuda")

    def perm(self, n):
        return torch.randperm(n, generator=self.host)

    def ints(self, lo, hi, n):
        return torch.randint(lo, hi, (n,), generator=self.host)


def _pool(r, num_blocks, dtype, sigma=1.0):
    """A pool of filled pages, as the write of normal rows leaves it, and its page scales."""
    if dtype == "bf16":
        kv = torch.empty(num_blocks, PAGE, 1, D_QK, dtype=torch.bfloat16, device="cuda")
        for part in kv.split(4096):
            part.copy_(r.normal(*part.shape) * sigma)
        return kv, None
    kv = torch.empty(num_blocks, PAGE, 1, D_QK, dtype=E4M3, device="cuda")
    scales = torch.empty(num_blocks, 1, device="cuda")
    for part, sc in zip(kv.split(4096), scales.split(4096)):
        _quantise(r.normal(*part.shape) * sigma, part, sc)
    return kv, scales


def _quantise(x, part, sc):
    s = _pow2(_exp_of(x.abs().amax(dim=(1, 2, 3))))
    part.copy_((x / s[:, None, None, None]).to(E4M3))
    sc.copy_(s[:, None])


def _table(r, lens, num_blocks, rows=None, width=None):
    """Pages dealt at random to the requests; unused entries -1."""
    rows = rows or len(lens)
    width = width or max(1, max(_pages(n) for n in lens))
    ids = r.perm(num_blocks).to(torch.int32)
    bt = torch.full((rows, width), -1, dtype=torch.int32)
    k = 0
    for b, n in enumerate(lens):
        bt[b, :_pages(n)] = ids[k:k + _pages(n)]
        k += _pages(n)
    return bt


def prepare(case, seed):
    r = _Rand(seed)
    s = dict(case)
    op = case["op"]
    if op == "rope":
        dtype = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        s["x"] = r.normal(case["tokens"], case["heads"], D_IN).to(dtype)
        s["positions"] = r.ints(0, case["top"], case["tokens"]).to(torch.int32).cuda()
        s["out"] = torch.empty_like(s["x"])
    elif op == "append":
        order = r.perm(case["batch"]).tolist()
        new = _spread(case["new_lo"], case["new_hi"], case["batch"])
        ctx = [_spread(case["ctx_lo"], case["ctx_hi"], case["batch"])[i] for i in order]
        lens = [a + b for a, b in zip(ctx, new)]
        num_blocks = sum(_pages(n) for n in ctx) + sum(_pages(n) for n in new) + 8
        s["kv"], s["scales"] = _pool(r, num_blocks, case["dtype"])
        s["bt"] = _table(r, lens, num_blocks).cuda()
        s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
        off = [0]
        for n in new:
            off.append(off[-1] + n)
        s["off"] = torch.tensor(off, dtype=torch.int32).cuda()
        # one projection's output: 512 latent columns, then the 64 of the RoPE key
        rows = (r.normal(off[-1], D_QK) * 1.5).to(torch.bfloat16)
        s["c_kv"], s["k_pe"] = rows[:, :D_V], rows[:, D_V:]
        s["tokens"], s["touched"] = off[-1], max((n + PAGE - 2) // PAGE + 1 for n in new)
    elif op == "attend":
        lens = _attend_lens(case)
        lens = [lens[i] for i in r.perm(len(lens)).tolist()]
        num_blocks = sum(_pages(n) for n in lens) + 8
        bt = _table(r, lens, num_blocks)
        s["q"] = (r.normal(case["batch"], case["s_q"], case["heads"], D_QK) * case["sigma"]).to(torch.bfloat16)
        s["kv"] = torch.empty(num_blocks, PAGE, 1, D_QK, dtype=E4M3, device="cuda")
        s["scales"] = torch.empty(num_blocks, 1, device="cuda")
        for part, sc in zip(s["kv"].split(4096), s["scales"].split(4096)):
            x = r.normal(*part.shape) * case["sigma"]
            if case["peaked"]:  # one row in a hundred is eight times the others
                x *= 1 + 7 * (torch.rand(x.shape[:3], generator=r.gpu, device="cuda") < 0.01)[..., None]
            _quantise(x, part, sc)
        s["bt"], s["lens"] = bt.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        if own:  # the decoder a program keeps for a shape of batch: plan and workspace buffers
            from mla_decode_attention_15_b200 import Q8Decoder
            s["decoder"] = Q8Decoder(case["batch"], case["s_q"], case["heads"], num_blocks, bt.shape[1],
                                     causal=case["s_q"] > 1, device=torch.device("cuda"), inline_plan=True)
            s["decoder"].plan(s["lens"])
    elif op == "fork":
        lens = _spread(case["lo"], case["hi"], case["parents"])
        lens = [lens[i] for i in r.perm(len(lens)).tolist()]
        children = case["parents"] * case["times"]
        num_blocks = sum(_pages(n) for n in lens) + children + 8
        bt = _table(r, lens, num_blocks, rows=case["parents"] + children, width=max(_pages(n) for n in lens) + 4)
        s["kv"], s["scales"] = _pool(r, num_blocks, case["dtype"])
        _books(s, bt, lens, num_blocks)
        s["src"] = torch.arange(children, dtype=torch.int32).remainder(case["parents"]).cuda()
        s["dst"] = (case["parents"] + r.perm(children)).to(torch.int32).cuda()
    else:
        lens = _spread(case["lo"], case["hi"], case["batch"])
        lens = [lens[i] for i in r.perm(len(lens)).tolist()]
        num_blocks = sum(_pages(n) for n in lens) + 8
        s["kv"], s["scales"] = _pool(r, num_blocks, case["dtype"])
        bt = _table(r, lens, num_blocks)
        _books(s, bt, lens, num_blocks)
        rows = r.perm(case["batch"])[:case["ended"]]
        s["rows"] = rows.to(torch.int32).cuda()
        # a program that keeps its books on the host too knows how many pages stay, and how many of them move
        stay = bt.index_fill(0, rows, -1)
        stay = stay[stay >= 0]
        s["left"] = stay.numel()
        s["moves"] = int((stay >= stay.numel()).sum())
    return s


def _books(s, bt, lens, num_blocks):
    refs = torch.zeros(num_blocks, dtype=torch.int32)
    refs[bt[bt >= 0].long()] = 1
    full = torch.zeros(bt.shape[0], dtype=torch.int32)
    full[:len(lens)] = torch.tensor(lens, dtype=torch.int32)
    s["bt0"], s["lens0"], s["refs0"] = bt.cuda(), full.cuda(), refs.cuda()
    s["bt"], s["lens"], s["refs"] = s["bt0"].clone(), s["lens0"].clone(), s["refs0"].clone()


def _attend_lens(case):
    return [max(n, case["s_q"]) for n in _spread(case["lo"], case["hi"], case["batch"])]


# ------------------------------------------------------------------ runs
def _rope_config(layout, scaling):
    return dict(YARN if scaling == "yarn" else PLAIN_ROPE, interleaved=layout == "interleaved")


def run(s):
    return {"rope": _rope, "append": _append, "attend": _attend, "fork": _fork, "compact": _compact}[s["op"]](s)


def _inv_freq(cfg, device):
    i = torch.arange(D_ROPE // 2, dtype=torch.float64, device=device)
    f = torch.exp(-(2 * i / D_ROPE) * math.log(cfg["theta"]))
    if cfg["scaling"] == "yarn":
        at = [D_ROPE * math.log(cfg["original_max_position"] / (b * 2 * math.pi)) / (2 * math.log(cfg["theta"]))
              for b in (cfg["beta_fast"], cfg["beta_slow"])]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), D_ROPE - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / cfg["factor"] * ramp
    return f


def _rotate(x, positions, cfg, transpose=False):
    """Rotates the last 64 columns of x [T, ..., 64] in 32 bits, angles in 64."""
    angle = positions.double()[:, None] * _inv_freq(cfg, x.device)
    cos, sin = (angle.cos() * cfg["amplitude"]).float(), (angle.sin() * cfg["amplitude"]).float()
    if transpose:
        sin = -sin
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (D_ROPE // 2,)
    cos, sin, x = cos.view(shape), sin.view(shape), x.float()
    if cfg["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    a, b = x[..., :D_ROPE // 2], x[..., D_ROPE // 2:]
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1)


def _rope(s):
    cfg = _rope_config(s["layout"], s["scaling"])
    if own:
        from mla_decode_attention_15_b200 import make_rope, rope_apply
        if "rope" not in s:
            s["rope"] = make_rope(**cfg)
        return rope_apply(s["x"], s["positions"], s["rope"], offset=ROPE_AT, out=s["out"], transpose=s["transpose"])
    y = s["out"]
    y.copy_(s["x"])
    y[..., ROPE_AT:] = _rotate(s["x"][..., ROPE_AT:], s["positions"], cfg, s["transpose"]).to(y.dtype)
    return y


def _append(s):
    cfg = _rope_config(s["layout"], s["scaling"])
    kv, scales = s["kv"], s["scales"]
    if own:
        from mla_decode_attention_15_b200 import cache_append, make_rope
        if "rope" not in s:
            s["rope"] = make_rope(**cfg)
        cache_append(s["c_kv"], s["k_pe"], s["off"], s["bt"], s["lens"], kv, scales, rope=s["rope"])
        return (kv, scales) if scales is not None else kv
    lens, off, bt = s["lens"].long(), s["off"].long(), s["bt"].long()
    n = off[1:] - off[:-1]
    start = lens - n
    t = torch.arange(s["tokens"], device="cuda")
    b = torch.searchsorted(off[1:], t, right=True)
    pos = start[b] + t - off[b]
    rows = torch.cat((s["c_kv"].float(), _rotate(s["k_pe"], pos, cfg)), -1)
    phys, slot = bt[b, pos // PAGE], pos % PAGE
    if scales is None:
        kv[phys, slot, 0] = rows.to(kv.dtype)
        return kv
    # pages that the call touches: [request, j]
    first = start // PAGE
    page = first[:, None] + torch.arange(s["touched"], device="cuda")
    hit = page * PAGE < lens[:, None]
    ids = bt.gather(1, page.clamp(max=bt.shape[1] - 1))
    amax = torch.zeros(ids.shape, device="cuda")
    amax.view(-1).scatter_reduce_(0, b * s["touched"] + pos // PAGE - first[b], rows.abs().amax(-1), "amax")
    new = _pow2(_exp_of(amax))
    # the first page of a request may hold rows already: it keeps the larger scale, and they are rescaled
    held = start % PAGE
    old = scales[ids[:, 0], 0]
    new[:, 0] = torch.where(held > 0, torch.maximum(old, new[:, 0]), new[:, 0])
    raw = kv.view(torch.uint8)
    before = raw[ids[:, 0], :, 0]
    again = (before.view(E4M3).float() * (old / new[:, 0])[:, None, None]).to(E4M3).view(torch.uint8)
    keep = torch.arange(PAGE, device="cuda")[None, :, None] < held[:, None, None]
    raw[ids[:, 0], :, 0] = torch.where(keep, again, before)
    mine = new[b, pos // PAGE - first[b]]
    raw[phys, slot, 0] = (rows / mine[:, None]).to(E4M3).view(torch.uint8)
    # (a place of no page repeats its request's first page and scale)
    ids, new = torch.where(hit, ids, ids[:, :1]), torch.where(hit, new, new[:, :1])
    scales[ids.flatten(), 0] = new.flatten()
    return kv, scales


def _attend(s):
    q, kv, scales, bt, lens = s["q"], s["kv"], s["scales"], s["bt"], s["lens"]
    if own:
        return s["decoder"](q, kv, scales, bt, lens, SCALE)
    B, s_q, h, _ = q.shape
    ids = bt.clamp(min=0).long()
    rows = kv.view(torch.uint8)[ids].view(E4M3).float() * scales[ids][..., None, None]
    rows = rows.view(B, -1, D_QK)
    z = torch.bmm(q.float().view(B, s_q * h, D_QK), rows.transpose(1, 2)) * SCALE
    z = z.view(B, s_q, h, -1)
    seen = lens[:, None] - s_q + 1 + torch.arange(s_q, device="cuda") if s_q > 1 else lens[:, None]
    z.masked_fill_(torch.arange(z.shape[-1], device="cuda") >= seen[:, :, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m)
    l = p.sum(-1, keepdim=True)
    out = torch.bmm((p / l).view(B, s_q * h, -1), rows[..., :D_V]).view(B, s_q, h, D_V)
    return out.to(torch.bfloat16), (m + torch.log(l)).squeeze(-1).transpose(1, 2).contiguous()


def _reset(s):
    """The books as they were before the call: a program's own copy of them."""
    for k in ("bt", "lens", "refs"):
        s[k].copy_(s[k + "0"])
    return s["bt"], s["lens"], s["refs"]


def _state(s):
    pool = (s["kv"],) if s["scales"] is None else (s["kv"], s["scales"])
    return (s["bt"], s["lens"], s["refs"]) + pool


def _fork(s):
    bt, lens, refs = _reset(s)
    kv, scales, src, dst = s["kv"], s["scales"], s["src"].long(), s["dst"].long()
    if own:
        from mla_decode_attention_15_b200 import cache_fork
        cache_fork(s["src"], s["dst"], bt, lens, refs, kv, scales)
        return _state(s)
    L = lens[src].long()
    part, last = L % PAGE > 0, L // PAGE
    # the k-th fork that ends inside a page takes the k-th free page
    order = torch.sort((refs > 0).to(torch.int8), stable=True).indices
    fresh = order[(part.cumsum(0) - 1).clamp(min=0)]
    rows = bt[src]
    used = torch.arange(bt.shape[1], device="cuda")[None] < -(-L // PAGE)[:, None]
    whole = torch.arange(bt.shape[1], device="cuda")[None] < last[:, None]
    old = rows.gather(1, last.clamp(max=bt.shape[1] - 1)[:, None])[:, 0].long()
    mine = torch.where(used, rows, bt[dst])
    mine = torch.where(used & ~whole, fresh[:, None].to(torch.int32), mine)
    refs.index_add_(0, rows.clamp(min=0).long().flatten(), whole.flatten().to(torch.int32))
    refs.index_add_(0, fresh, part.to(torch.int32))
    bt[dst] = mine
    lens[dst] = L.to(torch.int32)
    # a fork that ends on a page's border copies nothing: its source onto itself
    old = torch.where(part, old, rows[:, 0].long())
    to = torch.where(part, fresh, old)
    raw = kv.view(torch.uint8)
    raw[to] = raw[old]
    if scales is not None:
        scales[to] = scales[old]
    return _state(s)


def _compact(s):
    bt, lens, refs = _reset(s)
    kv, scales, rows = s["kv"], s["scales"], s["rows"].long()
    if own:
        from mla_decode_attention_15_b200 import cache_compact, cache_free
        cache_free(s["rows"], bt, lens, refs)
        if "compact_space" not in s:
            from mla_decode_attention_15_b200 import cache_compact_workspace
            s["compact_space"] = cache_compact_workspace(kv.shape[0], kv.device)
        cache_compact(bt, lens, refs, kv, scales, workspace=s["compact_space"])
        return _state(s)
    place = torch.arange(bt.shape[1], device="cuda")[None]
    used = place < -(-lens[:, None] // PAGE)
    gone = used[rows]
    refs.index_add_(0, bt[rows].clamp(min=0).long().flatten(), -gone.flatten().to(torch.int32))
    bt[rows] = torch.where(gone, -1, bt[rows])
    lens[rows] = 0
    # the k-th live page behind the first `left` goes to the k-th free one among them
    live, at = refs > 0, torch.arange(refs.shape[0], device="cuda")
    low = at < s["left"]
    dst = torch.sort((live | ~low).to(torch.int8), stable=True).indices[:s["moves"]]
    src = torch.sort((~live | low).to(torch.int8), stable=True).indices[:s["moves"]]
    raw = kv.view(torch.uint8)
    raw[dst] = raw[src]
    if scales is not None:
        scales[dst] = scales[src]
    to = at.clone()
    to[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    used = place < -(-lens[:, None] // PAGE)
    bt.copy_(torch.where(used, to[bt.clamp(min=0).long()].to(torch.int32), bt))
    return _state(s)


# ------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "rope":
        size = 4 if case["dtype"] == "fp32" else 2
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * D_IN * size + 4 * case["tokens"], "flops": 3 * n * D_ROPE}
    if op == "append":
        t = sum(_spread(case["new_lo"], case["new_hi"], case["batch"]))
        return {"bytes": t * D_QK * (2 + (1 if case["dtype"] == "e4m3" else 2)) + 12 * case["batch"], "flops": 6 * t * D_ROPE}
    if op == "attend":
        t, n = sum(_attend_lens(case)), case["heads"] * case["s_q"]
        return {"bytes": t * D_QK + 8 * _pages(t) + case["batch"] * n * (2 * (D_QK + D_V) + 4),
                "flops": 2 * n * t * (D_QK + D_V)}
    page = PAGE * D_QK * (1 if case["dtype"] == "e4m3" else 2)
    if op == "fork":
        lens = _spread(case["lo"], case["hi"], case["parents"])
        copies = case["times"] * sum(n % PAGE > 0 for n in lens)
        return {"bytes": 2 * page * copies + 16 * case["times"] * sum(_pages(n) for n in lens), "flops": 0}
    lens = _spread(case["lo"], case["hi"], case["batch"])
    total = sum(_pages(n) for n in lens)
    left = total * (case["batch"] - case["ended"]) // case["batch"]
    # in a shuffled pool a live page sits behind the border with the share of the pool that lies there
    moves = left * (total + 8 - left) // (total + 8)
    return {"bytes": 2 * page * moves + 16 * total, "flops": 0}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The same from the definitions in 64 bits, a request or a token at a time.  Moves of pages compute no numbers."""
    if case["op"] not in ("rope", "append", "attend"):
        return None
    global own
    held, own = own, False
    s = prepare(case, seed)
    own = held
    return {"rope": _exact_rope, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)


def _exact_turn(x, positions, cfg, transpose=False):
    """x [T, H, 64] as complex numbers, turned by pos * f in 64 bits."""
    f = torch.tensor([cfg["theta"] ** (-2.0 * i / D_ROPE) for i in range(D_ROPE // 2)], dtype=torch.float64)
    if cfg["scaling"] == "yarn":
        turns = lambda b: D_ROPE * math.log(cfg["original_max_position"] / (2 * math.pi * b)) / (2 * math.log(cfg["theta"]))  # noqa: E731
        low, high = max(0, math.floor(turns(cfg["beta_fast"]))), min(D_ROPE - 1, math.ceil(turns(cfg["beta_slow"])))
        for i in range(D_ROPE // 2):
            w = min(1.0, max(0.0, (i - low) / max(high - low, 0.001)))
            f[i] = f[i] / cfg["factor"] * w + f[i] * (1 - w)
    angle = positions.double()[:, None] * f.to(x.device)
    turn = torch.polar(torch.full_like(angle, cfg["amplitude"]), -angle if transpose else angle)[:, None]
    half = D_ROPE // 2
    pairs = x.double().unflatten(-1, (half, 2)) if cfg["interleaved"] else x.double().unflatten(-1, (2, half)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    return (y if cfg["interleaved"] else y.transpose(-1, -2)).flatten(-2)


def _exact_rope(s):
    y = s["x"].double()
    y[..., ROPE_AT:] = _exact_turn(s["x"][..., ROPE_AT:], s["positions"], _rope_config(s["layout"], s["scaling"]), s["transpose"])
    return y


def _exact_append(s):
    cfg = _rope_config(s["layout"], s["scaling"])
    off, lens, kv = s["off"].tolist(), s["lens"].tolist(), s["kv"].double()
    scales = None if s["scales"] is None else s["scales"].double()
    for b, L in enumerate(lens):
        lo, hi = off[b], off[b + 1]
        at = torch.arange(L - (hi - lo), L, device="cuda")
        turned = _exact_turn(s["k_pe"][lo:hi, None], at, cfg)[:, 0]
        rows = torch.cat((s["c_kv"][lo:hi].double(), turned), -1)
        for page in range((L - (hi - lo)) // PAGE, _pages(L)):
            mine = (at // PAGE) == page
            x, slots, phys = rows[mine], at[mine] % PAGE, int(s["bt"][b, page])
            if scales is None:
                kv[phys, slots, 0] = x
                continue
            amax, first = float(x.abs().max()), int(slots[0])
            e = MIN_EXP if amax == 0 else max(MIN_EXP, min(MAX_EXP, math.ceil(math.log2(amax / E4M3_MAX))))
            scale = max(2.0 ** e, float(scales[phys]) if first > 0 else 0.0)
            kv[phys, :first, 0] = (kv[phys, :first, 0] * (float(scales[phys]) / scale)).to(E4M3).double()
            kv[phys, slots, 0] = (x / scale).to(E4M3).double()
            scales[phys] = scale
    return kv if scales is None else (kv, scales)


def _exact_attend(s):
    q, lens = s["q"].double(), s["lens"].tolist()
    B, s_q, h, _ = q.shape
    out = torch.zeros(B, s_q, h, D_V, dtype=torch.float64, device="cuda")
    lse = torch.full((B, h, s_q), -math.inf, dtype=torch.float64, device="cuda")
    for b, L in enumerate(lens):
        ids = s["bt"][b, :_pages(L)].long()
        k = s["kv"].view(torch.uint8)[ids].view(E4M3).double() * s["scales"][ids].double()[:, :, None, None]
        k = k.view(-1, D_QK)
        for i in range(s_q):
            n = L - s_q + 1 + i
            if n > 0:
                z = q[b, i] @ k[:n].T * SCALE
                lse[b, :, i] = torch.logsumexp(z, -1)
                out[b, i] = torch.exp(z - lse[b, :, i, None]) @ k[:n, :D_V]
    return out, lse
