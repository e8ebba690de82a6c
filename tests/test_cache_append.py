"""The write of new rows into the paged cache against the fp64 oracle.

Tolerance: latent columns are bf16 already, so a bf16 cache holds them bit for bit, and an
e4m3 cache holds exactly the nearest e4m3 value of x / scale (a power of two: the
quotient is exact).  RoPE columns carry the fp32 rotation's error, below 2^-20 of the
pair's length (tests/test_rope.py), before their one rounding: they are within half
a step of their type plus that."""
import numpy as np
import pytest
import torch

from mla_decode_attention_15_b200 import _build, binding as bd, cache as ca
from oracle import cache as oc

pytestmark = pytest.mark.gpu
ROPE = dict(scaling="yarn", factor=40.0, original_max_position=4096)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    _build.build()
    return torch.device("cuda:0")


def _make(ctx, new, q8, seed, sigma=1.0, spare=3):
    """A pool holding ctx rows per request (from earlier rows of size sigma), then new ones."""
    g = torch.Generator().manual_seed(seed)
    B = len(ctx)
    lens = [c + n for c, n in zip(ctx, new)]
    pages = [oc.pages_of(n) for n in lens]
    nb, width = sum(pages) + spare, max(max(pages), 1) + 1
    ids = torch.randperm(nb, generator=g).int()
    bt = torch.full((B, width), -1, dtype=torch.int32)
    k = 0
    for b, p in enumerate(pages):
        bt[b, :p] = ids[k:k + p]
        k += p
    off = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32)
    rows = (torch.randn(sum(new), 576, generator=g) * 3).bfloat16()
    pool = torch.randn(nb, 64, 1, 576, generator=g) * sigma
    if q8:
        scales = torch.tensor([oc.scale_of(float(p.abs().max())) for p in pool]).float()[:, None]
        pool = (pool / scales[:, :, None, None]).to(torch.float8_e4m3fn)
    else:
        scales, pool = None, pool.bfloat16()
    return dict(rows=rows, off=off, bt=bt, lens=torch.tensor(lens, dtype=torch.int32), pool=pool, scales=scales)


def _run(d, dev, rope, status=True):
    g = {k: v.to(dev) if v is not None else None for k, v in d.items()}
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    ca.cache_append(g["rows"][:, :512], g["rows"][:, 512:], g["off"], g["bt"], g["lens"], g["pool"], g["scales"], rope=rope,
                    status=st if status else None)
    torch.cuda.synchronize()
    return g["pool"].cpu(), None if d["scales"] is None else g["scales"].cpu(), int(st)


def _check(d, pool, scales, rope):
    q8 = scales is not None
    want = d["pool"].double().numpy()[:, :, 0].copy()
    ws = d["scales"].double().numpy()[:, 0].copy() if q8 else None
    seen = oc.append(d["rows"][:, :512].double().numpy(), d["rows"][:, 512:].double().numpy(), d["off"].tolist(), d["bt"].tolist(),
                     d["lens"].tolist(), want, ws, rope)
    got = pool.double().numpy()[:, :, 0]
    if q8:
        np.testing.assert_array_equal(scales.double().numpy()[:, 0], ws)
    # everything but the new rows' RoPE columns is exact
    mask = np.zeros(got.shape, dtype=bool)
    for phys, (first, x) in seen.items():
        mask[phys, first:first + len(x), 512:] = rope is not None
    np.testing.assert_array_equal(got[~mask], want[~mask])
    if rope is None:
        return
    inter = rope.get("interleaved", True)
    for phys, (first, x) in seen.items():
        s = ws[phys] if q8 else 1.0
        pe = x[:, 512:]
        r = np.sqrt(pe[:, 0::2] ** 2 + pe[:, 1::2] ** 2) if inter else np.sqrt(pe[:, :32] ** 2 + pe[:, 32:] ** 2)
        r = np.repeat(r, 2, -1) if inter else np.concatenate([r, r], -1)
        half = np.maximum(2.0 ** -4 * np.abs(pe), 2.0 ** -10 * s) if q8 else 2.0 ** -8 * np.abs(pe)
        err = np.abs(got[phys, first:first + len(x), 512:] * s - pe)
        assert (err <= half * (1 + 2.0 ** -15) + 2.0 ** -19 * r).all()


CASES = [([0], [1]), ([63], [1]), ([64], [1]), ([62], [2]), ([63], [2]), ([0], [64]), ([1], [64]), ([5], [129]), ([0, 10, 64], [0, 3, 0]),
         ([0, 63, 64, 1, 200], [200, 1, 2, 130, 5]), ([7] * 300, [1] * 300), ([30, 0], [0, 0])]


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("layout", [None, True, False])
@pytest.mark.parametrize("ctx,new", CASES, ids=lambda v: "x".join(map(str, v[:5])))
def test_append_parity(dev, ctx, new, layout, q8):
    d = _make(ctx, new, q8, seed=sum(ctx) + 3 * sum(new))
    rope = None if layout is None else dict(interleaved=layout, **ROPE)
    pool, scales, st = _run(d, dev, None if rope is None else ca.make_rope(**rope))
    assert st == 0
    _check(d, pool, scales, rope)


@pytest.mark.parametrize("sigma", [1e-4, 1.0, 30.0, 1e6])
def test_append_page_scale_grows_or_stays(dev, sigma):
    """Earlier rows far smaller than, like, and far larger than the new ones."""
    d = _make([10, 63, 100], [5, 2, 64], True, seed=int(sigma) + 1, sigma=sigma)
    pool, scales, st = _run(d, dev, None)
    assert st == 0
    _check(d, pool, scales, None)


def test_append_one_by_one_matches_definition(dev):
    """130 single rows of falling and rising size: each step against the oracle, started from the
    GPU's own cache, so each page's scale follows the rows it has held."""
    g = torch.Generator().manual_seed(5)
    amp = torch.exp2(torch.randint(-12, 12, (130, 1), generator=g).float())
    rows = (torch.randn(130, 576, generator=g) * amp).bfloat16()
    nb = 4
    pool = torch.zeros(nb, 64, 1, 576).to(torch.float8_e4m3fn).to(dev)
    scales = torch.zeros(nb, 1, device=dev)  # what a fresh pool holds is not looked at
    bt = torch.tensor([[2, 0, 3]], dtype=torch.int32)
    want, ws = np.zeros((nb, 64, 576)), np.zeros(nb)
    off = torch.tensor([0, 1], dtype=torch.int32)
    for t in range(130):
        ca.cache_append(rows[t:t + 1, :512].to(dev), rows[t:t + 1, 512:].to(dev), off.to(dev), bt.to(dev),
                        torch.tensor([t + 1], dtype=torch.int32, device=dev), pool, scales)
        oc.append(rows[t:t + 1, :512].double().numpy(), rows[t:t + 1, 512:].double().numpy(), [0, 1], bt.tolist(), [t + 1], want, ws)
    np.testing.assert_array_equal(pool.cpu().double().numpy()[:, :, 0], want)
    np.testing.assert_array_equal(scales.cpu().double().numpy()[:, 0], ws)
    # and no value is further off than two roundings at its page's scale
    for t in range(130):
        s = ws[[2, 0, 3][t // 64]]
        x = rows[t].double().numpy()
        err = np.abs(want[[2, 0, 3][t // 64], t % 64] * s - x)
        assert (err <= 2.0 ** -4 * np.abs(x) + 2 * 2.0 ** -10 * s).all()


def test_append_special_values(dev):
    d = _make([3, 0, 0], [2, 1, 3], True, seed=9)
    d["rows"][0, 7], d["rows"][0, 520], d["rows"][1, 3] = float("inf"), float("nan"), -float("inf")
    d["rows"][2] = 0.0                       # a page of zeros
    d["rows"][3:] = 3e38                     # the top of bf16's range
    d["rows"][4] = 1e-38
    pool, scales, st = _run(d, dev, None)
    assert st == 0
    _check(d, pool, scales, None)
    b1 = int(d["bt"][1, 0])
    assert float(scales[b1]) == 2.0 ** -100 and not pool[b1, 0].float().any()


def test_append_refuses_bad_requests(dev):
    """A request whose rows do not fit, or whose page is outside the pool, is left
    out with a status word; the others are written."""
    for q8 in (True, False):
        good = _make([5, 6, 7, 8], [2, 3, 66, 1], q8, seed=21)
        ref, rs, st = _run(good, dev, None)
        assert st == 0
        for change, word in (("len", ca.MLA_STATUS_BAD_ROW), ("far", ca.MLA_STATUS_BAD_ROW), ("neg", ca.MLA_STATUS_BAD_ROW),
                             ("page", bd.MLA_STATUS_BAD_BLOCK_TABLE), ("page2", bd.MLA_STATUS_BAD_BLOCK_TABLE)):
            d = {k: None if v is None else v.clone() for k, v in good.items()}
            if change == "len":
                d["lens"][1] = 2
            elif change == "far":
                d["lens"][1] = 64 * d["bt"].shape[1] + 1
            elif change == "neg":
                d["lens"][1] = -3
            else:
                d["bt"][1, 0] = -1 if change == "page" else d["pool"].shape[0]
            pool, scales, st = _run(d, dev, None)
            assert st == word, change
            page = int(good["bt"][1, 0])
            keep = torch.arange(pool.shape[0]) != page
            assert torch.equal(pool.view(torch.uint8)[keep], ref.view(torch.uint8)[keep]), change
            assert torch.equal(pool.view(torch.uint8)[page], good["pool"].view(torch.uint8)[page])
        d = {k: None if v is None else v.clone() for k, v in good.items()}
        d["off"][4] = 1000  # past the rows
        pool, _, st = _run(d, dev, None)
        assert st == ca.MLA_STATUS_BAD_ROW
        d["off"][4], d["off"][3] = 72, 80  # falling
        assert _run(d, dev, None)[2] == ca.MLA_STATUS_BAD_ROW


def test_append_far_into_a_large_pool(dev):
    """Byte offsets past 2^32: the pool's last pages."""
    nb = 117_000  # 4.3 GB
    pool = torch.empty(nb, 64, 1, 576, dtype=torch.float8_e4m3fn, device=dev)
    scales = torch.ones(nb, 1, device=dev)
    tail = pool[-4:].view(torch.uint8)
    tail.zero_()
    rows = torch.randn(70, 576, generator=torch.Generator().manual_seed(2)).bfloat16()
    bt = torch.tensor([[nb - 3, nb - 1]], dtype=torch.int32)
    ca.cache_append(rows[:, :512].to(dev), rows[:, 512:].to(dev), torch.tensor([0, 70], dtype=torch.int32, device=dev), bt.to(dev),
                    torch.tensor([70], dtype=torch.int32, device=dev), pool, scales)
    want, ws = np.zeros((4, 64, 576)), np.ones(4)
    oc.append(rows[:, :512].double().numpy(), rows[:, 512:].double().numpy(), [0, 70], [[1, 3]], [70], want, ws)
    np.testing.assert_array_equal(pool[-4:].cpu().double().numpy()[:, :, 0], want)
    np.testing.assert_array_equal(scales[-4:].cpu().double().numpy()[:, 0], ws)


def test_append_stream_and_graph(dev):
    d = _make([5, 64, 0], [3, 1, 70], True, seed=33)
    ref, rs, _ = _run(d, dev, ca.make_rope(**ROPE))
    g = {k: v.to(dev) for k, v in d.items()}
    rope = ca.make_rope(**ROPE)
    call = lambda stream=None: ca.cache_append(g["rows"][:, :512], g["rows"][:, 512:], g["off"], g["bt"], g["lens"], g["pool"],  # noqa: E731
                                               g["scales"], rope=rope, stream=stream)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    s.synchronize()
    assert torch.equal(g["pool"].cpu().view(torch.uint8), ref.view(torch.uint8)) and torch.equal(g["scales"].cpu(), rs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    g["pool"].copy_(d["pool"])
    g["scales"].copy_(d["scales"])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(g["pool"].cpu().view(torch.uint8), ref.view(torch.uint8)) and torch.equal(g["scales"].cpu(), rs)


@pytest.mark.parametrize("q8", [True, False])
@pytest.mark.parametrize("B,T", [(3, 2000), (4, 190), (601, 64)])
def test_append_with_falling_offsets(dev, B, T, q8):
    """Offsets 0, T, 0, T, ...: every second request is refused, and the others, which name the same rows, are
    written whole, although together they have more pages than T rows of requests in order."""
    d = _make([70] * B, [T] + [0] * (B - 1), q8, seed=B)
    good = list(range(0, B, 2))
    pages = oc.pages_of(70 + T)
    nb = pages * len(good) + 1
    g = torch.Generator().manual_seed(B + 1)
    d["bt"] = torch.full((B, pages), -1, dtype=torch.int32)
    d["bt"][good] = torch.randperm(nb, generator=g)[1:].int().view(len(good), pages)
    d["off"] = torch.tensor([0, T] * ((B + 2) // 2), dtype=torch.int32)[:B + 1]
    d["lens"] = torch.full((B,), 70 + T, dtype=torch.int32)
    d["pool"] = torch.zeros(nb, 64, 1, 576, dtype=torch.float8_e4m3fn if q8 else torch.bfloat16)
    d["scales"] = torch.ones(nb, 1) if q8 else None
    pool, scales, st = _run(d, dev, None)
    assert st == (ca.MLA_STATUS_BAD_ROW if B > 1 else 0)
    _check(d, pool, scales, None)  # (the oracle leaves out what falls)
