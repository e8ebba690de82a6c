"""Rotary positions on the GPU against the fp64 oracle and against differences.

Tolerance, from the arithmetic.  With r = amplitude * sqrt(a^2 + b^2) of a pair: the
angle's fraction of a turn is rounded once to fp32 (2^-25 turns, 2^-22.3 rad), sine and
cosine are within 2 units of 2^-24 each, and x cos - y sin rounds three times: below
2^-20 r in all.  The result is then rounded to its type once (half of eps)."""
import numpy as np
import pytest
import torch

from mla_decode_attention_15_b200 import _build, cache as ca
from oracle import cache as oc

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2, torch.float32: torch.finfo(torch.float32).eps / 2}
YARN = dict(scaling="yarn", factor=40.0, original_max_position=4096)


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    _build.build()
    return torch.device("cuda:0")


def _rand(shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def _check(got, x, pos, offset, interleaved=True, amplitude=1.0, transpose=False, **freq):
    """got, x: CPU tensors [T, h, W]"""
    sl = slice(offset, offset + 64)
    ref = oc.rotate(x[..., sl].double().numpy(), pos, interleaved, amplitude, transpose, **freq)
    v = x[..., sl].double().numpy()
    pair = (lambda z: z[..., 0::2] ** 2 + z[..., 1::2] ** 2) if interleaved else (lambda z: z[..., :32] ** 2 + z[..., 32:] ** 2)
    r = abs(amplitude) * np.sqrt(pair(v))
    r = np.repeat(r, 2, -1) if interleaved else np.concatenate([r, r], -1)
    tol = HALF[got.dtype] * np.abs(ref) + 2.0 ** -20 * r * (1 + HALF[got.dtype]) + 1e-38
    err = np.abs(got[..., sl].double().numpy() - ref)
    assert (err <= tol).all(), (err / tol).max()
    rest = torch.ones(x.shape[-1], dtype=torch.bool)
    rest[sl] = False
    assert torch.equal(got[..., rest], x[..., rest])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,h,W,offset", [(1, 1, 64, 0), (1, 16, 192, 128), (5, 3, 72, 8), (33, 1, 576, 512), (17, 128, 192, 128),
                                          (300, 2, 64, 0)])
def test_rope_parity(dev, dtype, interleaved, T, h, W, offset):
    x = _rand((T, h, W), dtype, 10 * T + h)
    pos = torch.randint(0, 1 << 20, (T,), generator=torch.Generator().manual_seed(T), dtype=torch.int64).to(torch.int32)
    for kw in (dict(), dict(amplitude=1.37, **YARN)):
        table = ca.make_rope(interleaved=interleaved, **kw)
        for transpose in (False, True):
            got = ca.rope_apply(x.to(dev), pos.to(dev), table, offset=offset, transpose=transpose)
            _check(got.cpu(), x, pos.tolist(), offset, interleaved, transpose=transpose, **kw)


def test_rope_extreme_positions(dev):
    """The first pair turns by one radian per token: at 2^31 - 1 the fp32 product
    alone would be 128 rad off.  Negative positions turn back."""
    pos = [0, 1, 2 ** 24 + 1, 2 ** 31 - 1, -1, -(2 ** 31)]
    x = _rand((len(pos), 2, 64), torch.float32, 3)
    got = ca.rope_apply(x.to(dev), torch.tensor(pos, dtype=torch.int64).to(torch.int32).to(dev), ca.make_rope())
    # 2^31 radians in turns: 2^28.4, of which 53 bits keep 2^-25 turns
    _check(got.cpu(), x, pos, 0)


@pytest.mark.parametrize("interleaved", [True, False])
def test_rope_strides_in_place_and_guard(dev, interleaved):
    """Rows of a wider projection, heads before tokens, in place: the columns around
    the rotated ones, and the rows and columns between the strided ones, stay."""
    T, h, W = 9, 4, 192
    table = ca.make_rope(interleaved=interleaved)
    pos = torch.arange(T, dtype=torch.int32) * 17
    wide = _rand((T, h + 1, W + 16), torch.bfloat16, 5)
    for perm in (False, True):
        buf = (wide.transpose(0, 1).contiguous().transpose(0, 1) if perm else wide.clone()).to(dev)
        buf = buf if perm else buf.contiguous()
        view = buf[:, :h, 8:8 + W]
        before = buf.cpu().clone()
        ref = ca.rope_apply(view, pos.to(dev), table, offset=128)
        _check(ref.cpu(), view.cpu(), pos.tolist(), 128, interleaved)
        assert torch.equal(buf.cpu(), before)
        got = ca.rope_apply(view, pos.to(dev), table, offset=128, out=view)
        assert got is view and torch.equal(view.cpu(), ref.cpu())
        after = buf.cpu()
        after[:, :h, 8:8 + W] = before[:, :h, 8:8 + W]
        assert torch.equal(after, before)


def test_rope_two_dimensions_empty_and_special(dev):
    table = ca.make_rope()
    x = _rand((7, 576), torch.bfloat16, 8)
    pos = torch.arange(7, dtype=torch.int32)
    got = ca.rope_apply(x.to(dev), pos.to(dev), table, offset=512).cpu()
    _check(got[:, None], x[:, None], pos.tolist(), 512)
    assert ca.rope_apply(x[:0].to(dev), pos[:0].to(dev), table).shape == (0, 576)
    y = x.float()
    y[2, 512], y[3, 513] = float("inf"), float("nan")
    z = ca.rope_apply(y.to(dev), pos.to(dev), table, offset=512).cpu()
    bad = ~torch.isfinite(z)
    want = torch.zeros_like(bad)
    want[2, 512:514] = want[3, 512:514] = True  # only the pairs they belong to
    assert torch.equal(bad, want)


def test_rope_gradient(dev):
    """The transposed call is the gradient: against the inner product, and against
    central differences of a scalar of the result (the map is linear, so the
    difference is exact up to fp32 rounding of values of size ~1)."""
    x, g = _rand((6, 3, 128), torch.float32, 1).to(dev), _rand((6, 3, 128), torch.float32, 2).to(dev)
    pos = torch.arange(6, dtype=torch.int32, device=dev) * 1000
    for inter in (True, False):
        table = ca.make_rope(interleaved=inter, amplitude=1.2, **YARN)
        dx = ca.rope_apply(g, pos, table, offset=32, transpose=True)
        y = ca.rope_apply(x, pos, table, offset=32)
        a, b = (y.double() * g.double()).sum(), (x.double() * dx.double()).sum()
        assert abs(float(a - b)) <= 2.0 ** -19 * float((y.double() * g.double()).abs().sum())
        for at in ((0, 0, 5), (2, 1, 33), (5, 2, 64), (4, 0, 95), (3, 1, 100)):
            e = torch.zeros_like(x)
            e[at] = 0.5
            diff = ca.rope_apply(x + e, pos, table, offset=32).double() - ca.rope_apply(x - e, pos, table, offset=32).double()
            assert abs(float((diff * g.double()).sum()) - float(dx[at])) <= 64 * 2.0 ** -22 * 20


def test_rope_stream_and_graph(dev):
    table = ca.make_rope()
    x, pos = _rand((40, 16, 192), torch.bfloat16, 4).to(dev), torch.arange(40, dtype=torch.int32, device=dev)
    ref = ca.rope_apply(x, pos, table, offset=128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(x)
    ca.rope_apply(x, pos, table, offset=128, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g):
        ca.rope_apply(x, pos, table, offset=128, out=out)
    x.copy_(x.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ca.rope_apply(x, pos, table, offset=128))


def test_result_of_another_stream_is_not_shared(dev):
    """Memory freed on the current stream, with work on it still queued, is not the result of a
    call on another stream."""
    table = ca.make_rope()
    x, pos = _rand((64, 16, 192), torch.bfloat16, 6).to(dev), torch.arange(64, dtype=torch.int32, device=dev)
    ref = ca.rope_apply(x, pos, table, offset=128)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = torch.empty_like(x)
    torch.cuda._sleep(20_000_000)
    old.fill_(7.0)
    del old
    got = ca.rope_apply(x, pos, table, offset=128, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, ref)
    with pytest.raises(ValueError):
        ca.rope_apply(x, pos, table, offset=128, stream=s.cuda_stream)
    ca.rope_apply(x, pos, table, offset=128, out=got, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(got, ref)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("transpose", [False, True])
def test_rope_small_sines_and_cosines(dev, interleaved, transpose):
    """A unit vector comes out as the cosine and the sine, each right to its own size: two units in the
    last place of the functions (2^-22), half a unit each for the remainder of the angle and the product
    with 1 (2^-23 in all), and the angle itself, a 53-bit product on either side (below 2^-50 of the
    position, in radians)."""
    T = 20_000
    pos = torch.randint(0, 1 << 20, (T,), generator=torch.Generator().manual_seed(77), dtype=torch.int64)
    x = torch.zeros(T, 1, 64)
    first = torch.arange(0, 64, 2) if interleaved else torch.arange(32)
    second = first + (1 if interleaved else 32)
    x[..., first] = 1
    got = ca.rope_apply(x.to(dev), pos.to(torch.int32).to(dev), ca.make_rope(interleaved=interleaved), transpose=transpose)
    got = got.cpu().double().numpy()[:, 0]
    f = oc.frequencies()
    ang = np.fmod(pos.numpy()[:, None].astype(np.float64) * f, 2 * np.pi)
    for cols, ref in ((first, np.cos(ang)), (second, np.sin(-ang if transpose else ang))):
        err = np.abs(got[:, cols.numpy()] - ref)
        tol = (2.0 ** -22 + 2.0 ** -23) * np.abs(ref) + 2.0 ** -50 * pos.numpy()[:, None]
        assert (err <= tol).all(), float((err / tol).max())
