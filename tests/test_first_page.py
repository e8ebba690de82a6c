"""The decode kernel's first page, issued before its wait on the grid before it."""
import pytest
import torch

from mla_decode_attention_15_b200 import _build, binding as bd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    _build.build()
    bd.lib()
    return torch.device("cuda:0")


def test_first_page_done_before_the_producer_starts(dev):
    """The page that is issued with the plan may be used up while the producer is still
    issuing Q and prefetches: no wait of its stage may be a phase late (a wait that runs out
    takes a second and sets the status).  A late producer is a matter of chance, so many steps
    with long items, and every step's result the same."""
    B, blocks = 16, 256
    g = torch.Generator().manual_seed(7)
    q = torch.randn(B, 1, 16, 576, generator=g).bfloat16().to(dev)
    kv = torch.randn(B * blocks, 64, 1, 576, generator=g).bfloat16().to(dev)
    bt = torch.randperm(B * blocks, generator=g).int().view(B, blocks).contiguous().to(dev)
    sl = torch.full((B,), blocks * 64, dtype=torch.int32, device=dev)
    dec = bd.MlaDecoder(B, 1, 16, B * blocks, blocks, False, 0, dev, inline_plan=True)
    dec.plan(sl)
    out, lse = (x.clone() for x in dec(q, kv, bt, sl, 576 ** -0.5))
    for _ in range(100):
        for _ in range(50):
            o, l = dec(q, kv, bt, sl, 576 ** -0.5)
        torch.cuda.synchronize()
        assert dec.status() == 0
        assert torch.equal(o, out) and torch.equal(l, lse)
