"""The step between two blocks with out in the residual's place."""
import os
import re

import pytest
import torch

import top_routing_expert_gb300 as moe

CSRC = os.path.join(os.path.dirname(moe.__file__), "csrc")


def test_residual_is_not_read_as_read_only():
    """The read-only path (__ldg) promises that nothing writes the memory while the
    kernel runs; the results do not show a broken promise, so the source is asked."""
    with open(os.path.join(CSRC, "moe_block.cu")) as f:
        text = f.read()
    assert "a.residual" in text
    assert not re.search(r"__ldg\([^;]*a\.residual", text)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,k", [(9001, 64, 1), (5000, 512, 8), (4001, 2048, 6), (3001, 4096, 2),
                                   (700, 16384, 2)])
@pytest.mark.parametrize("experts", [True, False])
def test_in_place(T, H, k, experts):
    """Many tokens to a block of threads, the next one's rows asked for while this one
    is written: the same bits as with a buffer of its own, also in a replayed graph."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.load_library()
    g = torch.Generator(device="cuda").manual_seed(T)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    k = k if experts else 1
    first, y = bf(T, H), bf(T * k, H)
    dest = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k) if experts else None
    w = torch.rand(T, k, generator=g, device="cuda") if experts else None
    cfg = moe.BlockConfig.make(residual_scale=0.5)
    step = lambda res, out, xn: moe.moe_block_norm(cfg, res, y, out, xn=xn, dest_row=dest, topk_w=w)
    one, two, xn1, xn2 = (torch.empty_like(first) for _ in range(4))
    step(first, one, xn1)
    step(one, two, xn2)
    h, xn = first.clone(), torch.empty_like(first)
    step(h, h, xn)
    assert torch.equal(h, one) and torch.equal(xn, xn1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(h, h, xn)
    h.copy_(first)
    for want, want_xn in ((one, xn1), (two, xn2)):
        graph.replay()
        assert torch.equal(h, want) and torch.equal(xn, want_xn)
