"""Sums over several gradients in a block's training step."""
import pytest
import torch

import top_routing_expert_gb300 as moe
from top_routing_expert_gb300.block import BlockWeights, TrainBlock

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.load_library()


def _make(T, H, E, k, h, cf, seed, bias=True):
    g = torch.Generator().manual_seed(seed)
    bf = lambda *n, std=1.0: (std * torch.randn(n, generator=g)).to(torch.bfloat16).to(DEV)
    f32 = lambda *n: torch.randn(n, generator=g).to(DEV)
    w = BlockWeights(bf(E, H, h, std=H ** -0.5), bf(E, h, H, std=h ** -0.5), bf(H, E, std=H ** -0.5),
                     1 + 0.2 * f32(H), 1 + 0.2 * f32(H), 0.5 * f32(E) if bias else None)
    block = TrainBlock(moe.MoeShape.make(T, H, E, k, h, cf), moe.RouteConfig.make("sigmoid"),
                       moe.BlockConfig.make())
    batches = [{n: bf(T, H) for n in ("h", "xn", "g_out", "g_xn")} for _ in range(2)]
    return block, w, batches


def _step(block, w, d, grads, next_norm=True, **kw):
    out, xn, gh, gx = (torch.empty_like(d["h"]) for _ in range(4))
    block.forward(d["h"], d["xn"], w, out, xn if next_norm else None)
    block.backward(d["g_out"], d["g_xn"] if next_norm else None, gh, gx, grads,
                   grad_aux=torch.full((1,), 0.3, device=DEV), **kw)
    return gh, gx


SHAPES = [(300, 128, 8, 2, 192, 4.0), (257, 256, 12, 3, 128, 0.75), (1, 64, 4, 2, 64, 4.0),
          (1000, 192, 64, 8, 64, 1.0)]


@pytest.mark.parametrize("shape", SHAPES)
def test_gradient_of_the_input_is_rounded_once(shape):
    """Its terms are the router's part and up to k rows, all bf16: fp32 additions of
    k + 1 terms, 2^-24 of their magnitudes each, and half a step of bf16."""
    block, w, (d, _) = _make(*shape, seed=shape[0])
    _, gx = _step(block, w, d, BlockWeights.zeros_like(w))
    dest, k = block.dest_row.long(), shape[3]
    rows, ref = block.g_x.double(), block.g_router.double()
    size = ref.abs()
    for j in range(k):
        kept = (dest[:, j] >= 0)[:, None]
        term = torch.where(kept, rows[dest[:, j].clamp(min=0)], 0.0)
        ref, size = ref + term, size + term.abs()
    err = (gx.double() - ref).abs()
    assert (err <= 2.0 ** -8 * ref.abs() + (k + 1) * 2.0 ** -24 * size).all()


NAMES = ("W1", "W2", "gate", "post", "pre", "gate_bias")


def _grads(w):
    return {n: getattr(w, n) for n in NAMES if getattr(w, n) is not None}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("next_norm", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_every_gradient_accumulates(shape, next_norm, bias):
    """Two micro-batches, and three from a replayed graph: sums of fp32 values in the
    batches' order, to the bit. (The products' gradients are added as whole sums.)"""
    block, w, batches = _make(*shape, seed=5, bias=bias)
    each = []
    for d in batches:
        g = BlockWeights.zeros_like(w)
        for t in _grads(g).values():
            t.fill_(3)                                     # written, not added
        _step(block, w, d, g, next_norm)
        each.append(_grads(g))
    total = BlockWeights.zeros_like(w)
    for d in batches:
        _step(block, w, d, total, next_norm, accumulate="all")
    for n, t in _grads(total).items():
        assert torch.equal(t, each[0][n] + each[1][n]), n
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _step(block, w, batches[0], total, next_norm, accumulate="all")
    want = {n: t.clone() for n, t in _grads(total).items()}
    for _ in range(2):
        graph.replay()
        for n, t in _grads(total).items():
            want[n] += each[0][n]
            assert torch.equal(t, want[n]), n


def test_accumulate_with_no_tokens_and_refusals():
    block, w, _ = _make(0, 128, 4, 2, 64, 1.0, seed=1)
    e = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    grads = BlockWeights.zeros_like(w)
    for t in _grads(grads).values():
        t.fill_(3)
    block.forward(e, e, w, e, e)
    block.backward(e, e, e, e, grads, accumulate="all")
    assert all((t == 3).all() for t in _grads(grads).values())
    for bad in ("some", None, 2):
        with pytest.raises(ValueError):
            block.backward(e, e, e, e, grads, accumulate=bad)
    block.backward(e, e, e, e, grads, accumulate=True)
    assert (grads.W1 == 3).all() and (grads.post == 0).all()
