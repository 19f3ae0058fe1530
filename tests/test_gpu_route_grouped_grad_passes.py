"""The routing gradient over batches that take a warp several passes, where rows
in shared memory are used again and the next tokens' rows are fetched ahead,
against the float64 oracle.

A gradient is a sum of products of factors that are each within (48 + 4 spread) u
of themselves (u = 2^-24, spread the largest difference of logits): the same share
of the largest magnitudes that enter it."""
import numpy as np
import pytest
import torch

import top_routing_expert_gb300 as moe
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.load_library()


# a pass is 38912 tokens of up to 32 experts, 19456 of up to 64, ... 4864 of 256;
# rows of a multiple of four experts are written in vectors, others one by one
@pytest.mark.parametrize("T,E,k", [(40003, 16, 2), (120011, 15, 3), (90007, 30, 5), (60007, 33, 8),
                                   (60001, 64, 8), (31013, 102, 4), (10007, 256, 8), (15013, 255, 7)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_over_several_passes(T, E, k, score):
    rng = np.random.default_rng(E)
    l = rng.standard_normal((T, E)).astype(np.float32)
    idx = np.argsort(-l, axis=1, kind="stable")[:, :k].astype(np.int32)
    gw = rng.standard_normal((T, k)).astype(np.float32)
    routed = np.bincount(idx.ravel(), minlength=E).astype(np.int32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    x, i, g, r = dev(l), dev(idx), dev(gw), dev(routed)
    s = moe.MoeShape.make(T, 64, E, k, 64, 1.0)
    spread = 2 * float(np.abs(l).max())
    for renorm in (True, False):
        for aux in (None, 0.25 * T):
            ga = None if aux is None else torch.full((1,), aux, device=DEV)
            grad = torch.full((T, E), float("nan"), device=DEV)
            call = lambda: moe.moe_route_grouped_bwd(
                s, moe.RouteConfig.make(score, renormalize=renorm, scale=1.5), x, i, g, grad, grad_aux=ga,
                routed_counts=None if aux is None else r)
            call()
            mine = grad.cpu().numpy()
            call()
            assert np.array_equal(mine, grad.cpu().numpy())
            ref = O.route_grouped_grad(l.astype(np.float64), idx, gw.astype(np.float64), score, renorm, 1.5,
                                       0.0 if aux is None else aux, None if aux is None else routed)
            size = 1.5 * np.abs(gw).max() + (0.0 if aux is None else aux * E / T * routed.max() / (T * k))
            assert np.abs(mine - ref).max() <= 2 * (48 + 4 * spread) * U * size
