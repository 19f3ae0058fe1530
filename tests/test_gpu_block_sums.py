"""Gradients that are sums over all tokens (of the two norms' weights), where many
partial sums are joined.

A group of threads adds up its tokens; there are G groups, of which a GB300 holds 152
(one to an SM) to 2432 (four to a block, four blocks to an SM, the most that the
workspace has rows for). Their sums are added in eight slices, and the slices in turn: a
value passes T / G + 1 + G / 8 + 8 additions at most, so T / 152 + 313, of 2^-24 of the
terms' magnitudes A each. The terms' own error is below 2^-15 A: three sums of fewer
than 64 additions feed one, with roots and products of a few 2^-23."""
import numpy as np
import pytest
import torch

import top_routing_expert_gb300 as moe
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("T,H", [(2501, 192), (2433, 64), (9727, 256), (9729, 512), (20001, 128),
                                 (3001, 1024), (1825, 2048)])
@pytest.mark.parametrize("post_norm", [True, False])
def test_sums_over_tokens(T, H, post_norm):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.load_library()
    g = torch.Generator().manual_seed(T)
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)
    h, y, g_out, g_xn = bf(T, H), bf(2 * T, H), bf(T, H), bf(T, H)
    dest = torch.randperm(2 * T, generator=g).to(torch.int32).view(T, 2)
    dest[torch.rand(T, 2, generator=g) < 0.1] = -1
    w, gate = torch.rand(T, 2, generator=g), torch.randn(T, generator=g)
    post, pre = torch.randn(H, generator=g), torch.randn(H, generator=g)
    got = [torch.full((H,), 7.0, device=DEV) for _ in range(2)]
    d = [t.to(DEV) for t in (h, y, g_out, g_xn, dest, w, post, gate, pre)]
    moe.moe_block_norm_bwd(moe.BlockConfig.make(post_norm=post_norm, residual_scale=0.75, eps=1e-5),
                           d[0], d[1], d[2], None, None, grad_xn=d[3], dest_row=d[4], topk_w=d[5],
                           post_weight=d[6], gate=d[7], pre_weight=d[8], grad_post=got[0],
                           grad_pre=got[1], ws=moe.BlockWorkspace(T, H))
    f = lambda t: t.float().numpy().astype(np.float64)
    args = (f(h), f(y), dest.numpy(), f(w), f(post), f(gate), f(pre), post_norm, 0.75, 1e-5, f(g_out),
            f(g_xn))
    want, size = O.block_norm_grad(*args), O.block_norm_grad_magnitude(*args)
    for n, t in zip(("g_post", "g_pre"), got):
        err = np.abs(t.cpu().numpy().astype(np.float64) - want[n])
        tol = 2.0 ** -24 * np.abs(want[n]) + (2.0 ** -15 + 2.0 ** -24 * (T / 152 + 313)) * size[n]
        assert (err <= tol).all(), (n, (err / tol).max())
