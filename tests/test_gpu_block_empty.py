"""A block whose output buffer has no rows (every slot dropped) between two blocks:
the forward passes the residual, and the gradient is that of tokens whose slots are
all dropped, which a buffer with rows gives too."""
import pytest
import torch

import top_routing_expert_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.load_library()


@pytest.mark.parametrize("T,H,k", [(1, 64, 1), (6, 256, 2), (9, 1024, 8), (40, 4096, 2), (3, 8256, 6)])
@pytest.mark.parametrize("post_norm", [True, False])
@pytest.mark.parametrize("given", ["both", "out", "xn"])
def test_no_rows(T, H, k, post_norm, given):
    g = torch.Generator().manual_seed(T + H)
    bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16).to(DEV)
    f32 = lambda *s: torch.randn(s, generator=g).to(DEV)
    cfg = moe.BlockConfig.make(post_norm=post_norm, residual_scale=0.5)
    h, g_out, g_xn = bf(T, H), bf(T, H), bf(T, H)
    post, gate, pre = f32(H), f32(T), f32(H)
    # as many slots as there may be: rows outside the buffer are no rows either
    dest = torch.randint(-3, 3, (T, k), generator=g, dtype=torch.int32).to(DEV)
    w = torch.full((T, k), float("nan"), device=DEV)

    def grad(y, dest):
        o = {"residual": torch.full((T, H), 7.0, dtype=torch.bfloat16, device=DEV),
             "w": torch.full((T, k), 7.0, device=DEV), "post": torch.full((H,), 7.0, device=DEV),
             "gate": torch.full((T,), 7.0, device=DEV),
             "pre": torch.full((H,), 7.0, device=DEV) if given != "out" else None}
        moe.moe_block_norm_bwd(cfg, h, y, g_out if given != "xn" else None, o["residual"],
                               torch.empty_like(y), grad_xn=g_xn if given != "out" else None,
                               dest_row=dest, topk_w=w, post_weight=post, gate=gate, pre_weight=pre,
                               grad_topk_w=o["w"], grad_post=o["post"], grad_gate=o["gate"],
                               grad_pre=o["pre"], ws=moe.BlockWorkspace(T, H))
        return o

    empty = grad(torch.empty(0, H, dtype=torch.bfloat16, device=DEV), dest)
    for n in ("w", "post", "gate"):
        assert (empty[n] == 0).all(), n
    dropped = grad(torch.full((5, H), float("nan"), dtype=torch.bfloat16, device=DEV),
                   torch.full_like(dest, -1))
    for n, t in dropped.items():
        assert t is None or torch.equal(t, empty[n]), n
    with pytest.raises(moe.MoeError):      # no block output at all has no such gradients
        moe.moe_block_norm_bwd(cfg, h, None, g_out, None, None, dest_row=dest, grad_topk_w=empty["w"])
