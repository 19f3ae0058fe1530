"""Grouped routing and the 4-bit operators on buffers of more than 2^31 elements:
the last rows of a large call are those of a small call on the same rows."""
import pytest
import torch

import top_routing_expert_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
FAR = 1 << 31


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.load_library()
    yield
    torch.cuda.empty_cache()


def test_routing_and_gradient():
    E, k, n = 250, 6, 1000                       # rows without vectors of four
    T = FAR // E + 2 * n
    g = torch.Generator(device=DEV).manual_seed(1)
    tail = torch.randn(n, E, generator=g, device=DEV)
    tail[::5] = torch.round(tail[::5] * 2) / 2   # ties
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    cfg = moe.RouteConfig.make("sigmoid", n_groups=5, topk_groups=3, group_top=1, scale=2.0)
    logits = torch.zeros(T, E, device=DEV)
    logits[-n:] = tail
    out = []
    for x in (logits, tail):
        s = moe.MoeShape.make(x.shape[0], 64, E, k, 64, 1.0)
        idx = torch.full((x.shape[0], k), -1, dtype=torch.int32, device=DEV)
        w = torch.zeros(x.shape[0], k, device=DEV)
        moe.moe_route_grouped(s, cfg, x, bias, idx, w, ws=moe.Workspace(s))
        gw = torch.ones_like(w) * torch.arange(k, device=DEV)
        routed = torch.ones(E, dtype=torch.int32, device=DEV)
        grad = torch.full_like(x, 9.0)
        moe.moe_route_grouped_bwd(s, cfg, x, idx, gw, grad, grad_aux=torch.zeros(1, device=DEV), routed_counts=routed)
        out.append([t[-n:].clone() for t in (idx, w, grad)])
        del idx, w, gw, grad
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_rows_and_product():
    K, N, n = 65536, 64, 300
    rows = FAR // K + n
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    x[-n:] = torch.randn(n, K, generator=g, device=DEV).to(torch.bfloat16)

    def packed(r, k):
        return (torch.empty(r, k // 2, dtype=torch.uint8, device=DEV),
                torch.empty((k + 127) // 128, r, 4, dtype=torch.uint8, device=DEV))

    q, s = packed(rows, K)
    moe.moe_quantize_rows_mx4(x, q, s)
    q2, s2 = packed(n, K)
    moe.moe_quantize_rows_mx4(x[-n:].contiguous(), q2, s2)
    assert torch.equal(q[-n:], q2) and torch.equal(s[:, -n:], s2)
    x.fill_(9.0)
    moe.moe_dequantize_rows_mx4(q, s, x)
    back = torch.empty(n, K, dtype=torch.bfloat16, device=DEV)
    moe.moe_dequantize_rows_mx4(q2, s2, back)
    assert torch.equal(x[-n:], back) and x[0].abs().max() == 0
    del x, q, s, back
    # a product of more than 2^31 outputs, the last expert's rows at its end
    K, N = 128, 65536
    rows = FAR // N + n
    a = torch.randn(n, K, generator=g, device=DEV).to(torch.bfloat16)
    W = torch.randn(2, K, N, generator=g, device=DEV).to(torch.bfloat16)
    w_q = torch.empty(2, N, K // 2, dtype=torch.uint8, device=DEV)
    w_s = torch.empty(2, N // 128, 1, 32, 4, 4, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_weights_mx4(W, w_q, w_s)
    full = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    full[-n:] = a
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = []
    for src, off in ((full, [0, rows - n, rows]), (a, [0, 0, n])):
        q, s = packed(src.shape[0], K)
        moe.moe_quantize_rows_mx4(src, q, s)
        out = torch.full((src.shape[0], N), 9.0, dtype=torch.bfloat16, device=DEV)
        moe.moe_expert_gemm_mx4(q, s, torch.tensor(off, dtype=torch.int32, device=DEV), w_q, w_s, out, dev_status=status)
        outs.append(out[-n:].clone())
        if src is full:
            assert out[:-n].abs().max() == 0
        del out
    assert torch.equal(*outs) and status.item() == 0
