"""The training products past 2^31 elements: rows and weights at the far end of
buffers of more than 4 GB, with values whose products are exact."""
import pytest
import torch

import top_routing_expert_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    moe.build()
    moe.load_library()


def _small(g, *n):
    """Whole numbers from -2 to 2: their sums of products are exact in fp32."""
    return torch.randint(-2, 3, n, generator=g, device=DEV).to(torch.bfloat16)


@pytest.mark.parametrize("transposed", [False, True])
def test_rows_past_2_31(transposed):
    g = torch.Generator(device=DEV).manual_seed(1)
    K, N = 64, 16384
    rows = (1 << 31) // N + 400                    # the last rows of out and pre lie past 2^31
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
    x[-300:] = _small(g, 300, K)
    W = _small(g, 2, *((N, K) if transposed else (K, N)))
    offsets = torch.tensor([rows - 300, rows - 170, rows], dtype=torch.int32, device=DEV)
    out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=DEV)
    pre = torch.full_like(out, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_expert_gemm(x, offsets, W, out, transposed=transposed, epilogue="gelu", pre=pre,
                        dev_status=status)
    for e, (lo, hi) in enumerate(((rows - 300, rows - 170), (rows - 170, rows))):
        w = W[e].float().T if transposed else W[e].float()
        ref = x[lo:hi].float() @ w
        assert torch.equal(pre[lo:hi], ref.to(torch.bfloat16))
    assert (pre[-310:-300] == 7).all() and (out[:4] == 7).all() and (out[-301] == 7).all()
    # the slope at 64 is 1; at -64 it is what it is at -7, where u is held: with s =
    # exp(-35.6) = 3.5e-16, 7 s (1.6 + 0.214 * 49) - s = 3e-14 < 2^-44 of the product
    pre[-300:] = 64
    pre[-1] = -64
    moe.moe_expert_gemm(x, offsets, W, out, transposed=transposed, epilogue="gelu_grad", pre=pre,
                        dev_status=status)
    w = W[1].float().T if transposed else W[1].float()
    assert torch.equal(out[-170:-1], (x[-170:-1].float() @ w).to(torch.bfloat16))
    assert (out[-1].float().abs() <= 2.0 ** -44 * (x[-1].float() @ w).abs()).all()
    assert int(status.item()) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weights_past_2_31(dtype):
    g = torch.Generator(device=DEV).manual_seed(2)
    E, K, N, rows = 10, 16384, 16384, 50
    x, y = _small(g, rows, K), _small(g, rows, N)
    offsets = torch.tensor([0] * E + [rows], dtype=torch.int32, device=DEV)   # the last expert's
    dW = torch.full((E, K, N), 7.0, dtype=dtype, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_expert_wgrad(x, y, offsets, dW, dev_status=status)
    assert torch.equal(dW[-1], (x.float().T @ y.float()).to(dtype))
    assert not dW[:-1].any() and int(status.item()) == 0
    del dW
    # weights past 2^31 elements, read
    W = torch.zeros(E, K, N, dtype=torch.bfloat16, device=DEV)
    W[-1] = _small(g, K, N)
    out = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_gemm(x, offsets, W, out, dev_status=status)
    assert torch.equal(out, (x.float() @ W[-1].float()).to(torch.bfloat16))
    moe.moe_expert_gemm(x, offsets, W, out, transposed=True, dev_status=status)
    assert torch.equal(out, (x.float() @ W[-1].float().T).to(torch.bfloat16))
