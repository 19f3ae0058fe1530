"""GELU of the 4-bit product over the whole range of its argument.

A row has one value other than zero and so has a weight's column, so that the
accumulator is their product exactly. The tanh form u / (1 + exp(-2 z)) is
within 2^-8 (the rounding to bf16) and 2^-16 (|2 z| up to 42: the rounding of an
exponent of up to 60, 2^-19 of the value, an exponential and two products) of
itself, and anything as small where it is below 2^-57."""
import numpy as np
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


def _gelu(u):
    z = 2.0 * np.sqrt(2.0 / np.pi) * (u + 0.044715 * u ** 3)
    with np.errstate(over="ignore"):
        return u / (1.0 + np.exp(-z))


# (experts, rows of each, output columns): one CTA to a tile, then CTA pairs
@pytest.mark.parametrize("E,rows,N", [(1, 40, 64), (2, 45, 128), (1, 200, 64), (2, 90, 640)])
def test_gelu_over_its_range(E, rows, N):
    K = 64
    rng = np.random.default_rng(rows)
    e2m1 = np.array([1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
    draw = lambda n, lo, hi: rng.choice(e2m1, n) * np.exp2(rng.integers(lo, hi, n).astype(np.float64)) * rng.choice([-1.0, 1.0], n)
    a = draw(E * rows, -4, 3)
    a[::5] = draw(len(a[::5]), 3, 62)          # products up to 2^126 or so
    w = draw(E * N, -3, 2).reshape(E, N)
    w[:, ::4] = draw(E * len(range(0, N, 4)), 2, 58).reshape(E, -1)
    x = torch.zeros(E * rows, K)
    x[:, 3] = torch.from_numpy(a.astype(np.float32))
    W = torch.zeros(E, K, N)
    W[:, 3] = torch.from_numpy(w.astype(np.float32))
    x_q = torch.empty(E * rows, K // 2, dtype=torch.uint8, device=DEV)
    x_s = torch.empty(1, E * rows, 4, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_rows_mx4(x.to(torch.bfloat16).to(DEV), x_q, x_s)
    w_q = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    w_s = torch.empty(E, (N + 127) // 128, 1, 32, 4, 4, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_weights_mx4(W.to(torch.bfloat16).to(DEV), w_q, w_s)
    off = torch.arange(0, E * rows + 1, rows, dtype=torch.int32, device=DEV)
    out = torch.empty(E * rows, N, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_expert_gemm_mx4(x_q, x_s, off, w_q, w_s, out, gelu=True, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    got = out.float().cpu().numpy().astype(np.float64).reshape(E, rows, N)
    ref = _gelu(a.reshape(E, rows, 1) * w[:, None, :])
    assert np.abs(ref).max() > 1e30 and (ref == 0).any()
    bad = ~(np.abs(got - ref) <= (2.0 ** -8 + 2.0 ** -16) * np.abs(ref) + 2.0 ** -57)
    assert not bad.any(), (bad.sum(), got[bad][:8], ref[bad][:8])


def test_gelu_of_nan_leaves_the_neighbours():
    """Tokens share a reciprocal in twos; a row that is NaN leaves all others alone."""
    g = torch.Generator().manual_seed(5)
    rows, K, N = 90, 128, 192
    x = torch.randn(rows, K, generator=g).to(torch.bfloat16).to(DEV)
    W = (torch.randn(1, K, N, generator=g) / K ** 0.5).to(torch.bfloat16).to(DEV)
    w = moe.Mx4Weights(W, W.transpose(1, 2).contiguous())
    q = torch.empty(rows, K // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(1, rows, 4, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_rows_mx4(x, q, s)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    outs = []
    for bad in ([], [0, 7, 32, 33, 89]):
        t = s.clone()
        t[0, bad, 1] = 255
        out = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV)
        moe.moe_expert_gemm_mx4(q, t, off, w.W1q, w.w1_scale, out, gelu=True, dev_status=status)
        outs.append(out.float().cpu().numpy())
    assert np.isnan(outs[1][bad]).all()
    keep = np.setdiff1d(np.arange(rows), bad)
    # its factor of the shared reciprocal is 2^60 in place of its own: the last bits may differ
    assert (np.abs(outs[1][keep] - outs[0][keep]) <= 2.0 ** -7 * np.abs(outs[0][keep])).all()
