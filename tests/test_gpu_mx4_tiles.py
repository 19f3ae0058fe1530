"""The 4-bit product where a CTA or a CTA pair works through several tiles of
several K stages: accumulators, ring slots and token scales in use again and again.

Codes and scale bytes are drawn as such, so the operands are exact. The error is
the fp32 accumulation's and the rounding to bf16 (half a step, 2^-8): with S = sum
|x w|, one addition per 64 products costs at most 2^-23 S and the sum inside an
instruction at most 2^-20 S. GELU's slope is below 1.13 and its own evaluation
within 2^-16 of the value; |u| is below 2^10, so that a value that is held where
the exponential would overflow is below 2^-50."""
import math

import numpy as np
import pytest
import torch

import top_routing_expert_gb300 as moe

pytestmark = pytest.mark.gpu
DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.load_library()


def _values(codes, byte):
    """codes [..., K/2] and scale bytes [..., K/32] -> fp64 values [..., K]."""
    lut = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    v = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), dim=-1).flatten(-2)
    return v * torch.exp2(byte.double() - 127.0).repeat_interleave(32, dim=-1)


def _bytes(g, lo, hi, *shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)


def _weights(g, E, K, N):
    shift = round(math.log2(3.0 * 3.0 * math.sqrt(K)))
    q = _bytes(g, 0, 256, E, N, K // 2)
    byte = _bytes(g, 126 - shift, 129 - shift, E, N, K // 32)
    tn, tk = -(-N // 128), -(-K // 128)
    pad = torch.zeros(E, tn * 128, tk * 4, dtype=torch.uint8, device=DEV)
    pad[:, :N, :K // 32] = byte
    return q, byte, pad.view(E, tn, 4, 32, tk, 4).permute(0, 1, 4, 3, 2, 5).contiguous()


def _rows_scale(byte):
    R, n = byte.shape
    pad = torch.zeros(R, -(-n // 4) * 4, dtype=torch.uint8, device=DEV)
    pad[:, :n] = byte
    return pad.view(R, -1, 4).transpose(0, 1).contiguous()


def _check(out, x_q, x_byte, w_q, w_byte, counts, gelu):
    K, r = 2 * x_q.shape[1], 0
    for e, n in enumerate(counts):
        if n == 0:
            continue
        a, w = _values(x_q[r:r + n], x_byte[r:r + n]), _values(w_q[e], w_byte[e])
        ref, mag = a @ w.T, a.abs() @ w.abs().T
        tol = (K / 64 * 2.0 ** -23 + 2.0 ** -20) * mag
        if gelu:
            assert ref.abs().max() < 1024
            ref = ref / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (ref + 0.044715 * ref ** 3)))
            tol = 1.13 * tol + 2.0 ** -16 * ref.abs() + 2.0 ** -50
        bad = ~((out[r:r + n].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + tol)
        assert not bad.any(), (e, n, bad.nonzero()[:4].tolist())
        r += n
    assert (out[r:] == 7.0).all()


def _ragged(E, mean, seed):
    rng = np.random.default_rng(seed)
    counts = (mean * np.exp(0.5 * rng.standard_normal(E))).astype(int)
    if E >= 8:
        counts[:: E // 3] = rng.integers(0, 3, len(counts[:: E // 3]))
    return counts.tolist()


# experts, mean rows, K, N: a K block of 256 is a stage, a ring has 4 to 10 of them,
# and a pair's tile is 512 columns, half of it where N ends sooner
@pytest.mark.parametrize("E,mean,K,N", [
    (16, 1500, 832, 1408), (16, 1500, 2112, 1408), (16, 520, 256, 1408), (8, 2900, 576, 1728),
    (8, 2300, 1088, 1984), (4, 1700, 4160, 3136), (100, 40, 832, 1408), (64, 16, 1600, 2240),
    (256, 70, 320, 704), (3, 19000, 448, 320), (64, 50, 4096, 960), (2, 30, 2112, 30016),
])
@pytest.mark.parametrize("gelu", [False, True])
def test_several_tiles_and_stages(E, mean, K, N, gelu):
    counts = _ragged(E, mean, K + N)
    g = torch.Generator(device=DEV).manual_seed(N)
    rows = sum(counts) + 5
    w_q, w_byte, w_scale = _weights(g, E, K, N)
    x_q = _bytes(g, 0, 256, rows, K // 2)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    out = torch.empty(rows, N, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    for _ in range(2):   # other scales in the same places the second time
        x_byte = _bytes(g, 125, 130, rows, K // 32)
        out.fill_(7.0)
        moe.moe_expert_gemm_mx4(x_q, _rows_scale(x_byte), off, w_q, w_scale, out, gelu=gelu, dev_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        _check(out, x_q, x_byte, w_q, w_byte, counts, gelu)


# at least 64 rows to an expert, or many columns, make it CTA pairs; these do not
@pytest.mark.parametrize("E,mean,K,N", [(40, 30, 832, 320), (128, 12, 1088, 192), (60, 50, 320, 448),
                                        (16, 40, 2112, 1600)])
def test_several_tiles_of_single_ctas(E, mean, K, N):
    counts = _ragged(E, mean, K)
    assert sum(counts) + 5 < 64 * E and 2 * E * N < 3 * 512 * 76
    g = torch.Generator(device=DEV).manual_seed(K)
    rows = sum(counts) + 5
    w_q, w_byte, w_scale = _weights(g, E, K, N)
    x_q, x_byte = _bytes(g, 0, 256, rows, K // 2), _bytes(g, 125, 130, rows, K // 32)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    for gelu in (False, True):
        out = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device=DEV)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        moe.moe_expert_gemm_mx4(x_q, _rows_scale(x_byte), off, w_q, w_scale, out, gelu=gelu, dev_status=status)
        torch.cuda.synchronize()
        assert status.item() == 0
        _check(out, x_q, x_byte, w_q, w_byte, counts, gelu)
