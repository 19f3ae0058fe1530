"""The experts' grouped product and its gradients on the GPU, against float64.

Operands are bf16, so products are exact in fp32 and an output's error is its
accumulation's and one rounding to its type. With S = sum |x w| over a
contraction of n terms, one addition per 16 terms costs at most 2^-23 S and the
sum inside an instruction at most 2^-20 S:
    |err| <= half a step of the type |ref| + (n/16 2^-23 + 2^-20) S.
gelu_tanh has a slope below 1.13 and its fp32 evaluation is within 2^-16 |u|. The
slope's own evaluation: z = 1.6 u + 0.07 u^3 carries 2^-22 |z|, which enters as
|z| s(1-s) (1 + |u| (1.6 + 0.22 u^2)) < 0.7 for every u; with exp's and the
quotient's few units, 2^-18."""
import itertools

import numpy as np
import pytest
import torch

import top_routing_expert_gb300 as moe
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
NONE = 7.0  # what outputs hold before a call


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.load_library()


def _draw(g, *shape, std=1.0):
    return (std * torch.randn(shape, generator=g)).to(torch.bfloat16)


def _offsets(lengths, first=0):
    return [first] + [first + n for n in itertools.accumulate(lengths)]


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


# segments: one row; lengths around every K step and stage; empty ones at both
# ends and in the middle; rows before the first and behind the last segment
SEGMENTS = {
    "one_row": ([1], 0, 0),
    "steps": ([15, 16, 17, 1, 31, 33], 0, 0),
    "stages": ([127, 128, 129, 255, 256, 257], 0, 5),
    "empty": ([0, 0, 40, 0, 300, 0], 0, 3),
    "apart": ([70, 1, 0, 200], 9, 130),
    "none": ([0, 0, 0], 4, 4),
    "long": ([1000, 3], 0, 1),
}
WIDTHS = [(64, 64), (128, 320), (192, 256), (448, 704), (1024, 128)]


def _case(name, seed, *widths):
    """Segment offsets and rows of the widths; NaN and infinities in the rows of
    no segment."""
    lengths, first, behind = SEGMENTS[name]
    off = _offsets(lengths, first)
    rows = off[-1] + behind
    g = torch.Generator().manual_seed(seed)
    out = [torch.tensor(off, dtype=torch.int32), rows]
    for w in widths:
        x = _draw(g, rows, w)
        x[:first] = float("nan")
        x[off[-1]:] = float("inf")
        out.append(x)
    return [g, off] + out


def _check(got, ref, S, n, dtype=torch.bfloat16, extra=0.0, what=""):
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + (n / 16 * 2.0 ** -23 + 2.0 ** -20) * S + extra
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    worst = np.unravel_index(np.argmax(err - tol), err.shape) if err.size else ()
    assert (err <= tol).all(), (what, worst, err[worst], tol[worst])


@pytest.mark.parametrize("segments", SEGMENTS)
@pytest.mark.parametrize("K,N", WIDTHS)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("epilogue", [None, "gelu", "gelu_kept", "gelu_grad"])
def test_product(segments, K, N, transposed, epilogue):
    g, off, offsets, rows, x, u = _case(segments, 3, K, N)
    E = len(off) - 1
    W = _draw(g, E, *((N, K) if transposed else (K, N)), std=K ** -0.5)
    u[::2] *= 4                                # slopes on both sides of their range
    out = torch.full((rows, N), NONE, dtype=torch.bfloat16, device=DEV)
    pre = u.to(DEV) if epilogue == "gelu_grad" else torch.full_like(out, NONE)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_expert_gemm(x.to(DEV), offsets.to(DEV), W.to(DEV), out, transposed=transposed,
                        epilogue="gelu" if epilogue == "gelu_kept" else epilogue,
                        pre=None if epilogue in (None, "gelu") else pre, dev_status=status)
    assert int(status.item()) == 0
    out, kept = _f64(out), _f64(pre)
    outside = np.ones(rows, bool)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        outside[lo:hi] = False
        w = _f64(W[e]).T if transposed else _f64(W[e])
        ref, S = _f64(x[lo:hi]) @ w, np.abs(_f64(x[lo:hi])) @ np.abs(w)
        if epilogue in ("gelu", "gelu_kept"):
            if epilogue == "gelu_kept":
                _check(kept[lo:hi], ref, S, K, what="kept")
            _check(out[lo:hi], O.gelu_tanh(ref), 1.13 * S, K, extra=2.0 ** -16 * np.abs(ref))
        elif epilogue == "gelu_grad":
            slope = O.gelu_tanh_slope(_f64(u[lo:hi]))
            _check(out[lo:hi], ref * slope, 1.13 * S, K, extra=2.0 ** -18 * np.abs(ref))
        else:
            _check(out[lo:hi], ref, S, K)
    assert (out[outside] == NONE).all()        # rows of no segment stay as they were
    if epilogue == "gelu_kept":
        assert (kept[outside] == NONE).all()


def test_slope_at_the_ends():
    # a product of ones: the output is the slope itself
    u = torch.tensor([0.0, -0.0, 1.0, -1.0, 7.9, 8.0, 9.0, 60.0, 1e30, 3e38, -8.0, -9.0, -60.0, -1e30,
                      float("inf"), -float("inf"), float("nan"), 1e-40, -0.75, 2.5])
    x = torch.zeros(len(u), 64)
    x[:, 0] = 1
    W = torch.zeros(1, 64, 64)
    W[0, 0] = 1
    to = lambda t: t.to(torch.bfloat16).to(DEV)
    out = torch.empty(len(u), 64, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_gemm(to(x), torch.tensor([0, len(u)], dtype=torch.int32, device=DEV), to(W), out,
                        epilogue="gelu_grad", pre=to(u[:, None].expand(-1, 64).contiguous()),
                        dev_status=torch.zeros(1, dtype=torch.int32, device=DEV))
    got = _f64(out)[:, 0]
    b = _f64(u.to(torch.bfloat16))
    held = np.clip(b, -30, 30)                 # beyond, the slope is 0 or 1
    want = O.gelu_tanh_slope(held)
    nan = np.isnan(b)
    assert np.isnan(got[nan]).all() and not np.isnan(got[~nan]).any()
    assert (np.abs(got - want)[~nan] <= 2.0 ** -8 * np.abs(want[~nan]) + 2.0 ** -18).all()
    assert got[7:10].tolist() == [1, 1, 1] and np.abs(got[11:14]).max() < 1e-10


@pytest.mark.parametrize("segments", SEGMENTS)
@pytest.mark.parametrize("K,N", WIDTHS)
@pytest.mark.parametrize("dtype,accumulate", [(torch.float32, False), (torch.bfloat16, False),
                                              (torch.float32, True)])
def test_weight_gradient(segments, K, N, dtype, accumulate):
    g, off, offsets, rows, x, y = _case(segments, 4, K, N)
    E = len(off) - 1
    before = torch.randn(E, K, N, generator=g).to(dtype)
    dW = before.to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_expert_wgrad(x.to(DEV), y.to(DEV), offsets.to(DEV), dW, accumulate=accumulate,
                         dev_status=status)
    assert int(status.item()) == 0
    for e in range(E):
        a, b = _f64(x[off[e]:off[e + 1]]), _f64(y[off[e]:off[e + 1]])
        ref, S = a.T @ b, np.abs(a).T @ np.abs(b)
        if accumulate:
            S = S + np.abs(_f64(before[e]))    # one more addition
            ref = ref + _f64(before[e])
        _check(_f64(dW[e]), ref, S, len(a), dtype, what=e)
    if accumulate:                             # an expert without rows keeps its bits
        for e in range(E):
            if off[e] == off[e + 1]:
                assert torch.equal(dW[e].cpu(), before[e])


@pytest.mark.parametrize("lengths,first,behind", [([5000], 0, 0), ([2049], 3, 9), ([6300, 0, 7], 0, 5),
                                                  ([2100, 2050], 1, 0), ([64 * 40 + 1], 0, 100),
                                                  ([2130, 2000, 2120, 2115], 0, 0), ([10, 8200], 0, 0)])
@pytest.mark.parametrize("K,N", [(64, 64), (256, 128), (512, 704), (1024, 192)])
@pytest.mark.parametrize("dtype,accumulate", [(torch.float32, False), (torch.bfloat16, False),
                                              (torch.float32, True)])
def test_weight_gradient_of_few_tiles(lengths, first, behind, K, N, dtype, accumulate):
    """Long segments of few tiles, whose rows several pairs share."""
    off = _offsets(lengths, first)
    rows, E = off[-1] + behind, len(lengths)
    g = torch.Generator().manual_seed(12)
    x, y = _draw(g, rows, K), _draw(g, rows, N)
    for t in (x, y):
        t[:first] = float("nan")
        t[off[-1]:] = float("inf")
    before = torch.randn(E, K, N, generator=g).to(dtype)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    runs = []
    for _ in range(2):
        dW = before.to(DEV)
        moe.moe_expert_wgrad(x.to(DEV), y.to(DEV), torch.tensor(off, dtype=torch.int32, device=DEV), dW,
                             accumulate=accumulate, dev_status=status)
        runs.append(dW)
    assert int(status.item()) == 0 and torch.equal(runs[0], runs[1])
    for e in range(E):
        a, b = _f64(x[off[e]:off[e + 1]]), _f64(y[off[e]:off[e + 1]])
        ref, S = a.T @ b, np.abs(a).T @ np.abs(b)
        if accumulate:
            S, ref = S + np.abs(_f64(before[e])), ref + _f64(before[e])
        _check(_f64(runs[0][e]), ref, S, len(a), dtype, what=e)


def test_nan_of_one_expert_stays_there():
    g, off, offsets, rows, x, y = _case("steps", 5, 128, 128)
    x[off[2], 3] = float("nan")
    y[off[4], 5] = float("inf")
    dW = torch.empty(6, 128, 128, device=DEV)
    moe.moe_expert_wgrad(x.to(DEV), y.to(DEV), offsets.to(DEV), dW,
                         dev_status=torch.zeros(1, dtype=torch.int32, device=DEV))
    bad = ~torch.isfinite(dW)
    assert bad[2, 3].all() and int(bad[2].sum()) == 128
    assert bad[4, :, 5].all() and int(bad[4].sum()) == 128
    assert not bad[[0, 1, 3, 5]].any()


def test_offsets_out_of_range_stay_in_the_buffers():
    # device data that no dispatch writes: read as the nearest sound segments
    x, y = (torch.ones(20, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    W = torch.ones(3, 64, 64, dtype=torch.bfloat16, device=DEV)
    offsets = torch.tensor([-5, 8, 4, 99], dtype=torch.int32, device=DEV)   # [0,8), [8,8), [8,20)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.zeros(20, 64, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_gemm(x, offsets, W, out, dev_status=status)
    assert (out == 64).all()
    dW = torch.full((3, 64, 64), NONE, device=DEV)
    moe.moe_expert_wgrad(x, y, offsets, dW, dev_status=status)
    assert (dW[0] == 8).all() and (dW[1] == 0).all() and (dW[2] == 12).all()
    assert int(status.item()) == 0


def test_no_rows():
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    offsets = torch.zeros(4, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    W = torch.ones(3, 64, 128, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_gemm(x, offsets, W, torch.empty(0, 128, dtype=torch.bfloat16, device=DEV),
                        dev_status=status)
    g = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        dW = torch.full((3, 64, 128), NONE, dtype=dtype, device=DEV)
        moe.moe_expert_wgrad(x, g, offsets, dW, dev_status=status)
        assert (dW == 0).all()
    dW = torch.full((3, 64, 128), NONE, device=DEV)
    moe.moe_expert_wgrad(x, g, offsets, dW, accumulate=True, dev_status=status)
    assert (dW == NONE).all()


def test_many_experts():
    # the largest expert count, most of them with few rows
    E, K, N = 256, 64, 192
    g = torch.Generator().manual_seed(8)
    lengths = torch.randint(0, 5, (E,), generator=g).tolist()
    lengths[17] = 700
    off = _offsets(lengths)
    x, y = _draw(g, off[-1], K), _draw(g, off[-1], N)
    W = _draw(g, E, K, N, std=0.125)
    offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.empty(off[-1], N, dtype=torch.bfloat16, device=DEV)
    moe.moe_expert_gemm(x.to(DEV), offsets, W.to(DEV), out, dev_status=status)
    dW = torch.empty(E, K, N, device=DEV)
    moe.moe_expert_wgrad(x.to(DEV), y.to(DEV), offsets, dW, dev_status=status)
    assert int(status.item()) == 0
    out, dW = _f64(out), _f64(dW)
    for e in range(E):
        a, b, w = _f64(x[off[e]:off[e + 1]]), _f64(y[off[e]:off[e + 1]]), _f64(W[e])
        _check(out[off[e]:off[e + 1]], a @ w, np.abs(a) @ np.abs(w), K)
        _check(dW[e], a.T @ b, np.abs(a).T @ np.abs(b), len(a), torch.float32)


def test_gradients_against_differences():
    # <D, du W^T> and <x^T du, V> against central differences of the loss
    # sum du . gelu(x W) in float64, in random directions
    g, off, offsets, rows, x = _case("steps", 6, 64)
    E, N = len(off) - 1, 128
    W, gy = _draw(g, E, 64, N, std=0.125), _draw(g, rows, N)
    d = lambda t: t.to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    new = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device=DEV)
    a, u = new(rows, N), new(rows, N)
    moe.moe_expert_gemm(d(x), d(offsets), d(W), a, epilogue="gelu", pre=u, dev_status=status)
    # gelu'(u) gy as a product with the identity
    eye = torch.eye(N, dtype=torch.bfloat16, device=DEV).expand(E, N, N).contiguous()
    gu, gx, dW = new(rows, N), new(rows, 64), new(E, 64, N, dt=torch.float32)
    moe.moe_expert_gemm(d(gy), d(offsets), eye, gu, transposed=True, epilogue="gelu_grad", pre=u,
                        dev_status=status)
    moe.moe_expert_gemm(gu, d(offsets), d(W), gx, transposed=True, dev_status=status)
    moe.moe_expert_wgrad(d(x), gu, d(offsets), dW, dev_status=status)
    x64, W64, g64 = _f64(x), _f64(W), _f64(gy)

    def loss(x, W):
        return sum((g64[lo:hi] * O.gelu_tanh(x[lo:hi] @ W[e])).sum()
                   for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])))

    rng = np.random.default_rng(0)
    h = 1e-5
    for _ in range(4):
        vx, vw = rng.standard_normal(x64.shape), rng.standard_normal(W64.shape)
        # bf16 roundings on the way: u, gu and gx, 2^-8 each of terms that add up
        # in random signs: 4 times their 2-norm's share, of 2^-8 sqrt(3)
        for got, v, num in ((_f64(gx), vx, (loss(x64 + h * vx, W64) - loss(x64 - h * vx, W64)) / (2 * h)),
                            (_f64(dW), vw, (loss(x64, W64 + h * vw) - loss(x64, W64 - h * vw)) / (2 * h))):
            assert abs((got * v).sum() - num) <= 4 * 2.0 ** -8 * 3 ** 0.5 * np.linalg.norm(got * v)


def test_streams_and_repeats():
    # the same bits on another stream and in a replayed graph
    g, off, offsets, rows, x, y = _case("stages", 7, 448, 704)
    E = len(off) - 1
    x, y, offsets, W = x.to(DEV), y.to(DEV), offsets.to(DEV), _draw(g, E, 448, 704, std=0.05).to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    new = lambda: (torch.zeros(rows, 704, dtype=torch.bfloat16, device=DEV),
                   torch.zeros(rows, 704, dtype=torch.bfloat16, device=DEV),
                   torch.zeros(E, 448, 704, device=DEV))

    def both(out, pre, dW):
        moe.moe_expert_gemm(x, offsets, W, out, epilogue="gelu", pre=pre, dev_status=status)
        moe.moe_expert_wgrad(x, y, offsets, dW, dev_status=status)

    first = new()
    both(*first)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    second = new()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        both(*second)
    stream.synchronize()
    third = new()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(*third)
    for _ in range(2):
        for t in third:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(first, second, third):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_device_refusals():
    """Strided, misaligned, mistyped and missing tensors are refused before a launch."""
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    x, W, out, dW = bf(4, 64), bf(1, 64, 128), torch.full((4, 128), NONE, dtype=torch.bfloat16, device=DEV), bf(1, 64, 128)
    gemm, wgrad = moe.moe_expert_gemm, moe.moe_expert_wgrad
    wide = bf(4, 128)
    for call in (lambda: gemm(wide[:, :64], off, W, out, dev_status=st),
                 lambda: gemm(x, off, W.transpose(1, 2), out, transposed=True, dev_status=st),
                 lambda: gemm(x.float(), off, W, out, dev_status=st),
                 lambda: gemm(x, off.long(), W, out, dev_status=st),
                 lambda: gemm(x, off[:1], W, out, dev_status=st),
                 lambda: gemm(x, off, W, out, epilogue="gelu", pre=wide[:, :64], dev_status=st),
                 lambda: wgrad(wide[:, :64], bf(4, 128), off, dW, dev_status=st),
                 lambda: wgrad(x, bf(4, 128).T.contiguous().T, off, dW, dev_status=st),
                 lambda: wgrad(x, bf(4, 128), off, dW.half(), dev_status=st)):
        with pytest.raises(ValueError):
            call()
    shifted = bf(4 * 64 + 8)[4:4 + 4 * 64].view(4, 64)          # 8 bytes past an aligned address
    for code, call in ((5, lambda: gemm(shifted, off, W, out, dev_status=st)),
                       (5, lambda: wgrad(shifted, bf(4, 128), off, dW, dev_status=st)),
                       (1, lambda: gemm(x, off, W, out)),
                       (1, lambda: gemm(x, off, W, out, epilogue="gelu_grad", dev_status=st)),
                       (2, lambda: gemm(x, off, W, out, pre=wide, dev_status=st)),
                       (3, lambda: wgrad(x, bf(4, 128), off, dW, accumulate=True, dev_status=st)),
                       (3, lambda: gemm(bf(4, 32), off, bf(1, 32, 128), out, dev_status=st))):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code == code
    assert (out == NONE).all()
