"""Microscaled 4-bit quantisation and the experts' product on the GPU.

Codes and scale bytes are compared exactly with the float64 oracle. A product's
operands are exact, so its error is the fp32 accumulation's and the rounding to
bf16 (half a step, 2^-8): with S = sum |x w|, one addition per 64 products costs
at most 2^-23 S and the sum inside an instruction at most 2^-20 S, so
|err| <= 2^-8 |ref| + (K/64 2^-23 + 2^-20) S. GELU's slope is below 1.13 and
its own fp32 evaluation (|u| up to 8: exp's argument up to 2^6) is within 2^-16 |u|."""
import numpy as np
import pytest
import torch

import top_routing_expert_gb300 as moe
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.load_library()


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _quantize(x, n_rows=None, fill=0xAB):
    rows, K = x.shape
    q = torch.full((rows, K // 2), fill, dtype=torch.uint8, device=DEV)
    s = torch.full(((K + 127) // 128, rows, 4), fill, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_rows_mx4(x, q, s, n_rows=n_rows)
    return q, s


def _rows(rows, K, seed):
    """Rows over many binades, with the values where rounding and scaling turn."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g) * torch.exp2(torch.randint(-6, 7, (rows, K // 32), generator=g)).repeat_interleave(32, 1)
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.75, -0.25, -0.75, -5.0, 4.0, 0.0, -0.0, 1e-38])
    x[0, :16] = mids
    x[0, 16:32] = 0
    if rows > 3:
        x[1] = 0
        x[2, :32] = 1e-39                      # below the smallest scale
        x[2, 32:64] = 3.3e38
        x[3, 5] = float("inf")
        x[3, 40] = float("nan")
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("rows,K", [(1, 64), (3, 128), (5, 192), (24, 2048), (33, 1408), (130, 320),
                                    (1000, 4096), (2, 14336)])
def test_quantize_rows(rows, K):
    x = _rows(rows, K, rows)
    q, s = _quantize(x.to(DEV))
    code, byte = O.quantize_mx4(_f64(x))
    wq, ws = O.pack_mx4_rows(code, byte)
    np.testing.assert_array_equal(q.cpu().numpy(), wq)
    np.testing.assert_array_equal(s.cpu().numpy(), ws)
    back = torch.full((rows, K), 7.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_dequantize_rows_mx4(q, s, back)
    np.testing.assert_array_equal(_f64(back), O.mx4_values(code, byte))


def test_quantize_stops_at_the_device_row_count():
    x = _rows(50, 256, 1).to(DEV)
    whole_q, whole_s = _quantize(x)
    for n in (0, 1, 17, 50, 60, -3):
        count = torch.tensor([n], dtype=torch.int32, device=DEV)
        q, s = _quantize(x, count, fill=0x5C)
        m = min(max(n, 0), 50)
        assert torch.equal(q[:m], whole_q[:m]) and torch.equal(s[:, :m], whole_s[:, :m])
        assert (q[m:] == 0x5C).all() and (s[:, m:] == 0x5C).all()


@pytest.mark.parametrize("E,K,N", [(1, 64, 64), (3, 192, 320), (2, 1408, 128)])
def test_quantize_weights(E, K, N):
    W = torch.stack([_rows(K, N, e) for e in range(E)])
    q = torch.full((E, N, K // 2), 0xAB, dtype=torch.uint8, device=DEV)
    s = torch.full((E, (N + 127) // 128, (K + 127) // 128, 32, 4, 4), 0xAB, dtype=torch.uint8, device=DEV)
    moe.moe_quantize_weights_mx4(W.to(DEV), q, s)
    for e in range(E):
        code, byte = O.quantize_mx4(_f64(W[e]).T)
        np.testing.assert_array_equal(q[e].cpu().numpy(), code[:, 0::2] | (code[:, 1::2] << 4))
        np.testing.assert_array_equal(s[e].cpu().numpy(), O.pack_mx4_weight_scale(byte))


def _problem(counts, K, N, seed, spare=0):
    """Segments of the given lengths; `spare` rows past the last segment."""
    E, rows = len(counts), sum(counts) + spare
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g).to(torch.bfloat16)
    W = (torch.randn(E, K, N, generator=g) / K ** 0.5).to(torch.bfloat16)
    # block scales that differ from one another by powers of two
    x *= torch.exp2(torch.randint(-2, 3, (rows, K // 32), generator=g)).repeat_interleave(32, 1).to(torch.bfloat16)
    W *= torch.exp2(torch.randint(-2, 3, (E, K // 32, N), generator=g)).repeat_interleave(32, 1).to(torch.bfloat16)
    q, s = _quantize(x.to(DEV))
    weights = moe.Mx4Weights(W.to(DEV), W.transpose(1, 2).contiguous().to(DEV))
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    return x, W, q, s, weights, off


def _product(q, s, off, wq, ws, gelu=False, fill=7.0):
    out = torch.full((q.shape[0], wq.shape[1]), fill, dtype=torch.bfloat16, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_expert_gemm_mx4(q, s, off, wq, ws, out, gelu=gelu, dev_status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    return out


def _check(out, x, W, counts, gelu=False):
    xv = O.mx4_values(*O.quantize_mx4(_f64(x)))
    K = xv.shape[1]
    r = 0
    for e, n in enumerate(counts):
        if n == 0:
            continue
        wv = O.mx4_values(*O.quantize_mx4(_f64(W[e]).T))
        a = xv[r:r + n]
        ref, mag = a @ wv.T, np.abs(a) @ np.abs(wv).T
        tol = (K / 64 * 2.0 ** -23 + 2.0 ** -20) * mag
        if gelu:
            tol = 1.13 * tol + 2.0 ** -16 * np.abs(ref)
            ref = O.gelu_tanh(ref)
        got = _f64(out[r:r + n])
        err = np.abs(got - ref)
        assert np.isfinite(got).all()
        assert (err <= 2.0 ** -8 * np.abs(ref) + tol + 1e-30).all(), (e, err.max(), np.abs(ref).max())
        r += n
    assert (_f64(out[r:]) == 7.0).all()           # rows past the segments are left alone


PRODUCTS = [  # rows of each expert, K, N
    ([1], 64, 64), ([16], 128, 128), ([5, 0, 3], 192, 320), ([1, 1, 1, 1], 256, 256),
    ([0, 0, 7, 0], 320, 64), ([17, 250, 1, 90], 1408, 192), ([239, 240, 241, 2], 512, 128),
    ([700, 3, 0, 129, 481], 640, 448), ([33] * 20, 1088, 64), ([1500, 900], 2048, 1408),
]


@pytest.mark.parametrize("counts,K,N", PRODUCTS)
def test_product(counts, K, N):
    x, W, q, s, w, off = _problem(counts, K, N, len(counts) + K, spare=3)
    _check(_product(q, s, off, w.W1q, w.w1_scale), x, W, counts)


@pytest.mark.parametrize("counts,K,N", [([5, 0, 3], 192, 320), ([300, 100], 1408, 256)])
def test_product_with_gelu(counts, K, N):
    x, W, q, s, w, off = _problem(counts, K, N, 3)
    _check(_product(q, s, off, w.W1q, w.w1_scale, gelu=True), x, W, counts, gelu=True)


def test_product_many_experts_and_a_long_reduction():
    counts = [i % 5 for i in range(256)]
    x, W, q, s, w, off = _problem(counts, 128, 64, 1)
    _check(_product(q, s, off, w.W1q, w.w1_scale), x, W, counts)
    x, W, q, s, w, off = _problem([9, 4], 14336, 128, 2)
    _check(_product(q, s, off, w.W1q, w.w1_scale), x, W, [9, 4])


def test_product_of_short_segments_with_many_columns():
    """Few rows to each of many experts: tiles of 512 columns, mostly 16 tokens wide."""
    counts = [(3 * i) % 5 if i % 7 else 17 * (i % 3) for i in range(100)]
    x, W, q, s, w, off = _problem(counts, 192, 640, 8, spare=2)
    _check(_product(q, s, off, w.W1q, w.w1_scale), x, W, counts)


def test_product_of_nan_blocks():
    """A block that stands for NaN makes its row NaN, and no other."""
    x, W, q, s, w, off = _problem([20, 12], 256, 128, 4)
    s[1, 7, 2] = 255
    out = _f64(_product(q, s, off, w.W1q, w.w1_scale))
    assert np.isnan(out[7]).all()
    keep = np.arange(32) != 7
    s[1, 7, 2] = 127
    again = _f64(_product(q, s, off, w.W1q, w.w1_scale))
    assert np.array_equal(out[keep], again[keep])


def test_product_offsets_are_held_to_the_buffer():
    """Offsets that run past the buffer or fall back are cut, never followed."""
    x, W, q, s, w, off = _problem([20, 12], 256, 128, 5)
    good = _product(q, s, off, w.W1q, w.w1_scale)
    wild = torch.tensor([0, 20, 4000], dtype=torch.int32, device=DEV)
    assert torch.equal(_product(q, s, wild, w.W1q, w.w1_scale), good)
    back = torch.tensor([-5, 20, 3], dtype=torch.int32, device=DEV)
    out = _product(q, s, back, w.W1q, w.w1_scale)
    assert torch.equal(out[:20], good[:20]) and (out[20:] == 7.0).all()


def test_product_repeats_on_another_stream_and_in_a_graph():
    x, W, q, s, w, off = _problem([300, 0, 77, 512], 1024, 512, 6)
    a = _product(q, s, off, w.W1q, w.w1_scale)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = _product(q, s, off, w.W1q, w.w1_scale)
    assert torch.equal(a, b)
    out = torch.zeros_like(a)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    xd = x.to(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_quantize_rows_mx4(xd, q, s)
        moe.moe_expert_gemm_mx4(q, s, off, w.W1q, w.w1_scale, out, dev_status=status)
    q.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out) and status.item() == 0


# ------------------------------------------------------------------ layer ----

@pytest.mark.parametrize("T,H,E,k,h,cf,score", [(257, 192, 16, 3, 320, 1.0, "sigmoid"),
                                                (1, 128, 8, 2, 128, 1.25, "softmax"),
                                                (700, 256, 32, 4, 128, 2.0, "sigmoid")])
def test_layer_step_by_step(T, H, E, k, h, cf, score):
    """Each step of the layer against the oracle on that step's own inputs
    (rounding to 4 bits in between would let a last-bit difference grow)."""
    from top_routing_expert_gb300.mx4 import Mx4Layer
    g = torch.Generator().manual_seed(T)
    draw = lambda *n, std=1.0: (std * torch.randn(n, generator=g)).to(torch.bfloat16).to(DEV)
    x, gate = draw(T, H), draw(H, E, std=H ** -0.5)
    W1, W2 = draw(E, H, h, std=H ** -0.5), draw(E, h, H, std=h ** -0.5)
    cfg = dict(score=score, n_groups=4, topk_groups=2, group_top=2, scale=1.5)
    bias = (0.05 * torch.randn(E, generator=g)).to(DEV)
    layer = Mx4Layer(moe.MoeShape.make(T, H, E, k, h, cf), moe.RouteConfig.make(**cfg), W1, W2)
    for t in (layer.act, layer.x_perm, layer.y_perm):
        t.fill_(7.0)
    y = torch.empty_like(x)
    layer.forward(x, gate, y, select_bias=bias)
    torch.cuda.synchronize()
    assert layer.dev_status.item() == 0
    idx, w, _ = O.route_grouped(layer.logits.cpu().numpy().astype(np.float64),
                                bias.cpu().numpy().astype(np.float64), k, **cfg)
    np.testing.assert_array_equal(layer.topk_idx.cpu().numpy(), idx)
    d = O.dispatch_plan(idx, E, O.capacity(T, E, k, cf))
    np.testing.assert_array_equal(layer.dest_row.cpu().numpy(), d.dest_row)
    n = int(d.offsets[-1])
    counts = np.diff(d.offsets).tolist()
    _check(layer.act, layer.x_perm[:n], W1.cpu(), counts, gelu=True)
    _check(layer.y_perm, layer.act[:n], W2.cpu(), counts)
    # combine: an fp32 sum of k products and one rounding to bf16 (the sum itself,
    # not the oracle's combine, which is rounded to bf16 already)
    rows = np.where(d.dest_row >= 0, d.dest_row, 0)
    terms = (_f64(layer.y_perm)[rows] * (d.dest_row >= 0)[:, :, None]
             * layer.topk_w.cpu().numpy().astype(np.float64)[:, :, None])
    ref, mag = terms.sum(axis=1), np.abs(terms).sum(axis=1)
    assert (np.abs(_f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) + 16 * 2.0 ** -24 * mag + 1e-30).all()
    # the router's gradient for the weights' gradient of a sum of y times v
    grad = layer.router_grad(torch.ones_like(layer.topk_w), torch.empty_like(layer.logits))
    l = layer.logits.cpu().numpy().astype(np.float64)
    want = O.route_grouped_grad(l, idx, np.ones((T, k)), score, True, 1.5)
    assert np.abs(grad.cpu().numpy() - want).max() <= 2 * (48 + 8 * np.abs(l).max()) * 2.0 ** -24 * 1.5


def test_layer_in_a_graph_and_with_no_tokens():
    from top_routing_expert_gb300.mx4 import Mx4Layer
    T, H, E, k, h = 300, 128, 8, 2, 192
    g = torch.Generator().manual_seed(0)
    draw = lambda *n: (0.1 * torch.randn(n, generator=g)).to(torch.bfloat16).to(DEV)
    x, gate, W1, W2 = draw(T, H), draw(H, E), draw(E, H, h), draw(E, h, H)
    layer = Mx4Layer(moe.MoeShape.make(T, H, E, k, h, 1.0), moe.RouteConfig.make(), W1, W2)
    y, want = torch.empty_like(x), torch.empty_like(x)
    layer.forward(x, gate, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.forward(x, gate, y)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and layer.dev_status.item() == 0
    none = Mx4Layer(moe.MoeShape.make(0, H, E, k, h, 1.0), moe.RouteConfig.make(), W1, W2)
    none.forward(x[:0], gate, y[:0])
    torch.cuda.synchronize()
    assert none.aux.item() == 0 and none.routed_counts.sum().item() == 0
    with pytest.raises(ValueError):
        Mx4Layer(moe.MoeShape.make(T, H, E, k, h, 1.0), moe.RouteConfig.make(), W2, W1)
