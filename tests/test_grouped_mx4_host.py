"""Grouped routing and the 4-bit operators without a GPU: the oracle's own
checks, and the argument checks that run before any launch."""
import ctypes

import numpy as np
import pytest
import torch

import top_routing_expert_gb300 as moe
from oracle import moe_oracle as O

FAKE = 0x10000  # never dereferenced: every call below fails its host checks


@pytest.fixture(scope="module")
def lib():
    moe.build()
    return moe.load_library()


# ---------------------------------------------------------------- oracle ----

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("aux", [True, False])
def test_oracle_gradient_against_differences(score, renormalize, aux):
    rng = np.random.default_rng(3)
    T, E, k = 5, 12, 3
    l = rng.standard_normal((T, E))
    idx, _, _ = O.route_grouped(l, None, k, score, 4, 2, 2, renormalize, 1.7)
    g = rng.standard_normal((T, k))
    routed = rng.integers(0, 9, E) if aux else None
    args = (idx, g, score, renormalize, 1.7, 3.0, routed)
    grad = O.route_grouped_grad(l, *args)
    h = 1e-5  # central differences: error about h^2 and 2^-53 / h
    for e in range(E):
        d = np.zeros((T, E))
        d[:, e] = h
        num = (O.route_grouped_loss(l + d, *args) - O.route_grouped_loss(l - d, *args)) / (2 * h)
        assert np.abs(num - grad[:, e]).max() < 1e-8


def test_oracle_grouped_choice_by_hand():
    # 3 groups of 2: group values (top 1) .9, .8, .7: groups 0 and 1 are kept
    c = np.array([[0.9, 0.1, 0.2, 0.8, 0.7, 0.7]])
    l = np.log(c / (1 - c))
    idx, w, _ = O.route_grouped(l, None, 3, "sigmoid", 3, 2, 1, False)
    assert idx.tolist() == [[0, 3, 2]]
    # by the sum of two, group 2 (1.4) and then a tie of 1.0: the lower index
    idx, w, _ = O.route_grouped(l, None, 2, "sigmoid", 3, 1, 2, True)
    assert idx.tolist() == [[4, 5]]
    assert np.allclose(w, 0.5)
    # masked experts come last, with weight 0
    l[0, 4] = -np.inf
    idx, w, _ = O.route_grouped(l, None, 2, "sigmoid", 3, 1, 1, True)
    assert idx.tolist() == [[0, 1]]
    idx, w, _ = O.route_grouped(np.full((1, 4), -np.inf), None, 2, "softmax")
    assert idx.tolist() == [[0, 1]] and w.tolist() == [[0.0, 0.0]]


def test_oracle_mx4_grid():
    # a block whose scale is 1 (largest magnitude in [4, 8)): every midpoint and its neighbours
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    want = [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]      # ties to the even code
    eps = 2.0 ** -7
    row = np.zeros((1, 32))
    row[0, :7] = mids
    row[0, 7:14] = [m * (1 - eps) for m in mids]
    row[0, 14:21] = [-m * (1 + eps) for m in mids]
    row[0, 21] = 7.9                                # above 6: held at 6
    code, byte = O.quantize_mx4(row)
    v = O.mx4_values(code, byte)[0]
    assert byte.tolist() == [[127]]
    assert v[:7].tolist() == want
    assert v[7:14].tolist() == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0]
    assert v[14:21].tolist() == [-0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
    assert v[21] == 6.0
    assert O.quantize_mx4(np.zeros((1, 32)))[1].tolist() == [[0]]
    assert O.quantize_mx4(np.full((1, 32), np.inf))[1].tolist() == [[255]]


# -------------------------------------------------------------- refusals ----

def _cfg(**kw):
    return moe.RouteConfig.make(**kw)


def test_route_config_checks(lib):
    s = moe.MoeShape.make(64, 128, 16, 4, 128, 1.0)
    f = ctypes.c_void_p(FAKE)
    n = moe.workspace_size(s)

    def fwd(cfg, logits=f, bias=None, idx=f, w=f, ws=f, nb=n):
        c = None if cfg is None else ctypes.byref(cfg)
        return lib.moe_route_grouped(ctypes.byref(s), c, logits, bias, idx, w, None, None, None,
                                     None, ws, nb, None)

    good = _cfg(n_groups=4, topk_groups=2, group_top=2)
    assert fwd(None) == 1
    for bad in (dict(n_groups=0), dict(n_groups=3), dict(n_groups=4, topk_groups=0),
                dict(n_groups=4, topk_groups=5), dict(group_top=0), dict(group_top=3),
                dict(n_groups=16, topk_groups=8, group_top=2),      # groups of one expert
                dict(n_groups=8, topk_groups=1),                    # k = 4 > 2 experts kept
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert fwd(_cfg(**bad)) == 2, bad
    c = _cfg()
    c.score = 2
    assert fwd(c) == 2
    c = _cfg()
    c.renormalize = 5
    assert fwd(c) == 2
    s64 = moe.MoeShape.make(64, 128, 64, 4, 128, 1.0)
    assert lib.moe_route_grouped(ctypes.byref(s64), ctypes.byref(_cfg(n_groups=64, topk_groups=8)),
                                 f, None, f, f, None, None, None, None, f, 1 << 40, None) == 3
    assert fwd(good, logits=None) == 1
    assert fwd(good, idx=None) == 1
    assert fwd(good, w=ctypes.c_void_p(FAKE + 4)) == 5
    assert fwd(good, bias=ctypes.c_void_p(FAKE + 4)) == 5
    assert fwd(good, ws=None) == 1
    assert fwd(good, nb=n - 1) == 4
    with pytest.raises(ValueError):
        _cfg(score="tanh")

    def bwd(cfg=good, logits=f, idx=f, gw=f, ga=None, routed=None, out=f):
        return lib.moe_route_grouped_bwd(ctypes.byref(s), ctypes.byref(cfg), logits, idx, gw, ga,
                                         routed, out, None)

    assert bwd(logits=None) == 1 and bwd(idx=None) == 1 and bwd(gw=None) == 1 and bwd(out=None) == 1
    assert bwd(ga=f) == 1                                  # grad_aux without routed_counts
    assert bwd(ga=f, routed=ctypes.c_void_p(FAKE + 4)) == 5
    assert bwd(cfg=_cfg(n_groups=5)) == 2


def test_mx4_entry_points_reject_bad_arguments(lib):
    P = ctypes.c_void_p
    f, off = P(FAKE), P(FAKE + 8)
    q = lambda rows=8, K=128, x=f, n=None, xq=f, xs=f: lib.moe_quantize_rows_mx4(
        rows, K, x, n, xq, xs, None)
    assert q(rows=-1) == 2 and q(K=0) == 2 and q(K=96) == 3 and q(K=65600) == 3
    assert q(rows=2 ** 31) == 3
    assert q(x=None) == 1 and q(xq=None) == 1 and q(xs=None) == 1
    assert q(x=off) == 5 and q(xq=off) == 5 and q(xs=off) == 5 and q(n=P(FAKE + 2)) == 5
    assert q(rows=0, x=None) == 0                          # nothing to do
    d = lib.moe_dequantize_rows_mx4
    assert d(8, 96, f, f, f, None) == 3 and d(8, 128, None, f, f, None) == 1
    assert d(8, 128, f, off, f, None) == 5 and d(0, 128, None, None, None, None) == 0
    w = lib.moe_quantize_weights_mx4
    assert w(0, 128, 128, f, f, f, None) == 2 and w(257, 128, 128, f, f, f, None) == 3
    assert w(8, 96, 128, f, f, f, None) == 3 and w(8, 128, 96, f, f, f, None) == 3
    assert w(8, 128, 128, None, f, f, None) == 1 and w(8, 128, 128, f, off, f, None) == 5

    def g(E=8, rows=16, K=128, N=128, xq=f, xs=f, o=f, wq=f, ws=f, gelu=0, D=f, st=f):
        return lib.moe_expert_gemm_mx4(E, rows, K, N, xq, xs, o, wq, ws, gelu, D, st, None)

    assert g(E=0) == 2 and g(N=0) == 2 and g(rows=-1) == 2 and g(gelu=2) == 2
    assert g(E=257) == 3 and g(K=96) == 3 and g(N=96) == 3 and g(N=65600) == 3
    for name in ("xq", "xs", "o", "wq", "ws", "D", "st"):
        assert g(**{name: None}) == 1, name
        assert g(**{name: off}) == 5, name
    assert g(rows=0, xq=None) == 0


def test_binding_checks_layouts():
    x_q = torch.zeros(6, 64, dtype=torch.uint8)
    s = torch.zeros(1, 6, 4, dtype=torch.uint8)
    assert moe._mx4_rows(x_q, s) == (6, 128)
    for bad in (torch.zeros(6, 4), torch.zeros(2, 6, 4), torch.zeros(1, 5, 4)):
        with pytest.raises(ValueError):
            moe._mx4_rows(x_q, bad)
    with pytest.raises(ValueError):
        moe._mx4_rows(x_q[0], s)
    wq = torch.zeros(3, 192, 96, dtype=torch.uint8)
    assert moe._mx4_weights(wq, torch.zeros(3, 2, 2, 32, 4, 4)) == (3, 192, 192)
    with pytest.raises(ValueError):
        moe._mx4_weights(wq, torch.zeros(3, 1, 2, 32, 4, 4))
    with pytest.raises(ValueError):            # host tensors are refused
        moe.moe_dequantize_rows_mx4(x_q, s, torch.zeros(6, 128, dtype=torch.bfloat16))
