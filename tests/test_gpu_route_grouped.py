"""Grouped routing and its gradient on the GPU against the float64 oracle.

The chosen experts are compared exactly. Tolerances count fp32 roundings
(u = 2^-24): an exponential of a difference d costs |d| u for its argument and
a few u itself, a score a few more for the sum (64-term trees: under 8 u) and
the divisions, so a weight is within (32 + 4 max|d|) u of itself, and likewise
P (relative, its terms being positive). A gradient is a sum of products of
such factors: the same factor times the largest magnitude that enters it."""
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


def _run(logits, bias, k, stats=True, stream=None, **cfg):
    T, E = logits.shape
    s = moe.MoeShape.make(T, 64, E, k, 64, 1.0)
    ws = moe.Workspace(s)
    out = {"idx": torch.full((T, k), -7, dtype=torch.int32, device=DEV),
           "w": torch.full((T, k), float("nan"), device=DEV),
           "routed": torch.full((E,), -7, dtype=torch.int32, device=DEV) if stats else None,
           "P": torch.full((E,), float("nan"), device=DEV) if stats else None,
           "aux": torch.full((1,), float("nan"), device=DEV) if stats else None,
           "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    moe.moe_route_grouped(s, moe.RouteConfig.make(**cfg), logits, bias, out["idx"], out["w"],
                          routed_counts=out["routed"], P=out["P"], aux=out["aux"],
                          dev_status=out["status"], ws=ws, stream=stream)
    torch.cuda.synchronize()
    return {n: None if t is None else t.cpu().numpy() for n, t in out.items()}


def _check(logits, bias, k, got, **cfg):
    l = logits.cpu().numpy().astype(np.float64)
    b = None if bias is None else bias.cpu().numpy().astype(np.float64)
    idx, w, s = O.route_grouped(l, b, k, **cfg)
    np.testing.assert_array_equal(got["idx"], idx)
    fin = np.where(np.isfinite(l), l, 0.0)
    # exp's argument: the logit for a sigmoid, the difference to another logit for a softmax
    spread = 2 * np.abs(fin).max() if l.size else 0.0
    tol = (32 + 4 * spread) * U
    assert (np.abs(got["w"] - w) <= tol * np.abs(w) + 1e-37).all()
    if got["P"] is not None and l.size:
        T, E = l.shape
        routed = np.bincount(idx.ravel(), minlength=E)
        np.testing.assert_array_equal(got["routed"], routed)
        tot = s.sum(axis=1, keepdims=True)
        P = np.divide(s, tot, out=np.zeros_like(s), where=tot > 0).mean(axis=0)
        assert (np.abs(got["P"] - P) <= (tol + 64 * U) * P + 1e-37).all()
        aux = E * (routed / (T * k) * P).sum()
        assert abs(got["aux"][0] - aux) <= (tol + 96 * U) * aux + 1e-37


def _logits(T, E, seed, spread=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return spread * torch.randn(T, E, generator=g, device=DEV), 0.1 * torch.randn(E, generator=g, device=DEV)


CASES = [  # T, E, k, n_groups, topk_groups, group_top
    (1, 1, 1, 1, 1, 1), (1, 8, 2, 1, 1, 1), (7, 8, 8, 1, 1, 1), (129, 12, 3, 4, 2, 2),
    (65, 15, 4, 5, 3, 2), (300, 16, 2, 16, 3, 1), (33, 32, 5, 32, 7, 1), (257, 60, 6, 4, 2, 2),
    (1000, 64, 6, 8, 3, 2), (77, 100, 8, 10, 5, 1), (130, 128, 2, 1, 1, 1), (511, 160, 6, 8, 3, 1),
    (200, 255, 7, 5, 2, 2), (1021, 256, 8, 8, 4, 2), (64, 256, 1, 2, 1, 1),
]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,keep,top", CASES)
def test_route_grouped(T, E, k, G, keep, top, score):
    logits, bias = _logits(T, E, T + E)
    for renorm, scale, b in ((True, 2.5, bias), (False, 1.0, None), (False, -0.5, bias), (True, 1.0, None)):
        cfg = dict(score=score, n_groups=G, topk_groups=keep, group_top=top, renormalize=renorm, scale=scale)
        got = _run(logits, b, k, stats=renorm, **cfg)
        assert got["status"][0] == 0
        _check(logits, b, k, got, **cfg)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_ties_and_exact_ties(score):
    """Logits on a coarse grid plus a few ulps: many selection values are
    equal or within fp32 error of one another; float64 tells them apart."""
    for T, E, k, G, keep, top in ((500, 64, 6, 8, 3, 2), (400, 256, 8, 1, 1, 1), (300, 16, 3, 1, 1, 1)):
        logits, bias = _logits(T, E, 5)
        logits = torch.round(logits * 4) / 4
        ulp = torch.randint(-2, 3, logits.shape, generator=torch.Generator().manual_seed(1)).to(DEV)
        near = logits * (1 + ulp * 2.0 ** -23)
        flat = torch.round(bias * 8) / 8
        for x in (logits, near):
            for b in (None, flat):
                cfg = dict(score=score, n_groups=G, topk_groups=keep, group_top=top)
                got = _run(x, b, k, **cfg)
                _check(x, b, k, got, **cfg)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(score):
    """Far from zero both ways, the type's lowest value, rows of one value."""
    T, E, k = 64, 40, 4
    logits, bias = _logits(T, E, 9, spread=20.0)
    logits[0] = -80.0 - torch.arange(E, device=DEV) / 8
    logits[1] = 60.0 + torch.arange(E, device=DEV) / 8
    logits[2, ::2] = torch.finfo(torch.float32).min
    logits[3] = 0.0
    logits[4] = 1e-30 * torch.arange(E, device=DEV)
    for b in (None, bias):
        cfg = dict(score=score, renormalize=True)
        got = _run(logits, b, k, **cfg)
        assert np.isfinite(got["w"]).all() and got["status"][0] == 0
        _check(logits[5:], b, k, {**got, "idx": got["idx"][5:], "w": got["w"][5:], "P": None}, **cfg)
        idx, w, _ = O.route_grouped(logits[:5].cpu().numpy().astype(np.float64),
                                    None if b is None else b.cpu().numpy().astype(np.float64), k, score)
        np.testing.assert_array_equal(got["idx"][:5], idx)
        # |logit| up to 90: (32 + 4 * 2 * 90) u
        assert (np.abs(got["w"][:5] - w) <= 800 * U * w + 1e-37).all()


@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_logits_a_last_place_apart(score, groups, keep):
    """Scores that fp32 cannot order: all logits of a token are within a few units
    in the last place of one value, so each decision needs the exact formulas.
    Scores differ by 2^-34 of themselves or more there, far above 2^-44. (Sums of
    two such scores need not: groups go by their best expert.)"""
    T, E, k = 96, 128, 6
    g = torch.Generator(device=DEV).manual_seed(11)
    base = torch.linspace(-9.0, 9.0, T, device=DEV).unsqueeze(1)
    steps = torch.randint(0, 40, (T, E), generator=g, device=DEV, dtype=torch.int32)
    logits = (base.contiguous().view(torch.int32) + steps).view(torch.float32)
    bias = 0.25 * torch.randint(0, 2, (E,), generator=g, device=DEV).float()
    for b in (None, bias):
        cfg = dict(score=score, n_groups=groups, topk_groups=keep)
        got = _run(logits, b, k, **cfg)
        assert got["status"][0] == 0
        _check(logits, b, k, got, **cfg)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_and_empty_rows(score):
    T, E, k = 130, 24, 4
    logits, bias = _logits(T, E, 2)
    logits[:, [1, 7, 8, 23]] = -float("inf")
    logits[5] = -float("inf")                     # nothing left
    logits[6, 3:] = -float("inf")                 # fewer than k left
    logits[7, :20] = -float("inf")                # one whole group and a bit
    for G, keep, top in ((1, 1, 1), (6, 3, 2), (6, 2, 1)):
        cfg = dict(score=score, n_groups=G, topk_groups=keep, group_top=top, scale=2.0)
        got = _run(logits, bias, k, **cfg)
        assert got["status"][0] == 0              # -inf is a mask, not an error
        assert (got["w"][5] == 0).all()
        _check(logits, bias, k, got, **cfg)


def test_not_a_number_is_reported_and_masked():
    logits, _ = _logits(9, 16, 3)
    logits[4, 2] = float("nan")
    logits[7, 9] = float("inf")
    got = _run(logits, None, 2, score="sigmoid")
    assert got["status"][0] == moe.DEV_NONFINITE
    assert np.isfinite(got["w"]).all() and 2 not in got["idx"][4] and 9 not in got["idx"][7]
    _check(logits, None, 2, got, score="sigmoid")


def test_empty_batch_and_partial_statistics():
    s = moe.MoeShape.make(0, 64, 8, 2, 64, 1.0)
    e = lambda *n, dt=torch.float32: torch.full(n, 5, dtype=dt, device=DEV)
    routed, P, aux = e(8, dt=torch.int32), e(8), e(1)
    moe.moe_route_grouped(s, moe.RouteConfig.make(), e(1), None, e(1, dt=torch.int32), e(1),
                          routed_counts=routed, P=P, aux=aux, ws=moe.Workspace(s))
    assert routed.sum() == 0 and P.sum() == 0 and aux.sum() == 0
    logits, _ = _logits(100, 8, 1)
    full = _run(logits, None, 2, score="softmax")
    s = moe.MoeShape.make(100, 64, 8, 2, 64, 1.0)
    ws = moe.Workspace(s)
    idx, w, only = e(100, 2, dt=torch.int32), e(100, 2), e(1)
    moe.moe_route_grouped(s, moe.RouteConfig.make(), logits, None, idx, w, aux=only, ws=ws)
    assert only.item() == full["aux"][0]


def test_large_batch_repeats_and_other_stream():
    """More tokens than one pass of the grid; two runs agree bit for bit, and
    so does one on a stream of its own."""
    logits, bias = _logits(40003, 64, 4)
    cfg = dict(score="sigmoid", n_groups=8, topk_groups=4, group_top=2, scale=2.5)
    a = _run(logits, bias, 6, **cfg)
    b = _run(logits, bias, 6, **cfg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = _run(logits, bias, 6, **cfg)
    for n in ("idx", "w", "routed", "P", "aux"):
        assert np.array_equal(a[n], b[n]) and np.array_equal(a[n], c[n]), n
    _check(logits[:3000], bias, 6, {**a, "idx": a["idx"][:3000], "w": a["w"][:3000], "P": None}, **cfg)


# -------------------------------------------------------------- gradient ----

def _bwd(logits, idx, gw, ga=None, routed=None, **cfg):
    T, E = logits.shape
    s = moe.MoeShape.make(T, 64, E, idx.shape[1], 64, 1.0)
    grad = torch.full((T, E), float("nan"), device=DEV)
    moe.moe_route_grouped_bwd(s, moe.RouteConfig.make(**cfg), logits, idx, gw, grad, grad_aux=ga,
                              routed_counts=routed)
    torch.cuda.synchronize()
    return grad.cpu().numpy()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (5, 1, 1), (67, 12, 3), (513, 16, 2), (100, 60, 6),
                                   (300, 64, 8), (129, 128, 1), (77, 255, 7), (256, 256, 8)])
def test_gradient(T, E, k, score, renorm):
    logits, _ = _logits(T, E, T)
    got = _run(logits, None, k, stats=True, score=score)
    idx = torch.from_numpy(got["idx"]).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    gw = torch.randn(T, k, generator=g, device=DEV)
    routed = torch.from_numpy(got["routed"]).to(DEV)
    for aux in (None, 0.5 * T):
        ga = None if aux is None else torch.full((1,), aux, device=DEV)
        mine = _bwd(logits, idx, gw, ga, None if aux is None else routed, score=score,
                    renormalize=renorm, scale=1.5)
        l = logits.cpu().numpy().astype(np.float64)
        ref = O.route_grouped_grad(l, got["idx"].astype(np.int64), gw.cpu().numpy().astype(np.float64),
                                   score, renorm, 1.5, 0.0 if aux is None else aux,
                                   None if aux is None else got["routed"])
        spread = 2 * np.abs(l).max()
        size = 1.5 * np.abs(gw.cpu().numpy()).max() + (0 if aux is None else 0.5 * E / k)
        assert np.abs(mine - ref).max() <= 2 * (48 + 4 * spread) * U * size


def test_gradient_of_masked_and_bad_indices():
    T, E, k = 40, 16, 3
    logits, _ = _logits(T, E, 8)
    logits[:, 5] = -float("inf")
    logits[3] = -float("inf")
    got = _run(logits, None, k, score="softmax")
    idx = torch.from_numpy(got["idx"]).to(DEV)
    gw = torch.ones(T, k, device=DEV) * torch.arange(1, k + 1, device=DEV)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            grad = _bwd(logits, idx, gw, score=score, renormalize=renorm)
            assert np.isfinite(grad).all()
            assert (grad[:, 5] == 0).all() and (grad[3] == 0).all()
    bad = idx.clone()
    bad[0, 1], bad[1, 0] = -1, E
    grad = _bwd(logits, bad, gw, score="sigmoid", renormalize=False)
    whole = _bwd(logits, idx, gw, score="sigmoid", renormalize=False)
    for t, j in ((0, 1), (1, 0)):
        whole[t, got["idx"][t, j]] = 0
    assert np.array_equal(grad, whole)


def test_forward_and_gradient_in_a_graph():
    T, E, k = 200, 64, 6
    logits, bias = _logits(T, E, 6)
    s = moe.MoeShape.make(T, 64, E, k, 64, 1.0)
    ws, cfg = moe.Workspace(s), moe.RouteConfig.make("sigmoid", 8, 3, 2)
    idx = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    w = torch.zeros(T, k, device=DEV)
    routed = torch.zeros(E, dtype=torch.int32, device=DEV)
    P, aux = torch.zeros(E, device=DEV), torch.zeros(1, device=DEV)
    gw, ga = torch.randn(T, k, device=DEV), torch.ones(1, device=DEV)
    grad = torch.zeros(T, E, device=DEV)

    def step():
        moe.moe_route_grouped(s, cfg, logits, bias, idx, w, routed_counts=routed, P=P, aux=aux, ws=ws)
        moe.moe_route_grouped_bwd(s, cfg, logits, idx, gw, grad, grad_aux=ga, routed_counts=routed)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    logits.copy_(_logits(T, E, 7)[0])
    graph.replay()
    torch.cuda.synchronize()
    replay = [t.clone() for t in (idx, w, routed, P, aux, grad)]
    step()
    torch.cuda.synchronize()
    for a, b in zip(replay, (idx, w, routed, P, aux, grad)):
        assert torch.equal(a, b)
