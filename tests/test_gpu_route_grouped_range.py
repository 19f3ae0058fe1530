"""Statistics and gradient of grouped routing where logits are far from zero, or
all at the type's lowest value, against the float64 oracle.

Tolerances count fp32 roundings (u = 2^-24). A share p = s / sum s has the
rounding of exp's argument, 1.5 |d| u for a difference d of logits (or a logit),
and under 48 u for the exponential, sums and divisions; 1 - s has the same bound
relative to itself."""
import numpy as np
import pytest
import torch

import top_routing_expert_gb300 as moe
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
LOWEST = np.finfo(np.float32).min


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.load_library()


def _statistics(l, k, score, bias=None, **cfg):
    T, E = l.shape
    x = torch.from_numpy(np.ascontiguousarray(l, np.float32)).to(DEV)
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).to(DEV)
    s = moe.MoeShape.make(T, 64, E, k, 64, 1.0)
    idx = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    w, P, aux = torch.zeros(T, k, device=DEV), torch.zeros(E, device=DEV), torch.zeros(1, device=DEV)
    routed = torch.zeros(E, dtype=torch.int32, device=DEV)
    moe.moe_route_grouped(s, moe.RouteConfig.make(score, **cfg), x, b, idx, w, routed_counts=routed,
                          P=P, aux=aux, ws=moe.Workspace(s))
    torch.cuda.synchronize()
    return tuple(t.cpu().numpy().astype(np.float64) for t in (idx, w, routed, P, aux))


def _gradient(l, idx, gw, score, renormalize, scale=1.0, grad_aux=None, routed=None):
    T, E = l.shape
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a, t)).to(DEV)
    s = moe.MoeShape.make(T, 64, E, idx.shape[1], 64, 1.0)
    grad = torch.full((T, E), float("nan"), device=DEV)
    moe.moe_route_grouped_bwd(s, moe.RouteConfig.make(score, renormalize=renormalize, scale=scale),
                              dev(l, np.float32), dev(idx, np.int32), dev(gw, np.float32), grad,
                              grad_aux=None if grad_aux is None else dev([grad_aux], np.float32),
                              routed_counts=None if routed is None else dev(routed, np.int32))
    torch.cuda.synchronize()
    return grad.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("E", [6, 20, 32, 100, 200, 255, 256])
def test_rows_at_the_lowest_value(E):
    """Softmax over E equal logits is 1 / E, the type's lowest value among them;
    experts that fill a vector up past E take no part."""
    for T in (3, (1 << 19) // E + 7):
        rng = np.random.default_rng(E)
        l = rng.standard_normal((T, E)).astype(np.float32)
        l[: (T + 1) // 2] = LOWEST
        k = min(4, E)
        idx, w, routed, P, aux = _statistics(l, k, "softmax")
        p = O.grouped_scores(l.astype(np.float64), "softmax")
        want = p.mean(axis=0)
        # a lane sums at most T / 500 tokens and blocks add up in a tree
        tol = (48 + 12 + T / 500 + 64) * U
        assert (np.abs(P - want) <= tol * want).all()
        f = np.bincount(idx.astype(np.int64).ravel(), minlength=E) / (T * k)
        assert abs(aux[0] - E * (f * want).sum()) <= 2 * tol * aux[0]
        assert (idx[: (T + 1) // 2] == np.arange(k)).all()


@pytest.mark.parametrize("E", [8, 20, 64, 100, 200])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_of_rows_at_the_lowest_value(E, renormalize):
    T, k = 37, 4
    rng = np.random.default_rng(E)
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[::2] = LOWEST
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    gw = rng.standard_normal((T, k)).astype(np.float32)
    routed = rng.integers(0, 9, E)
    for ga in (None, 3.0):
        mine = _gradient(l, idx, gw, "softmax", renormalize, 1.5, ga, None if ga is None else routed)
        ref = O.route_grouped_grad(l.astype(np.float64), idx, gw.astype(np.float64), "softmax",
                                   renormalize, 1.5, 0.0 if ga is None else ga,
                                   None if ga is None else routed)
        # every factor of a term is below 1 but these two
        size = 1.5 * np.abs(gw).max() + (0 if ga is None else ga * E / T * routed.max() / (T * k))
        assert np.abs(mine - ref).max() <= 2 * (48 + 4 * 8) * U * size
        # p is 1 / E on those rows, and so is the largest gradient's share
        assert np.abs(mine[::2] - ref[::2]).max() <= 2 * (48 + 4 * 8) * U * size * (1.0 if renormalize else 4.0 / E)


LOW = (-39.0, -41.0, -62.0, -80.0, -86.0, -95.0, -200.0, -600.0)


@pytest.mark.parametrize("E", [6, 32, 100, 256])
def test_shares_of_small_sigmoid_scores(E):
    """P and the balance loss take ratios of scores, which hold where the scores
    themselves are below fp32's smallest value."""
    for T in (len(LOW), (1 << 19) // E + 7):
        rng = np.random.default_rng(E)
        l = (np.resize(LOW, T)[:, None] + 2.0 * rng.standard_normal((T, E))).astype(np.float32)
        k = 3
        for bias in (None, 0.1 * rng.standard_normal(E)):
            idx, w, routed, P, aux = _statistics(l, k, "sigmoid", bias)
            b = None if bias is None else bias.astype(np.float32).astype(np.float64)
            wi, ww, s = O.route_grouped(l[:64].astype(np.float64), b, k, "sigmoid")
            assert (idx[:64] == wi).all()
            s = O.grouped_scores(l.astype(np.float64), "sigmoid")
            want = (s / s.sum(axis=1, keepdims=True)).mean(axis=0)
            # differences of logits within a row: under 24; exp(l) of l itself: under 64
            tol = (48 + 1.5 * 64 + T / 500 + 64) * U
            assert (np.abs(P - want) <= tol * want).all()
            assert abs(aux[0] - E * (routed / (T * k) * want).sum()) <= 2 * tol * aux[0]


@pytest.mark.parametrize("E", [8, 20, 64, 200])
def test_balance_gradient_of_small_sigmoid_scores(E):
    T, k = 3 * len(LOW), 2
    rng = np.random.default_rng(E)
    l = (np.resize(LOW, T)[:, None] + 2.0 * rng.standard_normal((T, E))).astype(np.float32)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    gw = np.zeros((T, k), np.float32)
    routed = rng.integers(0, 9, E)
    ga = float(T)
    ref = O.route_grouped_grad(l.astype(np.float64), idx, gw.astype(np.float64), "sigmoid", True, 1.0, ga, routed)
    mine = _gradient(l, idx, gw, "sigmoid", True, 1.0, ga, routed)
    s = O.grouped_scores(l.astype(np.float64), "sigmoid")
    p = s / s.sum(axis=1, keepdims=True)
    h = ga * E / T * routed / (T * k)
    # p_e (h_e - sum p h): each p to (48 + 1.5 * 64) u, and the difference's own terms
    tol = 2 * (48 + 1.5 * 64) * U * p * (h + (p * h).sum(axis=1, keepdims=True))
    assert (np.abs(mine - ref) <= tol + 1e-37).all()


@pytest.mark.parametrize("E", [8, 20, 64, 256])
@pytest.mark.parametrize("masked", [False, True])
def test_balance_gradient_of_large_sigmoid_scores(E, masked):
    """The slope s (1 - s) of scores next to 1 to a few roundings of itself, not
    of s; logits to both sides in one row."""
    T, k = 120, 2
    rng = np.random.default_rng(E)
    l = np.resize([2.0, 6.0, 10.0, 15.0, 18.0, 30.0, 60.0], T)[:, None] + rng.standard_normal((T, E))
    l[5::7] *= np.where(rng.random((len(l[5::7]), E)) < 0.5, -1.0, 1.0)
    l[6::14, 0] = -300.0
    l[3::14, 1] = 300.0
    l = l.astype(np.float32)
    if masked:
        l[::2, 3] = -np.inf
        l[4, 4] = np.nan
        l[11] = -np.inf
        l[13, 5] = LOWEST
    idx = np.tile([0, 1], (T, 1))
    gw = np.zeros((T, k), np.float32)
    routed = rng.integers(1, 9, E)
    ga = float(T)
    mine = _gradient(l, idx, gw, "sigmoid", True, 1.0, ga, routed)
    x = l.astype(np.float64)
    ok = np.isfinite(x)
    x = np.where(ok, x, 0.0)
    t = np.exp(-np.abs(x))
    s = np.where(ok, np.where(x >= 0, 1.0, t) / (1.0 + t), 0.0)
    rest = np.where(x >= 0, t, 1.0) / (1.0 + t)               # 1 - s
    total = s.sum(axis=1, keepdims=True)
    p = np.divide(s, total, out=np.zeros_like(s), where=total > 0)
    h = ga * E / T * routed / (T * k)
    ph = (p * h).sum(axis=1, keepdims=True)
    ref = p * rest * (h - ph)
    # p and 1 - s to (48 + 1.5 |l|) u of themselves, sum p h to (48 + 1.5 max |l|) u where p counts
    tol = 4 * (48 + 1.5 * np.minimum(np.abs(x), 100.0)) * U * p * rest * (h + ph)
    assert (np.abs(mine - ref) <= tol + 1e-37).all()


@pytest.mark.parametrize("E,k", [(16, 3), (100, 8), (255, 5)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_slots_that_contribute_nothing(E, k, score):
    """Whatever gradient stands in the slot of a masked expert or of an index outside
    the experts: the token's others are as if it were 0."""
    T = 70
    rng = np.random.default_rng(k)
    l = rng.standard_normal((T, E)).astype(np.float32)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    gw = rng.standard_normal((T, k)).astype(np.float32)
    l[np.arange(0, T, 3), idx[::3, 0]] = -np.inf
    idx[1::3, 1] = np.where(np.arange(len(idx[1::3])) % 2 == 0, -1, E)
    zero, bad = gw.copy(), gw.copy()
    for x, v in ((zero, (0.0, 0.0)), (bad, (np.nan, np.inf))):
        x[::3, 0], x[1::3, 1] = v
    routed = rng.integers(0, 9, E)
    for renormalize in (True, False):
        for ga in (None, 2.0):
            one, other = (_gradient(l, idx, g, score, renormalize, 1.5, ga, None if ga is None else routed)
                          for g in (zero, bad))
            assert np.isfinite(one).all() and np.array_equal(one, other)


def test_weights_of_scores_below_fp32_beside_larger_ones():
    """Renormalised sigmoid weights are ratios to a few roundings, also of a score that
    fp32 does not hold to one that it does; and so is their gradient."""
    T, E, k = 200, 16, 5
    rng = np.random.default_rng(4)
    l = (-95.0 + 4.0 * rng.standard_normal((T, E))).astype(np.float32)
    l[:, 3] = np.resize([-12.0, -25.0, -33.0, -39.0, -41.0, -70.0], T)
    idx, w, _, _, _ = _statistics(l, k, "sigmoid")
    want, ww, s = O.route_grouped(l.astype(np.float64), None, k, "sigmoid")
    assert (idx == want).all() and ww.min() > 0
    # ratios below fp32's smallest value (a logit 87 below the largest) are 0
    tol = (48 + 1.5 * 120) * U
    assert (np.abs(w - ww) <= tol * ww + 2.0 ** -126).all()
    gw = rng.standard_normal((T, k)).astype(np.float32)
    mine = _gradient(l, want, gw, "sigmoid", True)
    q = ww[:, :, None] * (gw[:, :, None] - (ww * gw).sum(axis=1)[:, None, None])
    mag = ww * (np.abs(gw) + (ww * np.abs(gw)).sum(axis=1, keepdims=True))
    rest = 1.0 / (1.0 + np.exp(np.take_along_axis(l.astype(np.float64), want, axis=1)))
    got = np.take_along_axis(mine, want, axis=1)
    assert (np.abs(got - q[:, :, 0] * rest) <= 3 * tol * mag + 2.0 ** -126).all()
