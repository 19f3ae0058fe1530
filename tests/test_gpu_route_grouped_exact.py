"""Where grouped routing's choice hangs on values that fp32 cannot order, or on
values at the ends of fp32's and binary64's ranges: the chosen experts are those
of the float64 oracle, exactly.

The rows are made so that two compared values (single selection values, or group
values that are sums of two) are a few fp32 roundings apart: one logit is solved
for in float64, rounded to fp32 and moved by a few units in the last place. Rows
whose values differ by less than 2^-40 of the largest magnitude in them are left
out (the choice is promised for exponentials to 2^-44)."""
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


def _route(logits, bias, k, stats=True, **cfg):
    l = torch.from_numpy(np.ascontiguousarray(logits, np.float32)).to(DEV)
    b = None if bias is None else torch.from_numpy(np.ascontiguousarray(bias, np.float32)).to(DEV)
    T, E = l.shape
    s = moe.MoeShape.make(T, 64, E, k, 64, 1.0)
    idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), float("nan"), device=DEV)
    routed = torch.full((E,), -7, dtype=torch.int32, device=DEV)
    P, aux = torch.full((E,), float("nan"), device=DEV), torch.full((1,), float("nan"), device=DEV)
    moe.moe_route_grouped(s, moe.RouteConfig.make(**cfg), l, b, idx, w,
                          routed_counts=routed if stats else None, P=P if stats else None,
                          aux=aux if stats else None, ws=moe.Workspace(s))
    torch.cuda.synchronize()
    return tuple(t.cpu().numpy() for t in (idx, w, routed, P, aux))


def _values(l, bias, score):
    return O.grouped_scores(l, score) + (0.0 if bias is None else np.asarray(bias, np.float64)[None, :])


def _close_rows(rng, n, E, score, base, bias, pair):
    """fp32 logits [m, E] whose experts 0 and 1 against 2 and 3 (pair), or 0
    against 2, have nearly equal selection values; the others are lower."""
    l = base - np.abs(rng.standard_normal((n, E))) * 0.02
    l[:, 4:] -= 1.0 + np.abs(rng.standard_normal((n, E - 4)))
    if not pair:
        l[:, [1, 3]] -= 1.0
    l = l.astype(np.float32).astype(np.float64)

    def ahead(x):  # by how much the second side is ahead with logit x of expert 2
        y = l.copy()
        y[:, 2] = x
        c = _values(y, bias, score)
        return c[:, 2] - c[:, 0] + (c[:, 3] - c[:, 1] if pair else 0.0)

    lo, hi = np.full(n, base - 6.0), np.full(n, base + 6.0)
    solved = (ahead(lo) < 0) & (ahead(hi) > 0)
    for _ in range(70):
        mid = 0.5 * (lo + hi)
        up = ahead(mid) > 0
        lo, hi = np.where(up, lo, mid), np.where(up, mid, hi)
    x = lo.astype(np.float32)
    x = (x.view(np.int32) + rng.integers(-2, 3, n).astype(np.int32)).view(np.float32)
    l[:, 2] = x
    c = _values(l, bias, score)
    rel = np.abs(ahead(l[:, 2])) / np.abs(c).max(axis=1)
    return l[solved & (rel > 2.0 ** -40)].astype(np.float32)


def _assert_choice(l, bias, k, score, **cfg):
    idx = _route(l, bias, k, score=score, **cfg)[0]
    b = None if bias is None else np.asarray(bias, np.float32).astype(np.float64)
    want = O.route_grouped(l.astype(np.float64), b, k, score, **cfg)[0]
    wrong = (idx != want).any(axis=1)
    assert not wrong.any(), f"{wrong.sum()} of {len(l)} tokens"


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("base", [-12.0, -6.9, -6.0, -5.0, -3.0, 0.0, 2.0])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_sums_of_two_close(score, base, biased):
    """Groups of two by the sum of both."""
    rng = np.random.default_rng(7)
    top = 0.4 if score == "softmax" else 1.0 / (1.0 + np.exp(-base))
    bias = (top * np.array([0.25, -0.125, 0.0, 0.0625, 0, 0, 0, 0])).astype(np.float32) if biased else None
    l = _close_rows(rng, 12000, 8, score, base, bias, True)
    assert len(l) > 3000
    _assert_choice(l, bias, 2, score, n_groups=4, topk_groups=1, group_top=2)


@pytest.mark.parametrize("E", [8, 40, 64, 128, 200, 256])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_single_values_close(score, E):
    """One expert against another, with biases that differ, in the short and in
    the long form of the kernel."""
    rng = np.random.default_rng(E)
    bias = np.zeros(E, np.float32)
    # a share of the largest score, which E softmax scores of about equal size divide
    z = O.grouped_scores(_close_rows(rng, 8, E, score, -6.9, None, False).astype(np.float64), score).max()
    bias[0], bias[2] = 0.5 * z, -0.25 * z
    for base in (-6.9, 0.5):
        n = (1 << 19) // E * 2
        l = _close_rows(rng, n, E, score, base, bias, False)
        assert len(l) > n // 4
        want = _values(l.astype(np.float64), bias, score).argmax(axis=1)
        for rows in (n, 1500):
            idx = _route(l[:rows], bias, 1, score=score)[0][:, 0]
            assert (idx != want[:rows]).sum() == 0, (base, rows)


@pytest.mark.parametrize("score,lo,hi", [("sigmoid", -6.905, -6.7), ("sigmoid", -6.0, -5.0), ("sigmoid", -2.0, 1.0),
                                         ("softmax", -1.0, 1.0)])
def test_many_sums_of_two_close(score, lo, hi):
    """A million rows of two groups: the few where fp32's errors add up."""
    rng = np.random.default_rng(1)
    n = 1000000
    base = rng.uniform(lo, hi, (n, 1))
    l = (base - np.abs(rng.standard_normal((n, 4))) * 0.01).astype(np.float32).astype(np.float64)

    def ahead(x):
        y = l.copy()
        y[:, 2] = x
        c = _values(y, None, score)
        return c[:, 2] + c[:, 3] - c[:, 0] - c[:, 1]

    a, b = np.full(n, lo - 6.0), np.full(n, hi + 6.0)
    solved = (ahead(a) < 0) & (ahead(b) > 0)
    for _ in range(60):
        mid = 0.5 * (a + b)
        up = ahead(mid) > 0
        a, b = np.where(up, a, mid), np.where(up, mid, b)
    x = a.astype(np.float32)
    l[:, 2] = (x.view(np.int32) + rng.integers(-1, 2, n).astype(np.int32)).view(np.float32)
    c = _values(l, None, score)
    second = c[:, 2] + c[:, 3] > c[:, 0] + c[:, 1]
    keep = solved & (np.abs(ahead(l[:, 2])) > 2.0 ** -40 * c.max(axis=1))
    assert keep.sum() > 0.9 * n
    idx = _route(l[keep], None, 2, stats=False, score=score, n_groups=2, topk_groups=1, group_top=2)[0]
    assert ((idx[:, 0] // 2 == 1) != second[keep]).sum() == 0


def test_two_counterexamples():
    """Found by hand: groups a fp32 rounding apart whose order fp32 reverses."""
    rows = np.array([[-6.8737135, -6.8792887, -6.8786025, -6.8743963],
                     [float.fromhex(h) for h in ("-0x1.ba0076p+2", "-0x1.b9ce5cp+2",
                                                 "-0x1.b9f246p+2", "-0x1.b9dc84p+2")]], np.float32)
    for r in (rows, rows[:, [2, 3, 0, 1]]):
        _assert_choice(r, None, 2, "sigmoid", n_groups=2, topk_groups=1, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("big", [8.0, 1000.0, 1e5])
def test_group_sums_that_cancel(score, big):
    """Biases of opposite signs and far above the scores: a group's sum is much
    smaller than the two values whose fp32 roundings are in it."""
    rng = np.random.default_rng(int(big))
    T, E, G = 20000, 16, 8
    l = rng.standard_normal((T, E)).astype(np.float32)
    bias = np.tile([big, -big], G).astype(np.float32)
    _assert_choice(l, bias, 4, score, n_groups=G, topk_groups=3, group_top=2)
    bias[4:8] = [big, -big + 0.5, big, 0.25]
    _assert_choice(l, bias, 4, score, n_groups=G, topk_groups=3, group_top=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_group_sums_past_fp32(score):
    """Finite biases whose sums are not finite in fp32: they differ from one
    another, and from those of masked groups, all the same."""
    rng = np.random.default_rng(3)
    T, E, G = 500, 16, 8
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[:, 0:2] = -np.inf
    high = np.zeros(E, np.float32)
    high[4:10] = [2e38, 2e38, 3e38, 3e38, 3e38, 2e38]
    low = np.full(E, -3e38, np.float32)
    low[12:] = [-2.5e38, -2.0e38, -3.4e38, -3.4e38]
    for bias in (high, low):
        for keep in (1, 2, 3):
            _assert_choice(l, bias, 2, score, n_groups=G, topk_groups=keep, group_top=2)


def test_choice_where_scores_are_smallest():
    """Softmax differences and sigmoid logits beyond 700: binary64 tells the scores
    apart to exp(-745) and 1 / (1 + exp(709)), and beyond that they are equal."""
    row = np.array([0, -705, -701, -703, -720, -742, -740, -800, -900, -702.5], np.float32)
    rng = np.random.default_rng(0)
    l = np.stack([row[rng.permutation(10)] for _ in range(64)])
    l[::2] += np.float32(3.0)
    l[::3] = np.where(l[::3] == l[::3].max(axis=1, keepdims=True), l[::3], l[::3] - 0.125)
    for k in (3, 8):
        _assert_choice(l, None, k, "softmax")
        _assert_choice(l, np.full(10, 1e-30, np.float32), k, "softmax")
    _assert_choice(l, None, 4, "softmax", n_groups=5, topk_groups=3, group_top=2)
    low = np.array([-700.5, -703, -701, -708.25, -702, -699, -706, -701.5], np.float32)
    s = np.stack([low[rng.permutation(8)] for _ in range(64)])
    for k in (1, 4, 8):
        _assert_choice(s, None, k, "sigmoid")
    _assert_choice(s, None, 2, "sigmoid", n_groups=4, topk_groups=2, group_top=2)
    far = np.tile(np.array([-900, -1000, -800, -1e30], np.float32), (3, 1))
    assert (_route(far, None, 3, score="sigmoid")[0] == [0, 1, 2]).all()   # all are 0
