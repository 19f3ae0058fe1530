"""Grouped routing of batches that take the long form of the kernel (more than 2^19
logits), every list length and lane count of it, over more than one pass of the
grid, all tokens against float64.

Weights and P are within (32 + 4 spread) u of themselves (u = 2^-24, spread the
largest difference of logits), P with T / 500 + 64 u more for its sums: a lane adds
at most T / 500 tokens in sequence. Tokens whose kept and left groups differ in a sum
of two by less than 2^-40 of the values are not compared: the choice is promised for
exponentials to 2^-44, and sums that are equal but for fp64's last roundings, as
s(x) + s(-x) is for every x, have no order there."""
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


def _oracle(l, bias, k, score, G, keep, top, renormalize, scale):
    """O.route_grouped for all tokens at once."""
    T, E = l.shape
    s = O.grouped_scores(l, score)
    c = np.where(np.isfinite(l), s + (0.0 if bias is None else bias[None, :]), -np.inf)
    if G > 1:
        value = -np.sort(-c.reshape(T, G, E // G), axis=2)[:, :, :top].sum(axis=2)
        kept = np.argsort(-value, axis=1, kind="stable")[:, :keep]
        out = np.ones((T, G), bool)
        np.put_along_axis(out, kept, False, axis=1)
        c = np.where(np.repeat(out, E // G, axis=1), np.nan, c)      # after masked ones
    idx = np.argsort(-c, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(s, idx, axis=1)
    if renormalize:
        d = w.sum(axis=1, keepdims=True)
        w = np.divide(w, d, out=np.zeros_like(w), where=d > 0)
    return idx, scale * w, s


def _compare(l, bias, k, score, G=1, keep=1, top=1, renormalize=True, scale=1.0, stats=True,
             same=False):
    """same: groups whose sums are equal have the same two values."""
    T, E = l.shape
    x = torch.from_numpy(l).to(DEV)
    b = None if bias is None else torch.from_numpy(bias).to(DEV)
    s = moe.MoeShape.make(T, 64, E, k, 64, 1.0)
    cfg = moe.RouteConfig.make(score, G, keep, top, renormalize, scale)
    idx = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), float("nan"), device=DEV)
    routed = torch.full((E,), -7, dtype=torch.int32, device=DEV) if stats else None
    P, aux = (torch.full((n,), float("nan"), device=DEV) if stats else None for n in (E, 1))
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    moe.moe_route_grouped(s, cfg, x, b, idx, w, routed_counts=routed, P=P, aux=aux, dev_status=status,
                          ws=moe.Workspace(s))
    torch.cuda.synchronize()
    assert status.item() == 0
    l64 = l.astype(np.float64)
    want, ww, sc = _oracle(l64, None if bias is None else bias.astype(np.float64), k, score, G, keep, top,
                           renormalize, scale)
    got = idx.cpu().numpy()
    told = np.ones(T, bool)
    if G > keep and top == 2:
        c = np.where(np.isfinite(l64), sc + (0.0 if bias is None else bias.astype(np.float64)[None, :]), -np.inf)
        v = -np.sort(-(-np.sort(-c.reshape(T, G, E // G), axis=2)[:, :, :2].sum(axis=2)), axis=1)
        with np.errstate(invalid="ignore"):   # masked groups: the lower index
            gap = np.abs(v[:, keep - 1] - v[:, keep])
            told = ~(gap <= 2.0 ** -40 * np.where(np.isfinite(c), np.abs(c), 0).max(axis=1)) | (same & (gap == 0))
        assert told.mean() > 0.9
    wrong = (got != want).any(axis=1) & told
    assert not wrong.any(), (wrong.sum(), np.nonzero(wrong)[0][:5])
    tol = (32 + 4 * 2 * np.abs(l64[np.isfinite(l64)]).max()) * U
    assert (np.abs(w.cpu().numpy() - ww) <= tol * np.abs(ww) + 1e-37)[told].all()
    if stats:
        n = np.bincount(got.ravel(), minlength=E)
        assert (routed.cpu().numpy() == n).all()
        total = sc.sum(axis=1, keepdims=True)
        p = np.divide(sc, total, out=np.zeros_like(sc), where=total > 0).mean(axis=0)
        tol += (T / 500 + 64) * U
        assert (np.abs(P.cpu().numpy() - p) <= tol * p + 1e-37).all()
        a = E * (n / (T * k) * p).sum()
        assert abs(aux.item() - a) <= 2 * tol * a


def _batch(T, E, seed):
    """Random rows, with ones in between that are on a coarse grid (ties), a few
    units in the last place off it, masked in places, or masked all but one."""
    rng = np.random.default_rng(seed)
    l = rng.standard_normal((T, E)).astype(np.float32)
    l[::9] = np.round(l[::9] * 4) / 4
    near = np.round(l[4::9] * 4) / 4
    l[4::9] = near * (1 + rng.integers(-2, 3, near.shape) * 2.0 ** -23)
    part = l[1::7]
    part[rng.random(part.shape) < 0.3] = -np.inf
    l[1::7] = part
    l[5::1001] = -np.inf
    l[6::1001, 1:] = -np.inf
    return l, (np.round(0.4 * rng.standard_normal(E) * 8) / 8).astype(np.float32)


GROUPS = {24: (4, 2), 32: (8, 3), 60: (6, 3), 64: (8, 4), 100: (10, 4), 128: (8, 3), 255: (5, 2), 256: (8, 4)}
PASS = {24: 77824, 32: 77824, 60: 38912, 64: 38912, 100: 19456, 128: 19456, 255: 9728, 256: 9728}  # tokens


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 2, 3, 4, 6, 8])
@pytest.mark.parametrize("E", sorted(GROUPS))
def test_long_form(E, k, score):
    T = PASS[E] + PASS[E] // 8 + 5
    assert T * E > 1 << 19
    l, bias = _batch(T, E, E + k)
    G, keep = GROUPS[E]
    if k % 2:
        _compare(l, bias, k, score, renormalize=k == 1, scale=2.5, stats=True)
    else:
        _compare(l, bias if k < 8 else None, k, score, G, keep, 2 if k > 2 else 1, True, 1.0, stats=k != 4)


@pytest.mark.parametrize("E,k,T", [(32, 2, 160000), (24, 8, 160000), (64, 4, 160000), (128, 2, 160000), (256, 8, 160000)])
def test_lists_of_doubtful_tokens_fill(E, k, T):
    """Rows of one value leave every token in doubt: more than 64 to a warp."""
    rng = np.random.default_rng(E)
    l = np.repeat(np.round(rng.standard_normal((T, 1)), 1), E, axis=1).astype(np.float32)
    l[::50, 3] += 1.0
    l[::50, 2] -= 1.0
    _compare(l, None, k, "softmax")
    _compare(l, None, k, "sigmoid", 4, 2, 2, same=True)


def test_vectorised_oracle():
    l, bias = _batch(300, 24, 1)
    for G, keep, top in ((1, 1, 1), (4, 2, 2), (6, 3, 1)):
        got = _oracle(l.astype(np.float64), bias.astype(np.float64), 4, "sigmoid", G, keep, top, True, 2.0)
        want = O.route_grouped(l.astype(np.float64), bias.astype(np.float64), 4, "sigmoid", G, keep, top, True, 2.0)
        for a, b in zip(got, want):
            assert np.array_equal(a, b)
