"""The step between two blocks and its gradient on the GPU, against float64.

Every value is an fp32 expression of bf16 inputs, rounded once. Sums run over at
most 8 rows, then 32 values a thread, 5 shuffles and 16 warps, fewer than 64
additions deep, so a sum is within 2^-18 of its terms' magnitudes; reciprocal
roots and products add a few 2^-23. With A the same expression over magnitudes,
an output's error is half a step of its type plus 2^-16 A in the forward (two
such sums at most feed a value) and 2^-15 A in the gradient (three). Sums over
tokens add T terms to at most 1216 partial sums in order, T / 1216 + 1216 / 8 + 8
deep or T where fewer: 2^-24 times that more."""
import numpy as np
import pytest
import torch

import top_routing_expert_gb300 as moe
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.load_library()


def _f64(t):
    return None if t is None else t.float().cpu().numpy().astype(np.float64)


def _make(T, H, k, seed, experts=True, vectors=True, drop=0.2, extra=3):
    g = torch.Generator().manual_seed(seed)
    bf = lambda *s, std=1.0: (std * torch.randn(s, generator=g)).to(torch.bfloat16)
    v = {"residual": bf(T, H), "g_out": bf(T, H), "g_xn": bf(T, H), "h": bf(T, H, std=1.5)}
    rows = T * k + extra
    v["y"] = bf(rows, H, std=0.5)
    v["dest"] = v["w"] = None
    if experts:
        # dropped slots (-1), and rows outside the buffer, which are no rows either
        dest = torch.randperm(rows, generator=g)[:T * k].to(torch.int32)
        gone = torch.rand(T * k, generator=g) < drop
        dest[gone] = -1
        if T * k > 6:
            dest[5], gone[5] = rows, True
        named = torch.zeros(rows, dtype=torch.bool)
        named[dest[~gone].long()] = True
        v["y"][~named] = float("nan")          # rows that no slot names are not read
        v["dest"] = dest.view(T, k)
        v["w"] = torch.randn(T, k, generator=g)
        v["w"][gone.view(T, k)] = float("nan")
    v["post"] = torch.randn(H, generator=g) if vectors else None
    v["pre"] = torch.randn(H, generator=g) if vectors else None
    v["gate"] = torch.randn(T, generator=g) if vectors else None
    return v


def _dev(v):
    return {n: None if t is None else t.to(DEV) for n, t in v.items()}


def _oracle_w(v):
    return None if v["w"] is None else np.nan_to_num(_f64(v["w"]))


def _dest(v):
    return None if v["dest"] is None else v["dest"].numpy()


def _close(got, ref, A, factor, dtype, what):
    tol = torch.finfo(dtype).eps / 2 * np.abs(ref) + factor * A + 1e-37
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), what
    assert (err <= tol).all(), (what, np.unravel_index(np.argmax(err - tol), err.shape),
                                (err / tol).max())


WIDTHS = [64, 192, 256, 448, 960, 1024, 1408, 2048, 2816, 4096, 7168, 8192, 8256, 14336, 16384]
SHAPES = [(T, H, k) for H in WIDTHS for T, k in ((1, 2), (5, 1), (37, 8))] + [
    (3, 2048, 1), (9, 512, 3),                 # 48 KB of staged rows and weights, and next to it
    (700, 256, 2), (1500, 64, 4), (333, 4096, 2), (1300, 2048, 6), (2501, 192, 3)]


def _forward(cfg, d, xn=True, out=True, y=True, inplace=False):
    T, H = d["residual"].shape
    o = d["residual"] if inplace else torch.full((T, H), 7.0, dtype=torch.bfloat16, device=DEV)
    x = torch.full((T, H), 7.0, dtype=torch.bfloat16, device=DEV) if xn else None
    moe.moe_block_norm(cfg, d["residual"], d["y"] if y else None, o if out else None, xn=x,
                       dest_row=d["dest"] if y else None, topk_w=d["w"] if y else None,
                       post_weight=d["post"], gate=d["gate"], pre_weight=d["pre"])
    return o, x


@pytest.mark.parametrize("T,H,k", SHAPES)
@pytest.mark.parametrize("post_norm,vectors", [(True, True), (False, True), (True, False)])
def test_forward(T, H, k, post_norm, vectors):
    v = _make(T, H, k, T + H + k, experts=True, vectors=vectors)
    cfg = moe.BlockConfig.make(post_norm=post_norm, residual_scale=0.75, eps=EPS)
    out, xn = _forward(cfg, _dev(v))
    args = (_f64(v["post"]), _f64(v["gate"]), _f64(v["pre"]), post_norm, 0.75, EPS)
    y, w, dest = np.nan_to_num(_f64(v["y"])), _oracle_w(v), _dest(v)
    want, want_x = O.block_norm(_f64(v["residual"]), y, dest, w, *args)
    # magnitudes: the norm's factor is that of the signed sum
    rows, kept = O._token_rows(y, dest, T, k)
    ww = np.where(kept, w, 0)
    c = np.einsum("tk,tkh->th", ww, rows)
    rc = 1 / np.sqrt((c * c).mean(1, keepdims=True) + EPS) if post_norm else 1.0
    A = np.einsum("tk,tkh->th", np.abs(ww), np.abs(rows)) * rc
    for t, n in ((args[0], 1), (args[1], 0)):
        if t is not None:
            A = A * np.abs(t if n else t[:, None])
    A = A + 0.75 * np.abs(_f64(v["residual"]))
    _close(_f64(out), want, A, 2.0 ** -16, torch.bfloat16, "out")
    r = 1 / np.sqrt((want * want).mean(1, keepdims=True) + EPS)
    A = (A * r + np.abs(want) * r) * (1.0 if args[2] is None else np.abs(args[2]))
    _close(_f64(xn), want_x, A, 2.0 ** -16, torch.bfloat16, "xn")


@pytest.mark.parametrize("T,H", [(1, 64), (9, 1024), (130, 4096), (3, 16384)])
def test_forward_forms(T, H):
    """Without experts, without a block, one output or the other, in place."""
    v = _make(T, H, 1, H, experts=False)
    d = _dev(v)
    cfg = moe.BlockConfig.make(residual_scale=1.0, eps=EPS)
    out, xn = _forward(cfg, d)
    want, want_x = O.block_norm(_f64(v["residual"]), _f64(v["y"]), None, None, _f64(v["post"]),
                                _f64(v["gate"]), _f64(v["pre"]), True, 1.0, EPS)
    scale = np.abs(want).max(1, keepdims=True)
    _close(_f64(out), want, scale, 2.0 ** -16, torch.bfloat16, "out")
    only = _forward(cfg, d, xn=False)[0]
    assert torch.equal(out, only)
    untouched, x2 = _forward(cfg, d, out=False)
    assert torch.equal(xn, x2) and (untouched == 7).all()
    # no block output: the norm alone, as the first block begins
    o, x = _forward(cfg, d, y=False)
    assert torch.equal(o, d["residual"])
    _, want_x = O.block_norm(_f64(v["residual"]), None, None, None, None, None, _f64(v["pre"]), True,
                             1.0, EPS)
    _close(_f64(x), want_x, np.abs(want_x), 2.0 ** -16, torch.bfloat16, "xn alone")
    residual = d["residual"].clone()
    o, x = _forward(cfg, d, inplace=True)
    assert torch.equal(o, out) and torch.equal(x, xn) and not torch.equal(residual, o)


def _backward(cfg, d, skip=(), ws=None):
    T, H = d["h"].shape
    bf = lambda like: torch.full_like(like, 7.0)
    f32 = lambda *s: torch.full(s, 7.0, device=DEV)
    k = 1 if d["dest"] is None else d["dest"].shape[1]
    g = {"g_residual": bf(d["h"]), "g_y": bf(d["y"]) if d["y"] is not None else None,
         "g_w": f32(T, k), "g_post": f32(H), "g_gate": f32(T), "g_pre": f32(H)}
    if d["g_xn"] is None:
        g["g_pre"] = None
    if d["y"] is None:
        g["g_w"] = g["g_post"] = g["g_gate"] = None
    g = {n: None if n in skip else t for n, t in g.items()}
    moe.moe_block_norm_bwd(cfg, d["h"], d["y"], d["g_out"], g["g_residual"], g["g_y"],
                           grad_xn=d["g_xn"], dest_row=d["dest"], topk_w=d["w"],
                           post_weight=d["post"], gate=d["gate"], pre_weight=d["pre"],
                           grad_topk_w=g["g_w"], grad_post=g["g_post"], grad_gate=g["g_gate"],
                           grad_pre=g["g_pre"], ws=ws or moe.BlockWorkspace(T, H))
    return g


def _check_backward(v, got, post_norm, scale, eps=EPS):
    y = None if v["y"] is None else np.nan_to_num(_f64(v["y"]))
    args = (_f64(v["h"]), y, _dest(v), _oracle_w(v), _f64(v["post"]), _f64(v["gate"]),
            _f64(v["pre"]), post_norm, scale, eps, _f64(v["g_out"]), _f64(v["g_xn"]))
    want, mag = O.block_norm_grad(*args), O.block_norm_grad_magnitude(*args)
    T = len(args[0])
    for n, t in got.items():
        if t is None:
            continue
        ref, A, val = want[n], mag[n], _f64(t)
        factor = 2.0 ** -15
        if n in ("g_post", "g_pre"):
            factor += 2.0 ** -24 * min(T, T / 1216 + 160)
        if n == "g_y":
            kept = ~np.isnan(ref[:, 0])
            assert (val[~kept] == 7).all()     # rows that no slot names stay as they were
            val, ref, A = val[kept], ref[kept], A[kept]
        _close(val, ref, A, factor, t.dtype, n)


@pytest.mark.parametrize("T,H,k", SHAPES)
@pytest.mark.parametrize("post_norm,vectors", [(True, True), (False, True), (True, False)])
def test_backward(T, H, k, post_norm, vectors):
    v = _make(T, H, k, T + H + k + 1, vectors=vectors)
    cfg = moe.BlockConfig.make(post_norm=post_norm, residual_scale=0.75, eps=EPS)
    _check_backward(v, _backward(cfg, _dev(v)), post_norm, 0.75)


@pytest.mark.parametrize("T,H", [(1, 64), (9, 1024), (130, 4096), (3, 16384)])
def test_backward_forms(T, H):
    cfg = moe.BlockConfig.make(residual_scale=2.0, eps=EPS)
    v = _make(T, H, 1, H, experts=False)
    d = _dev(v)
    full = _backward(cfg, d)
    _check_backward(v, full, True, 2.0)
    for gone in ("g_out", "g_xn"):             # one of the two gradients alone
        w = v | {gone: None}
        _check_backward(w, _backward(cfg, _dev(w)), True, 2.0)
    w = v | {"y": None, "gate": None, "post": None}   # the norm alone
    _check_backward(w, _backward(cfg, _dev(w)), True, 2.0)
    # gradients that are not asked for change no others
    for skip in (("g_post", "g_pre"), ("g_w", "g_gate"), ("g_residual",), ("g_y",)):
        part = _backward(cfg, d, skip)
        for n, t in part.items():
            assert t is None or torch.equal(t, full[n]), (skip, n)
    # in place of grad_out
    go = d["g_out"].clone()
    moe.moe_block_norm_bwd(cfg, d["h"], d["y"], go, go, None, grad_xn=d["g_xn"],
                           post_weight=d["post"], gate=d["gate"], pre_weight=d["pre"])
    assert torch.equal(go, full["g_residual"])


def test_tokens_without_rows():
    """Every slot dropped: the residual passes alone, and nothing is not a number."""
    v = _make(6, 256, 2, 1)
    v["dest"][:] = -1
    v["y"][:] = float("nan")
    v["w"][:] = float("nan")
    d = _dev(v)
    cfg = moe.BlockConfig.make(eps=EPS)
    out, xn = _forward(cfg, d)
    assert torch.equal(out, d["residual"]) and torch.isfinite(xn).all()
    g = _backward(cfg, d)
    assert (g["g_w"] == 0).all() and (g["g_gate"] == 0).all() and (g["g_post"] == 0).all()
    assert (g["g_y"] == 7).all() and torch.isfinite(g["g_residual"]).all()
    v["y"] = v["y"][:0]                        # a block whose buffer holds no rows
    out2, _ = _forward(cfg, _dev(v))
    assert torch.equal(out2, out)


def test_no_tokens():
    cfg = moe.BlockConfig.make()
    e = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    moe.moe_block_norm(cfg, e, e, e, xn=e)
    post, pre = (torch.full((128,), 7.0, device=DEV) for _ in range(2))
    moe.moe_block_norm_bwd(cfg, e, e, e, e, e, grad_xn=e, grad_post=post, grad_pre=pre,
                           ws=moe.BlockWorkspace(0, 128))
    assert (post == 0).all() and (pre == 0).all()


def test_against_differences():
    """Every gradient's product with a random direction against central
    differences of the float64 forward."""
    T, H, k = 12, 192, 3
    v = _make(T, H, k, 11, drop=0.3)
    cfg = moe.BlockConfig.make(residual_scale=0.5, eps=1e-3)
    d = _dev(v)
    out, _ = _forward(cfg, d)
    d["h"] = out
    got = _backward(cfg, d)
    y, dest, w = np.nan_to_num(_f64(v["y"])), _dest(v), _oracle_w(v)
    names = {"residual": "g_residual", "y": "g_y", "w": "g_w", "post": "g_post", "gate": "g_gate",
             "pre": "g_pre"}
    at = {"residual": _f64(v["residual"]), "y": y, "w": w, "post": _f64(v["post"]),
          "gate": _f64(v["gate"]), "pre": _f64(v["pre"])}

    def loss(a):
        o, x = O.block_norm(a["residual"], a["y"], dest, a["w"], a["post"], a["gate"], a["pre"], True,
                            0.5, 1e-3)
        return (o * _f64(v["g_out"])).sum() + (x * _f64(v["g_xn"])).sum()

    rng = np.random.default_rng(2)
    named = np.zeros(len(y), bool)
    kept = (dest >= 0) & (dest < len(y))
    named[dest[kept]] = True
    for n, g in names.items():
        grad = _f64(got[g])
        if n == "y":
            grad = np.where(named[:, None], grad, 0)
        step = rng.standard_normal(at[n].shape)
        num = (loss(at | {n: at[n] + 1e-5 * step}) - loss(at | {n: at[n] - 1e-5 * step})) / 2e-5
        # the stream is stored in bf16 (2^-9 of each value on average below its
        # half step), as are the outputs: errors of random sign, 4 times the 2-norm
        tol = 4 * 2.0 ** -8 * np.linalg.norm(grad * step) * 2 ** 0.5
        assert abs((grad * step).sum() - num) <= tol, (n, (grad * step).sum(), num, tol)


def test_streams_graphs_and_repeats():
    v = _make(300, 1408, 4, 3)
    d = _dev(v)
    cfg = moe.BlockConfig.make(eps=EPS)
    ws = moe.BlockWorkspace(300, 1408)

    def both():
        return list(_forward(cfg, d)) + [t for t in _backward(cfg, d, ws=ws).values()]

    first = both()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        second = both()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = both()
    for _ in range(2):
        for t in third:
            t.zero_()
        d["g_out"].copy_(v["g_out"])
        third[3].fill_(7.0)                    # rows that no slot names are not written
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(first, second, third):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_far_rows():
    """Rows whose elements lie past 2^31 in y and in the stream."""
    H, k = 16384, 2
    T = (1 << 31) // H + 3                     # 131075 tokens: the last ones past 2^31 elements
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    g = torch.Generator(device=DEV).manual_seed(1)
    dest = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    rows = T + 5
    last = torch.arange(T - 4, T, device=DEV)
    dest[last, 0] = torch.tensor([rows - 1, rows - 3, rows - 4, 0], dtype=torch.int32, device=DEV)
    y = torch.zeros(rows, H, dtype=torch.bfloat16, device=DEV)
    y[-8:] = torch.randn(8, H, generator=g, device=DEV).to(torch.bfloat16)
    y[0] = 1
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[-4:] = torch.randn(4, H, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.full((T, k), 0.5, device=DEV)
    out, xn = torch.empty_like(x), torch.empty_like(x)
    cfg = moe.BlockConfig.make(post_norm=False)
    moe.moe_block_norm(cfg, x, y, out, xn=xn, dest_row=dest, topk_w=w)
    want = x[-4:].float() + 0.5 * y[dest[last, 0].long()].float()
    assert torch.equal(out[-4:], want.to(torch.bfloat16))
    assert not out[:-4].any() and not xn[:-4].any()
    gy = torch.zeros_like(y)
    gw = torch.empty(T, k, device=DEV)
    moe.moe_block_norm_bwd(cfg, out, y, x, xn, gy, dest_row=dest, topk_w=w, grad_topk_w=gw)
    assert torch.equal(xn, x)
    assert torch.equal(gy[dest[last, 0].long()], (0.5 * x[-4:].float()).to(torch.bfloat16))
    ref = (x[-4:].double() * y[dest[last, 0].long()].double()).sum(1)
    size = (x[-4:].double() * y[dest[last, 0].long()].double()).abs().sum(1)
    assert ((gw[-4:, 0].double() - ref).abs() <= 2.0 ** -18 * size).all()


def test_device_refusals():
    """Strided, mistyped, misaligned and undersized tensors are refused before a launch."""
    cfg = moe.BlockConfig.make()
    bf = lambda *n: torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    x, y, out = bf(4, 64), bf(8, 64), torch.full((4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    dest = torch.arange(8, dtype=torch.int32, device=DEV).view(4, 2)
    w, gp = torch.ones(4, 2, device=DEV), torch.zeros(64, device=DEV)
    fwd, bwd = moe.moe_block_norm, moe.moe_block_norm_bwd
    for call in (lambda: fwd(cfg, bf(4, 128)[:, :64], y, out, dest_row=dest, topk_w=w),
                 lambda: fwd(cfg, x, y.float(), out, dest_row=dest, topk_w=w),
                 lambda: fwd(cfg, x, y, out, dest_row=dest.long(), topk_w=w),
                 lambda: fwd(cfg, x, y, out, dest_row=dest, topk_w=w.double()),
                 lambda: fwd(cfg, x, y, out, dest_row=dest.T.contiguous().T, topk_w=w),
                 lambda: bwd(cfg, x, y, x.half(), out, None, dest_row=dest, topk_w=w),
                 lambda: bwd(cfg, x, None, x, out, y)):
        with pytest.raises(ValueError):
            call()
    shifted = bf(4 * 64 + 8)[4:4 + 4 * 64].view(4, 64)
    for code, call in ((5, lambda: fwd(cfg, shifted, y, out, dest_row=dest, topk_w=w)),
                       (2, lambda: fwd(cfg, x, y[:3], out)),
                       (1, lambda: fwd(cfg, x, y, None, dest_row=dest, topk_w=w)),
                       (1, lambda: bwd(cfg, x, y, x, out, None, dest_row=dest, topk_w=w, grad_post=gp)),
                       (1, lambda: bwd(cfg, x, y, None, out, None, dest_row=dest, topk_w=w)),
                       (4, lambda: bwd(cfg, x, y, x, out, None, dest_row=dest, topk_w=w, grad_post=gp,
                                       ws=moe.BlockWorkspace(0, 64)))):
        with pytest.raises(moe.MoeError) as e:
            call()
        assert e.value.code == code
    assert (out == 7).all()
