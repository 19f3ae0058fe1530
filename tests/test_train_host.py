"""The training operators without a GPU: the oracle's formulas against
differences, and the refusals that come before any launch."""
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

def test_gelu_slope_against_differences():
    u = np.linspace(-9, 9, 181)
    h = 1e-5   # central differences: error about h^2 and 2^-52 |gelu| / h
    num = (O.gelu_tanh(u + h) - O.gelu_tanh(u - h)) / (2 * h)
    assert np.abs(num - O.gelu_tanh_slope(u)).max() < 1e-9


def test_weight_gradient_by_hand():
    x, g = np.arange(6.0).reshape(3, 2), np.arange(3.0).reshape(3, 1) + 1
    dW = O.expert_weight_grad(x, g, [0, 2, 2, 3])
    assert dW[0].tolist() == [[0 * 1 + 2 * 2], [1 * 1 + 3 * 2]]
    assert dW[1].tolist() == [[0], [0]] and dW[2].tolist() == [[12], [15]]


@pytest.mark.parametrize("post_norm", [True, False])
@pytest.mark.parametrize("experts", [True, False])
@pytest.mark.parametrize("vectors", [True, False])
def test_block_gradient_against_differences(post_norm, experts, vectors):
    rng = np.random.default_rng(5)
    T, H, k, eps, scale = 4, 6, 3, 1e-3, 0.7
    n = lambda *s: rng.standard_normal(s)
    dest = np.array([[0, 5, -1], [1, 2, 3], [-1, -1, -1], [4, 6, -1]]) if experts else None
    v = {"residual": n(T, H), "y": n(8, H), "w": n(T, k) if experts else None,
         "post": n(H) if vectors else None, "gate": n(T) if vectors else None,
         "pre": n(H) if vectors else None}
    g_out, g_xn = n(T, H), n(T, H)

    def loss(d):
        out, xn = O.block_norm(d["residual"], d["y"], dest, d["w"], d["post"], d["gate"], d["pre"],
                               post_norm, scale, eps)
        return (out * g_out).sum() + (xn * g_xn).sum()

    h, _ = O.block_norm(v["residual"], v["y"], dest, v["w"], v["post"], v["gate"], v["pre"],
                        post_norm, scale, eps)
    grad = O.block_norm_grad(h, v["y"], dest, v["w"], v["post"], v["gate"], v["pre"], post_norm,
                             scale, eps, g_out, g_xn)
    for name, value in v.items():
        if value is None:
            continue
        got = np.nan_to_num(grad["g_" + name])
        num = np.zeros_like(value)
        for i in np.ndindex(value.shape):
            step = np.zeros_like(value)
            step[i] = 1e-5
            num[i] = (loss(v | {name: value + step}) - loss(v | {name: value - step})) / 2e-5
        # a token without rows has c = 0, where 1 / sqrt(eps) is large: still smooth
        assert np.abs(num - got).max() < 1e-7 * max(1.0, np.abs(got).max()), name


# -------------------------------------------------------------- refusals ----

def test_product_refusals(lib):
    P = ctypes.c_void_p
    f, off = P(FAKE), P(FAKE + 8)

    def gemm(E=8, rows=16, K=128, N=128, x=f, o=f, W=f, t=0, epi=0, pre=None, D=f, st=f):
        return lib.moe_expert_gemm(E, rows, K, N, x, o, W, t, epi, pre, D, st, None)

    assert gemm(E=0) == 2 and gemm(N=0) == 2 and gemm(K=0) == 2 and gemm(rows=-1) == 2
    assert gemm(t=2) == 2 and gemm(epi=3) == 2 and gemm(epi=-1) == 2
    assert gemm(E=257) == 3 and gemm(K=96) == 3 and gemm(N=96) == 3 and gemm(N=65600) == 3
    assert gemm(rows=2 ** 31) == 3
    assert gemm(pre=f) == 2                    # nothing to keep without a GELU
    assert gemm(epi=2) == 1                    # its slope needs the kept values
    assert gemm(epi=1, pre=off) == 5
    for name in ("x", "o", "W", "D", "st"):
        assert gemm(**{name: None}) == 1, name
        assert gemm(**{name: off}) == 5, name
    assert gemm(rows=0, x=None, W=None, D=None) == 0

    def dw(E=8, rows=16, K=128, N=128, x=f, g=f, o=f, dW=f, dtype=0, acc=0, st=f):
        return lib.moe_expert_wgrad(E, rows, K, N, x, g, o, dW, dtype, acc, st, None)

    assert dw(E=0) == 2 and dw(N=0) == 2 and dw(K=0) == 2 and dw(rows=-1) == 2
    assert dw(dtype=2) == 2 and dw(acc=2) == 2
    assert dw(dtype=1, acc=1) == 3             # bf16 would round every sum
    assert dw(E=257) == 3 and dw(K=96) == 3 and dw(N=96) == 3 and dw(rows=2 ** 31) == 3
    for name in ("x", "g", "o", "dW", "st"):
        assert dw(**{name: None}) == 1, name
        assert dw(**{name: off}) == 5, name
    assert dw(rows=0, acc=1, x=None, g=None) == 0


def _block(T=4, H=128, rows=8, k=2, post_norm=1, scale=1.0, eps=1e-6):
    return moe._Block(T, H, rows, k, post_norm, scale, eps)


def test_block_refusals(lib):
    P = ctypes.c_void_p
    f, off = P(FAKE), P(FAKE + 8)

    def fwd(b=_block(), res=f, y=f, dest=f, w=f, post=f, gate=f, pre=f, out=f, xn=f):
        return lib.moe_block_norm(None if b is None else ctypes.byref(b), res, y, dest, w, post,
                                  gate, pre, out, xn, None)

    def bwd(b=_block(), h=f, y=f, dest=f, w=f, post=f, gate=f, pre=f, go=f, gx=f, gr=f, gy=f, gw=f,
            gpost=f, ggate=f, gpre=f, ws=f, n=1 << 30):
        return lib.moe_block_norm_bwd(None if b is None else ctypes.byref(b), h, y, dest, w, post,
                                      gate, pre, go, gx, gr, gy, gw, gpost, ggate, gpre, ws, n, None)

    nan, inf = float("nan"), float("inf")
    for call in (fwd, bwd):
        assert call(b=None) == 1
        for bad in (dict(T=-1), dict(H=0), dict(rows=-1), dict(k=0), dict(post_norm=2),
                    dict(scale=nan), dict(scale=inf), dict(eps=0.0), dict(eps=nan), dict(eps=inf),
                    dict(eps=-1e-6)):
            assert call(b=_block(**bad)) == 2, bad
        for bad in (dict(H=96), dict(H=16448), dict(k=9), dict(T=2 ** 30, k=2), dict(rows=2 ** 31)):
            assert call(b=_block(**bad)) == 3, bad
        assert call(dest=None) == 2                            # two slots, one row a token
        assert call(b=_block(k=1, rows=3), dest=None) == 2     # fewer rows than tokens
        for name in ("y", "dest", "w", "post", "gate", "pre"):
            assert call(**{name: off}) == 5, name
    assert fwd(res=None) == 1 and fwd(out=None, xn=None) == 1
    assert fwd(res=off) == 5 and fwd(out=off) == 5 and fwd(xn=off) == 5
    assert fwd(b=_block(T=0), res=None, out=None, xn=None) == 0
    assert bwd(go=None, gx=None) == 1
    assert bwd(h=None) == 1                                    # grad_xn needs the stream
    assert bwd(gx=None) == 1                                   # grad_pre without grad_xn
    for name in ("gy", "gw", "gpost", "ggate"):
        only = dict(gy=None, gw=None, gpost=None, ggate=None) | {name: f}
        assert bwd(y=None, **only) == 1, name                  # gradients of what is not there
    assert bwd(ws=None) == 1 and bwd(ws=off) == 5
    assert bwd(n=moe.block_workspace_size(4, 128) - 1) == 4
    for name in ("h", "go", "gx", "gr", "gy", "gw", "gpost", "ggate", "gpre"):
        assert bwd(**{name: off}) == 5, name
    assert bwd(b=_block(T=0), gpost=None, gpre=None) == 0


def test_block_workspace_size(lib):
    n = ctypes.c_size_t()
    size = lambda T, H: lib.moe_block_norm_workspace_size(T, H, ctypes.byref(n))
    assert size(-1, 128) == 2 and size(1, 0) == 2 and size(1, 96) == 3 and size(1, 16448) == 3
    assert size(2 ** 31, 64) == 3
    assert lib.moe_block_norm_workspace_size(1, 64, None) == 1
    assert size(0, 64) == 0 and n.value == 0
    sizes = [moe.block_workspace_size(T, 4096) for T in (1, 7, 1000, 10 ** 6, 2 ** 31 - 1)]
    assert sizes == sorted(sizes) and sizes[0] > 0 and sizes[-1] < 1 << 28


def test_binding_refusals():
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)
    i32 = z(3, dt=torch.int32)
    bad = [lambda: moe.moe_expert_gemm(z(4, 64), i32, z(2, 64, 128), z(4, 128), epilogue="relu"),
           lambda: moe.moe_expert_gemm(z(4, 64), i32, z(2, 128, 64), z(4, 128)),
           lambda: moe.moe_expert_gemm(z(4, 64), i32, z(2, 64, 128), z(4, 64)),
           lambda: moe.moe_expert_gemm(z(4, 64), i32, z(2, 64, 128), z(4, 128), transposed=True),
           lambda: moe.moe_expert_gemm(z(4, 64), i32, z(2, 64, 128), z(4, 128), epilogue="gelu",
                                       pre=z(3, 128)),
           lambda: moe.moe_expert_gemm(z(4, 64), i32, z(2, 64, 128), z(4, 128)),      # on the host
           lambda: moe.moe_expert_wgrad(z(4, 64), z(5, 128), i32, z(2, 64, 128)),
           lambda: moe.moe_expert_wgrad(z(4, 64), z(4, 64), i32, z(2, 64, 128)),
           lambda: moe.moe_expert_wgrad(z(4, 64), z(4, 128), i32, z(2, 64, 128, dt=torch.float16)),
           lambda: moe.moe_expert_wgrad(z(4, 64), z(4, 128), i32, z(2, 64, 128))]
    cfg = moe.BlockConfig.make()
    dest = z(4, 2, dt=torch.int32)
    f32 = lambda *s: z(*s, dt=torch.float32)
    bad += [lambda: moe.moe_block_norm(cfg, z(4, 64), z(8, 128), z(4, 64), dest_row=dest),
            lambda: moe.moe_block_norm(cfg, z(4, 64), z(8, 64), z(4, 128), dest_row=dest),
            lambda: moe.moe_block_norm(cfg, z(4, 64), z(8, 64), z(4, 64), dest_row=dest[:3]),
            lambda: moe.moe_block_norm(cfg, z(4, 64), z(8, 64), z(4, 64), dest_row=dest,
                                       topk_w=f32(4, 1)),
            lambda: moe.moe_block_norm(cfg, z(4, 64), z(8, 64), z(4, 64), dest_row=dest,
                                       post_weight=f32(128)),
            lambda: moe.moe_block_norm(cfg, z(4, 64), z(8, 64), z(4, 64), dest_row=dest, gate=f32(5)),
            lambda: moe.moe_block_norm(cfg, z(4, 64), z(8, 64), z(4, 64), dest_row=dest),
            lambda: moe.moe_block_norm_bwd(cfg, z(4, 64), z(8, 64), z(4, 64), z(4, 64), z(7, 64),
                                           dest_row=dest),
            lambda: moe.moe_block_norm_bwd(cfg, z(4, 64), z(8, 64), z(4, 64), z(4, 64), z(8, 64),
                                           dest_row=dest, grad_topk_w=f32(4, 1)),
            lambda: moe.moe_block_norm_bwd(cfg, z(4, 64), None, z(4, 64), z(4, 64), z(8, 64))]
    for n, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(str(n))
