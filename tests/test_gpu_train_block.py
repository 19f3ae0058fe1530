"""A training step of a block: the products, the step between two blocks, the
router and the dispatch together, against float64 and automatic differentiation
of the same formulas with the GPU's own choice of experts and drops.

Between the steps values are rounded to bf16 (half a step, 2^-8 of the value):
xn, u, a, y, and on the way back g_out's successors g_y, g_u, g_x, the router's
scores and g_xn (twice). A gradient that passes n of them is off by about sqrt(n)
2^-8 / sqrt(3) of its 2-norm, as their errors have random signs; n is at most 8.
Outputs are held to twice that, 2^-8 sqrt(32 / 3) of the 2-norm. A factor or a
term that is missing shows as much more. The router's gradient comes from g_w_tj =
<g_c, y_j>, a sum over H products that cancel: its error goes by m_tj, the 2-norm
of the products, whatever is left of their sum, and the logits' by w_j (m_tj +
sum_i w_i m_ti), which the token's xn multiplies (the gate's gradient) or not (its
bias')."""
import numpy as np
import pytest
import torch

import top_routing_expert_gb300 as moe
from top_routing_expert_gb300.block import BlockWeights, TrainBlock

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 2.0 ** -8 * (32 / 3) ** 0.5


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    moe.build()
    moe.load_library()


def _make(T, H, E, k, h, cf, score, post_norm, scale, seed):
    g = torch.Generator().manual_seed(seed)
    bf = lambda *n, std=1.0: (std * torch.randn(n, generator=g)).to(torch.bfloat16).to(DEV)
    f32 = lambda *n: torch.randn(n, generator=g).to(DEV)
    w = BlockWeights(bf(E, H, h, std=H ** -0.5), bf(E, h, H, std=h ** -0.5), bf(H, E, std=H ** -0.5),
                     1 + 0.2 * f32(H), 1 + 0.2 * f32(H), 0.5 * f32(E) if T % 2 else None)
    block = TrainBlock(moe.MoeShape.make(T, H, E, k, h, cf), moe.RouteConfig.make(score),
                       moe.BlockConfig.make(post_norm=post_norm, residual_scale=scale, eps=1e-5))
    data = {"h": bf(T, H), "xn": bf(T, H), "gate": torch.rand(T, generator=g).to(DEV),
            "g_out": bf(T, H), "g_xn": bf(T, H), "g_aux": torch.full((1,), 0.3, device=DEV)}
    return block, w, data


def _step(block, w, d, grads=None, accumulate=False):
    T, H = d["h"].shape
    new = lambda: torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    out, xn, gh, gx = new(), new(), new(), new()
    g_gate = torch.empty(T, device=DEV)
    grads = grads or BlockWeights.zeros_like(w)
    block.forward(d["h"], d["xn"], w, out, xn, token_gate=d["gate"])
    block.backward(d["g_out"], d["g_xn"], gh, gx, grads, grad_token_gate=g_gate,
                   grad_aux=d["g_aux"], accumulate=accumulate)
    res = {"out": out, "xn_next": xn, "h": gh, "xn": gx, "token_gate": g_gate, "W1": grads.W1,
           "W2": grads.W2, "gate": grads.gate, "post": grads.post, "pre": grads.pre}
    return res if w.gate_bias is None else res | {"gate_bias": grads.gate_bias}


def _reference(block, w, d, score, post_norm, scale):
    f64 = lambda t: t.detach().double().requires_grad_()
    v = {n: f64(getattr(w, n)) for n in ("W1", "W2", "gate", "post", "pre")}
    v |= {"h": f64(d["h"]), "xn": f64(d["xn"]), "token_gate": f64(d["gate"])}
    s, eps = block.shape, 1e-5
    idx, dest = block.topk_idx.long(), block.dest_row
    logits = v["xn"] @ v["gate"]
    if w.gate_bias is not None:
        v["gate_bias"] = f64(w.gate_bias)
        logits = logits + v["gate_bias"]
    p = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    chosen = p.gather(1, idx)
    weights = chosen / chosen.sum(1, keepdim=True)
    P = (p / p.sum(1, keepdim=True)).mean(0)
    f = block.routed_counts.double() / (s.T * s.top_k)
    aux = s.E * (f * P).sum()
    c = torch.zeros(s.T, s.H, dtype=torch.float64, device=DEV)
    y = torch.zeros(s.T, s.top_k, s.H, dtype=torch.float64, device=DEV)
    for e in range(s.E):
        t, j = torch.nonzero((idx == e) & (dest >= 0), as_tuple=True)
        a = torch.nn.functional.gelu(v["xn"][t] @ v["W1"][e], approximate="tanh")
        row = a @ v["W2"][e]
        y[t, j] = row.detach()
        c = c.index_add(0, t, weights[t, j][:, None] * row)
    n = c / torch.sqrt((c * c).mean(1, keepdim=True) + eps) if post_norm else c
    out = scale * v["h"] + v["token_gate"][:, None] * n * v["post"]
    xn = out / torch.sqrt((out * out).mean(1, keepdim=True) + eps) * v["pre"]
    loss = (out * d["g_out"].double()).sum() + (xn * d["g_xn"].double()).sum() + aux * d["g_aux"].double()[0]
    names = list(v)
    g_c, *found = torch.autograd.grad(loss, [c] + [v[n] for n in names])
    m = (g_c[:, None] * y).norm(dim=2)
    wt = weights.detach()
    per_logit = wt * (m + (wt * m).sum(1, keepdim=True))
    router = {"gate": (d["xn"].double().norm(dim=1) * per_logit.norm(dim=1)).norm().item(),
              "gate_bias": per_logit.norm().item()}
    return {"out": out, "xn_next": xn} | dict(zip(names, found)), router


CASES = [
    # T, H, E, k, h, capacity factor, score, post_norm, residual scale
    (300, 128, 8, 2, 192, 4.0, "softmax", True, 1.0),
    (257, 256, 12, 3, 128, 1.0, "sigmoid", True, 0.5),     # dropped slots, E no multiple of 64
    (1000, 192, 64, 6, 64, 1.25, "sigmoid", False, 1.0),
    (1, 64, 4, 2, 64, 4.0, "softmax", True, 1.0),          # one token
    (513, 320, 1, 1, 448, 1.0, "softmax", True, 2.0),      # one expert
]


@pytest.mark.parametrize("case", CASES)
def test_step(case):
    T, H, E, k, h, cf, score, post_norm, scale = case
    block, w, d = _make(*case, seed=T)
    got = _step(block, w, d)
    assert int(block.dev_status.item()) == 0
    if cf < 4 and E > 1:
        assert int(block.offsets[E].item()) < T * k        # some slots were dropped
    want, router = _reference(block, w, d, score, post_norm, scale)
    for n, ref in want.items():
        err, size = (got[n].double() - ref).norm().item(), ref.norm().item()
        assert err <= TOL * (size + router.get(n, 0.0)) + 1e-6, (n, err / size)


def test_accumulation_graph_and_streams():
    block, w, d = _make(*CASES[1], seed=3)
    first = _step(block, w, d)
    twice = BlockWeights.zeros_like(w)
    for _ in range(2):
        _step(block, w, d, twice, accumulate=True)
    # x + x is exact
    assert torch.equal(twice.W1, 2 * first["W1"]) and torch.equal(twice.W2, 2 * first["W2"])
    assert torch.equal(twice.gate, first["gate"]) and torch.equal(twice.post, first["post"])
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        second = _step(block, w, d)
    stream.synchronize()
    grads = BlockWeights.zeros_like(w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = _step(block, w, d, grads)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for n in first:
            assert torch.equal(first[n], second[n]) and torch.equal(first[n], third[n]), n


def test_no_tokens_and_order():
    block, w, _ = _make(0, 128, 4, 2, 64, 1.0, "softmax", True, 1.0, seed=1)
    e = torch.empty(0, 128, dtype=torch.bfloat16, device=DEV)
    grads = BlockWeights.zeros_like(w)
    with pytest.raises(RuntimeError):
        block.backward(e, e, e, e, grads)
    grads.W1.fill_(1)
    block.forward(e, e, w, e, e)
    block.backward(e, e, e, e, grads, accumulate=True)
    assert (grads.W1 == 1).all() and (grads.gate == 0).all()
    block.backward(e, e, e, e, grads)
    assert (grads.W1 == 0).all()


def test_one_gradient_alone():
    block, w, d = _make(*CASES[0], seed=9)
    T, H = d["h"].shape
    new = lambda: torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    out, gh, gx = new(), new(), new()
    grads = BlockWeights.zeros_like(w)
    grads.pre.fill_(5)
    block.forward(d["h"], d["xn"], w, out)                 # the last block: no next norm
    block.backward(d["g_out"], None, gh, gx, grads)
    assert (grads.pre == 0).all()
    assert torch.equal(gh, d["g_out"])                     # the residual passes it on


def test_module_runs(capsys):
    from top_routing_expert_gb300 import block
    block.main()
    assert "status 0" in capsys.readouterr().out
