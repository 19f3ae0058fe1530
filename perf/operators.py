"""Cases of the expert-routing and 4-bit expert-product operators.

Four operators of a Mixture-of-Experts layer, in plain torch form and as the
framework's kernels:

  route     grouped top-k routing from fp32 logits: softmax or sigmoid scores,
            a bias that acts on the selection only, groups of experts,
            renormalised and scaled weights, balance statistics
  route_bwd its gradient with respect to the logits
  quantize  bf16 rows to microscaled 4-bit floating point (e2m1 elements, one
            power-of-two scale per 32) and back to the values they stand for
  product   the experts' grouped product of such operands over ragged
            segments of rows, with an optional tanh GELU
"""
import math

import torch

own = False  # False: plain torch forms; True: the framework's entry points

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases ----

def _route(name, T, E, k, score, groups=1, keep=1, top=1, renorm=True, scale=1.0, bias=False,
           masked=0, stats=False):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "groups": groups,
            "keep": keep, "top": top, "renorm": renorm, "scale": scale, "bias": bias,
            "masked": masked, "stats": stats}


def _bwd(name, T, E, k, score, renorm=True, scale=1.0, aux=False):
    return {"name": name, "op": "route_bwd", "T": T, "E": E, "k": k, "score": score,
            "renorm": renorm, "scale": scale, "aux": aux}


def _quantize(name, rows, K):
    return {"name": name, "op": "quantize", "rows": rows, "K": K}


def _product(name, rows, E, K, N, gelu=False, skew=0.0):
    return {"name": name, "op": "product", "rows": rows, "E": E, "K": K, "N": N, "gelu": gelu,
            "skew": skew}


def listed():
    return [
        # one token of a decoding step: sigmoid scores, balance bias, 3 of 8 groups of 8 experts
        _route("route_one_token", 1, 64, 6, "sigmoid", 8, 3, 2, True, 2.5, bias=True),
        # a ragged serving batch over 256 experts in 8 groups, some experts out of service
        _route("route_serving_256", 1021, 256, 8, "sigmoid", 8, 4, 2, True, 2.5, bias=True, masked=5),
        # a training step's tokens over 128 experts, with the balance statistics
        _route("route_training_128", 131072, 128, 2, "softmax", 1, 1, 1, True, 1.0, bias=True,
               stats=True),
        # gradient of a small odd batch over 16 experts
        _bwd("route_bwd_small", 4099, 16, 2, "softmax"),
        # gradient of a long training batch over 256 experts, balance loss included
        _bwd("route_bwd_long_256", 65536, 256, 8, "sigmoid", True, 2.5, aux=True),
        # the rows of a few decoded tokens
        _quantize("quantize_decode", 24, 2048),
        # the dispatched rows of a full training or prefill batch (32768 tokens, top-2)
        _quantize("quantize_prefill", 65536, 4096),
        # one decoded token per sequence, 8 large experts: the weights' bytes count
        _product("product_decode_large", 16, 8, 4096, 14336),
        # a decoding batch over 64 small experts, first product with GELU
        _product("product_decode_many", 96, 64, 2048, 1408, gelu=True),
        # a mid-size odd batch over 16 skewed experts, first product with GELU
        _product("product_ragged", 8191, 16, 1024, 2816, gelu=True, skew=1.0),
        # many small ragged segments, short reduction (second product)
        _product("product_fine_grained", 98304, 64, 1408, 2048, skew=0.3),
        # the first product of a full batch over 8 large experts
        _product("product_large", 65536, 8, 4096, 14336),
    ]


def _log_int(rng, lo, hi, unit=1):
    n = unit * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + unit if n == 3072 else n


def draw(rng):
    op = rng.choice(["route", "route_bwd", "quantize", "product", "product"])
    if op in ("route", "route_bwd"):
        E = rng.choice([8, 12, 16, 32, 48, 60, 64, 96, 128, 160, 192, 256])
        k = rng.randint(1, min(8, E // 4 + 1))
        T = _log_int(rng, 1, 131072 * 128 // E)
        score = rng.choice(["softmax", "sigmoid"])
        renorm, scale = rng.random() < 0.7, rng.choice([1.0, 2.5])
        if op == "route_bwd":
            k = max(k, 2)        # one renormalised weight is constant: nothing to compare
            return _pure(_bwd("", T, E, k, score, renorm, scale, rng.random() < 0.5))
        groups = rng.choice([g for g in (1, 2, 4, 8) if E % g == 0 and E // g >= 2])
        need = -(-k * groups // E)
        keep = rng.randint(need, groups)
        return _pure(_route("", T, E, k, score, groups, keep, rng.choice([1, 2]), renorm, scale,
                            rng.random() < 0.7, rng.choice([0, 0, 1]), rng.random() < 0.5))
    if op == "quantize":
        K = _log_int(rng, 4, 224, 64)
        return _pure(_quantize("", _log_int(rng, 1, (1 << 28) // K), K))
    E = rng.choice([4, 8, 16, 32, 64, 128])
    K, N = _log_int(rng, 4, 112, 64), _log_int(rng, 4, 112, 64)
    while E * K * N > 1 << 30:
        E //= 2
    rows = _log_int(rng, 1, min(98304, max(64, (1 << 40) // (2 * K * N))))
    return _pure(_product("", rows, E, K, N, rng.random() < 0.4, rng.choice([0.0, 0.5, 1.0])))


def _pure(case):
    return {k: v for k, v in case.items() if k != "name"}


# ----------------------------------------------------------------- inputs ----

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _segments(rows, E, skew, g):
    """Rows of each expert, as offsets [E + 1]: a multinomial draw whose
    probabilities fall off as (e + 1)^-skew (some experts may get no row)."""
    p = torch.arange(1, E + 1, device="cuda", dtype=torch.float64) ** -skew
    e = torch.multinomial((p / p.sum()).float(), rows, replacement=True, generator=g)
    count = torch.bincount(e, minlength=E)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = count.cumsum(0)
    return off


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    dev = dict(device="cuda")
    if op in ("route", "route_bwd"):
        T, E, k = case["T"], case["E"], case["k"]
        st = {"case": case, "logits": _randn(g, T, E)}   # x . gate of unit-variance tokens
        if op == "route":
            st["bias"] = 0.05 * _randn(g, E) if case["bias"] else None
            if case["masked"]:
                st["logits"][:, torch.randperm(E, generator=g, **dev)[:case["masked"]]] = -math.inf
            st["idx"] = torch.empty(T, k, dtype=torch.int32, **dev)
            st["w"] = torch.empty(T, k, **dev)
            stats = case["stats"]
            st["routed"] = torch.empty(E, dtype=torch.int32, **dev) if stats else None
            st["P"] = torch.empty(E, **dev) if stats else None
            st["aux"] = torch.empty(1, **dev) if stats else None
        else:
            # the k largest logits as routing choices, as int32 [T, k]
            st["idx"] = torch.topk(st["logits"], k, dim=1).indices.to(torch.int32).contiguous()
            st["grad_w"] = _randn(g, T, k)
            st["grad_aux"] = torch.full((1,), 0.01 * T, **dev) if case["aux"] else None
            st["routed"] = (torch.bincount(st["idx"].flatten().long(), minlength=E).to(torch.int32)
                            if case["aux"] else None)
            st["grad"] = torch.empty(T, E, **dev)
        return st
    if op == "quantize":
        rows, K = case["rows"], case["K"]
        x = _randn(g, rows, K).to(torch.bfloat16)
        if rows > 8:
            x[rows // 2] = 0                                # a row of zeros, as padding gives
        return {"case": case, "x": x,
                "q": torch.empty(rows, K // 2, dtype=torch.uint8, **dev),
                "scale": torch.empty(-(-K // 128), rows, 4, dtype=torch.uint8, **dev),
                "back": torch.empty_like(x)}
    rows, E, K, N = case["rows"], case["E"], case["K"], case["N"]
    off = _segments(rows, E, case["skew"], g)
    x_q, x_s = _quantize_packed(_randn(g, rows, K))
    w_q = torch.empty(E, N, K // 2, dtype=torch.uint8, **dev)
    w_s = torch.empty(E, N, K // 32, dtype=torch.uint8, **dev)
    for e in range(E):                                      # one expert at a time: less memory
        w_q[e], w_s[e] = _quantize_packed(_randn(g, N, K) / math.sqrt(K))
    return {"case": case, "x_q": x_q, "x_scale": _rows_scale(x_s), "offsets": off,
            "longest": int((off[1:] - off[:-1]).max()),
            "w_q": w_q, "w_scale": _weights_scale(w_s),
            "out": torch.empty(rows, N, dtype=torch.bfloat16, **dev),
            "status": torch.zeros(1, dtype=torch.int32, **dev)}


# --------------------------------------------------- microscaled 4 bits ----

def _quantize_values(x):
    """fp32 [R, K] -> the e2m1 values [R, K] and the scale bytes [R, K/32]."""
    R, K = x.shape
    b = x.view(R, K // 32, 32)
    amax = b.abs().amax(2)
    exp = torch.clamp(torch.frexp(amax)[1] - 3, min=-127)       # floor(log2(amax)) - 2
    exp = torch.where(amax > 0, exp, -127)
    v = torch.ldexp(b, -exp[:, :, None])                         # below 8 in magnitude
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    q = torch.copysign(torch.clamp(torch.round(a / step) * step, max=6.0), v)
    bad = ~torch.isfinite(amax)
    q = torch.where(bad[:, :, None], 0.0, q)
    byte = torch.where(bad, 255, exp + 127).to(torch.uint8)
    return q.view(R, K), byte


def _quantize_packed(x):
    """fp32 [R, K] -> codes [R, K/2] (the even element in the low half) and
    scale bytes [R, K/32]."""
    q, byte = _quantize_values(x)
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte


def _rows_scale(s):
    """Scale bytes [R, K/32] -> [ceil(K/128), R, 4], the layout of rows."""
    R, n = s.shape
    pad = torch.zeros(R, -(-n // 4) * 4, dtype=torch.uint8, device=s.device)
    pad[:, :n] = s
    return pad.view(R, -1, 4).transpose(0, 1).contiguous()


def _weights_scale(s):
    """Scale bytes [E, N, K/32] -> [E, ceil(N/128), ceil(K/128), 32, 4, 4], the
    layout of weights: output column n of a block of 128 at [n % 32, n / 32]."""
    E, N, n = s.shape
    tn, tk = -(-N // 128), -(-n // 4)
    pad = torch.zeros(E, tn * 128, tk * 4, dtype=torch.uint8, device=s.device)
    pad[:, :N, :n] = s
    return pad.view(E, tn, 4, 32, tk, 4).permute(0, 1, 4, 3, 2, 5).contiguous()


def _unpack(q, byte, dtype):
    """Codes [..., K/2] and scale bytes [..., K/32] -> values [..., K]."""
    lut = torch.tensor(_E2M1, dtype=dtype, device=q.device)
    v = torch.stack((lut[(q & 15).int()], lut[(q >> 4).int()]), dim=-1).flatten(-2)
    s = torch.ldexp(torch.ones_like(byte, dtype=dtype), byte.int() - 127)
    s = torch.where(byte == 255, math.nan, s)
    return (v.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def _plain_rows(q, scale, dtype):
    tk, R, _ = scale.shape
    return _unpack(q, scale.transpose(0, 1).reshape(R, tk * 4)[:, :q.shape[1] // 16], dtype)


def _plain_weights(q, scale, dtype):
    E, N, half = q.shape
    tn, tk = scale.shape[1:3]
    s = scale.permute(0, 1, 4, 3, 2, 5).reshape(E, tn * 128, tk * 4)[:, :N, :half // 16]
    return _unpack(q, s, dtype)


# ------------------------------------------------------------------- runs ----

def run(state):
    return _OWN[state["case"]["op"]](state) if own else _PLAIN[state["case"]["op"]](state)


def _scores(l, score):
    """Scores of logits l; a masked expert (logit -inf) scores 0."""
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    m = l.amax(1, keepdim=True)
    z = torch.exp(l - torch.where(torch.isfinite(m), m, 0.0))
    return z / z.sum(1, keepdim=True).clamp(min=1e-300)


def _plain_route(st):
    # 64 bits: which experts are chosen hangs on values next to one another
    c = st["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l = st["logits"].double()
    s = _scores(l, c["score"])
    v = s if st["bias"] is None else s + st["bias"].double()
    v = torch.where(torch.isneginf(l), -math.inf, v)
    value = torch.sort(v.view(T, G, E // G), dim=2, descending=True).values[:, :, :c["top"]].sum(2)
    kept = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :c["keep"]]
    out = torch.ones(T, G, dtype=torch.bool, device=l.device).scatter_(1, kept, False)
    # experts of groups that are out come after every masked one of a kept group
    # a masked expert comes after every other of its group, before those of groups left out
    order = torch.where(out[:, :, None].expand(T, G, E // G).reshape(T, E), -math.inf,
                        v.clamp(min=-1e300))
    idx = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    res = {"idx": idx.to(torch.int32), "w": (w * c["scale"]).float()}
    if c["stats"]:
        routed = torch.bincount(idx.flatten(), minlength=E)
        P = (s / s.sum(1, keepdim=True).clamp(min=1e-300)).mean(0)
        res |= {"routed": routed.to(torch.int32), "P": P.float(),
                "aux": (E * (routed.double() / (T * k) * P).sum()).float().view(1)}
    return res


def _plain_route_bwd(st):
    c = st["case"]
    return {"grad": _route_gradient(st["logits"], st["idx"].long(), st["grad_w"], c, st["grad_aux"],
                                    st["routed"])}


def _route_gradient(l, idx, g, c, grad_aux, routed):
    T, E, k = c["T"], c["E"], c["k"]
    s = _scores(l, c["score"])
    chosen = s.gather(1, idx)
    slope = 1 - s if c["score"] == "sigmoid" else torch.ones_like(s)
    grad = torch.zeros_like(l)
    if c["renorm"]:
        q = chosen / chosen.sum(1, keepdim=True)
        d = c["scale"] * q * (g - (q * g).sum(1, keepdim=True))
        grad.scatter_(1, idx, d * slope.gather(1, idx))
    elif c["score"] == "sigmoid":
        grad.scatter_(1, idx, c["scale"] * g * chosen * (1 - chosen))
    else:
        up = torch.zeros_like(l).scatter_(1, idx, c["scale"] * g)
        grad = s * (up - (s * up).sum(1, keepdim=True))
    if grad_aux is not None:
        p = s / s.sum(1, keepdim=True)
        h = grad_aux.to(l.dtype) * (E / (T * T * k)) * routed.to(l.dtype)
        grad = grad + p * slope * (h - (p * h).sum(1, keepdim=True))
    return grad


def _plain_quantize(st):
    q, byte = _quantize_values(st["x"].float())
    s = torch.ldexp(torch.ones_like(byte, dtype=torch.float32), byte.int() - 127)
    s = torch.where(byte == 255, math.nan, s)
    R, K = q.shape
    return {"values": (q.view(R, K // 32, 32) * s[:, :, None]).view(R, K).to(torch.bfloat16)}


def _gelu(u):
    return u / (1 + torch.exp(-1.5957691216057308 * (u + 0.044715 * u * u * u)))


def _plain_product(st):
    c, off = st["case"], st["offsets"]
    r = torch.arange(c["rows"], device=off.device)
    e = torch.bucketize(r, off[1:].long(), right=True)
    pos = r - off[e]
    a = torch.zeros(c["E"], st["longest"], c["K"], device=off.device)
    a[e, pos] = _plain_rows(st["x_q"], st["x_scale"], torch.float32)
    w = _plain_weights(st["w_q"], st["w_scale"], torch.float32)
    y = torch.bmm(a, w.transpose(1, 2))[e, pos]
    return {"out": (_gelu(y) if c["gelu"] else y).to(torch.bfloat16)}


def _own_route(st):
    import top_routing_expert_gb300 as moe
    c = st["case"]
    if "ws" not in st:   # a user's program keeps these from step to step
        st["shape"] = moe.MoeShape.make(c["T"], 64, c["E"], c["k"], 64, 1.0)
        st["cfg"] = moe.RouteConfig.make(c["score"], n_groups=c["groups"], topk_groups=c["keep"],
                                         group_top=c["top"], renormalize=c["renorm"],
                                         scale=c["scale"])
        st["ws"] = moe.Workspace(st["shape"])
    moe.moe_route_grouped(st["shape"], st["cfg"], st["logits"], st["bias"], st["idx"], st["w"],
                          routed_counts=st["routed"], P=st["P"], aux=st["aux"], ws=st["ws"])
    res = {"idx": st["idx"], "w": st["w"]}
    if c["stats"]:
        res |= {"routed": st["routed"], "P": st["P"], "aux": st["aux"]}
    return res


def _own_route_bwd(st):
    import top_routing_expert_gb300 as moe
    c = st["case"]
    if "cfg" not in st:
        st["shape"] = moe.MoeShape.make(c["T"], 64, c["E"], c["k"], 64, 1.0)
        st["cfg"] = moe.RouteConfig.make(c["score"], renormalize=c["renorm"], scale=c["scale"])
    moe.moe_route_grouped_bwd(st["shape"], st["cfg"], st["logits"], st["idx"], st["grad_w"],
                              st["grad"], grad_aux=st["grad_aux"], routed_counts=st["routed"])
    return {"grad": st["grad"]}


def _own_quantize(st):
    import top_routing_expert_gb300 as moe
    moe.moe_quantize_rows_mx4(st["x"], st["q"], st["scale"])
    moe.moe_dequantize_rows_mx4(st["q"], st["scale"], st["back"])
    return {"values": st["back"]}


def _own_product(st):
    import top_routing_expert_gb300 as moe
    moe.moe_expert_gemm_mx4(st["x_q"], st["x_scale"], st["offsets"], st["w_q"], st["w_scale"],
                            st["out"], gelu=st["case"]["gelu"], dev_status=st["status"])
    return {"out": st["out"]}


_PLAIN = {"route": _plain_route, "route_bwd": _plain_route_bwd, "quantize": _plain_quantize,
          "product": _plain_product}
_OWN = {"route": _own_route, "route_bwd": _own_route_bwd, "quantize": _own_quantize,
        "product": _own_product}


# ------------------------------------------------------------------- work ----

def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        stats = 12 * E if case["stats"] else 0
        return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0) + stats,
                "flops": 8 * T * E}
    if op == "route_bwd":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 8 * T * E + 8 * T * k + (4 * E if case["aux"] else 0),
                "flops": (12 if case["aux"] else 6) * T * E}
    if op == "quantize":
        # bf16 in, the packed form written and read back, bf16 values out
        n = case["rows"] * case["K"]
        return {"bytes": 2 * n + 2 * (n // 2 + n // 32) + 2 * n, "flops": 4 * n}
    rows, E, K, N = case["rows"], case["E"], case["K"], case["N"]
    # expected number of experts with a row, under the draw of the segments
    p = [(e + 1) ** -case["skew"] for e in range(E)]
    used = sum(1 - (1 - v / sum(p)) ** rows for v in p)
    return {"bytes": int(rows * K * 17 / 32 + used * N * K * 17 / 32 + 2 * rows * N),
            "flops": 2 * rows * K * N}


# ------------------------------------------------------------------ exact ----

def exact(case, seed):
    """The operators' definitions in 64 bits, written apart from the forms above."""
    st = prepare(case, seed)
    op = case["op"]
    f64 = dict(dtype=torch.float64, device="cuda")
    if op == "quantize":
        x = st["x"].double()
        R, K = x.shape
        mag = x.abs().view(R, K // 32, 32)
        scale = 2.0 ** torch.clamp(torch.floor(torch.log2(mag.amax(2, keepdim=True))) - 2, min=-127)
        y = mag / scale
        # nearest of the eight magnitudes; at a midpoint the one whose code is even
        out = torch.zeros_like(y)
        for mid, low_even, value in ((0.25, True, 0.5), (0.75, False, 1.0), (1.25, True, 1.5),
                                     (1.75, False, 2.0), (2.5, True, 3.0), (3.5, False, 4.0),
                                     (5.0, True, 6.0)):
            out = torch.where(y > mid if low_even else y >= mid, value, out)
        return {"values": (out * scale).view(R, K) * torch.sign(x)}
    if op == "product":
        rows, E, K, N = case["rows"], case["E"], case["K"], case["N"]
        cut = st["offsets"].tolist()
        block = torch.arange(K // 32, device="cuda")
        n = torch.arange(N, device="cuda")[:, None]
        out = torch.empty(rows, N, **f64)
        for e in range(E):
            lo, hi = cut[e], cut[e + 1]
            if hi == lo:
                continue
            r = torch.arange(lo, hi, device="cuda")[:, None]
            a = _exact_values(st["x_q"][lo:hi], st["x_scale"][block // 4, r, block % 4])
            w = _exact_values(st["w_q"][e], st["w_scale"][e, n // 128, block // 4, n % 32,
                                                          n % 128 // 32, block % 4])
            out[lo:hi] = a @ w.T
        if case["gelu"]:
            out = 0.5 * out * (1 + torch.tanh(math.sqrt(2 / math.pi) * (out + 0.044715 * out ** 3)))
        return {"out": out}
    T, E, k = case["T"], case["E"], case["k"]
    if op == "route_bwd":
        # automatic differentiation of the forward
        l = st["logits"].double().requires_grad_()
        s = _exact_scores(l, case["score"])
        w = s.gather(1, st["idx"].long())
        if case["renorm"]:
            w = w / w.sum(1, keepdim=True)
        loss = (case["scale"] * w * st["grad_w"].double()).sum()
        if case["aux"]:
            P = (s / s.sum(1, keepdim=True)).mean(0)
            loss = loss + st["grad_aux"].double()[0] * E * (st["routed"].double() / (T * k) * P).sum()
        return {"grad": torch.autograd.grad(loss, l)[0]}
    G = case["groups"]
    l = st["logits"].double()
    s = _exact_scores(l, case["score"])
    v = s.clone() if st["bias"] is None else s + st["bias"].double()
    v[torch.isneginf(l)] = -math.inf
    g = v.view(T, G, E // G).clone()
    total = torch.zeros(T, G, **f64)
    for _ in range(case["top"]):                      # a group's largest value, then the next
        best = g.max(2)
        total += best.values
        g.scatter_(2, best.indices[:, :, None], -math.inf)
    ahead = (total[:, None, :] > total[:, :, None]).sum(2)
    earlier = torch.ones(G, G, device="cuda").tril(-1).bool()
    ahead += ((total[:, None, :] == total[:, :, None]) & earlier).sum(2)
    left = (ahead < case["keep"]).repeat_interleave(E // G, 1)
    idx = torch.empty(T, k, dtype=torch.long, device="cuda")
    place = torch.arange(E, device="cuda").expand(T, E)
    for j in range(k):
        top = torch.where(left, v, -math.inf).amax(1, keepdim=True)
        at = torch.where(left & (v == top), place, E).amin(1)
        idx[:, j] = at
        left.scatter_(1, at[:, None], False)
    w = s.gather(1, idx)
    if case["renorm"]:
        w = torch.nan_to_num(w / w.sum(1, keepdim=True), nan=0.0)
    res = {"idx": idx.to(torch.int32), "w": case["scale"] * w}
    if case["stats"]:
        P = torch.nan_to_num(s / s.sum(1, keepdim=True), nan=0.0).mean(0)
        count = torch.zeros(E, **f64).index_add_(0, idx.flatten(), torch.ones(T * k, **f64))
        res |= {"routed": count.to(torch.int32), "P": P,
                "aux": (E * torch.dot(count / (T * k), P)).view(1)}
    return res


def _exact_scores(l, score):
    if score == "sigmoid":
        t = torch.exp(-l.abs())
        return torch.where(l >= 0, 1 / (1 + t), t / (1 + t))
    return torch.nan_to_num(torch.exp(l - torch.logsumexp(l, 1, keepdim=True)), nan=0.0)


def _exact_values(q, byte):
    """e2m1 codes [R, K/2] with their scale bytes [R, K/32], from the bits."""
    code = torch.stack((q % 16, q // 16), dim=2).flatten(1).int()
    exp, man = code // 2 % 4, (code % 2).double()
    mag = torch.where(exp == 0, 0.5 * man, 2.0 ** (exp - 1).double() * (1 + 0.5 * man))
    scale = 2.0 ** (byte.double() - 127)
    return torch.where(code >= 8, -mag, mag) * scale.repeat_interleave(32, dim=1)
