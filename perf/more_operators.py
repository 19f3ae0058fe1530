"""Cases of the operators that train a block of experts.

Five operators, in plain torch form and as the framework's kernels:

  product    the experts' grouped product over ragged segments of rows, its
             value before the GELU kept beside the one after it
  product_dx its gradient to the rows: the product with the transposed weights,
             multiplied by the GELU's slope at the kept values where there is one
  product_dw its gradient to the weights: each expert's rows against the rows of
             the gradient, summed over a segment of any length
  block      what lies between two blocks: the weighted sum of a token's expert
             rows, its norm, the token's gate, the scaled residual, and the norm
             that the next block begins with
  block_bwd  the gradient of that to everything that enters it
"""
import math

import torch

own = False  # False: plain torch forms; True: the framework's entry points

_EPS = 1e-6


# ------------------------------------------------------------------ cases ----

def _product(name, rows, E, K, N, gelu=True, skew=0.0):
    return {"name": name, "op": "product", "rows": rows, "E": E, "K": K, "N": N, "gelu": gelu,
            "skew": skew}


def _dx(name, rows, E, K, N, gelu=False, skew=0.0):
    # the gradient rows have K values, the weights are [E, N, K]
    return {"name": name, "op": "product_dx", "rows": rows, "E": E, "K": K, "N": N, "gelu": gelu,
            "skew": skew}


def _dw(name, rows, E, K, N, dtype="fp32", skew=0.0):
    return {"name": name, "op": "product_dw", "rows": rows, "E": E, "K": K, "N": N, "dtype": dtype,
            "skew": skew}


def _block(name, T, H, k, experts=True, post=True, gate=False, pre=True, scale=1.0, drop=0.0,
           bwd=False):
    return {"name": name, "op": "block_bwd" if bwd else "block", "T": T, "H": H, "k": k,
            "experts": experts, "post": post, "gate": gate, "pre": pre, "scale": scale,
            "drop": drop}


def listed():
    return [
        # a small layer's first product, every row of a short batch
        _product("product_small", 1024, 8, 256, 512),
        # the first product of a full training batch over 8 large experts
        _product("product_large", 65536, 8, 4096, 14336),
        # a mid-size odd batch over 16 skewed experts: gradient to the dispatched rows
        _dx("product_dx_ragged", 8191, 16, 2816, 1024, skew=1.0),
        # many small segments: gradient through the second product and the GELU
        _dx("product_dx_fine_grained", 98304, 64, 2048, 1408, gelu=True, skew=0.3),
        # a small layer's weight gradient
        _dw("product_dw_small", 1023, 8, 256, 512),
        # many experts, some of them with few rows: the gradient's own bytes count
        _dw("product_dw_many_expert", 65535, 128, 4096, 2048, "bf16", skew=0.5),
        # the weight gradient of a full training batch over 8 large experts
        _dw("product_dw_large", 65536, 8, 4096, 14336),
        # one token of a decoding step between two blocks
        _block("block_one_token", 1, 4096, 2),
        # a full batch between two blocks, a tenth of the slots over capacity
        _block("block_long", 32768, 4096, 2, drop=0.1),
        # gradient of a small batch
        _block("block_bwd_small", 509, 256, 2, gate=True, bwd=True),
        # gradient of an odd batch with six experts a token, gate and residual scale
        _block("block_bwd_six", 16383, 2048, 6, gate=True, scale=0.5, drop=0.05, bwd=True),
        # gradient of a full batch between two blocks
        _block("block_bwd_long", 32768, 4096, 2, drop=0.1, bwd=True),
    ]


def _log_int(rng, lo, hi, unit=1):
    return unit * int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["product", "product_dx", "product_dw", "block", "block_bwd"])
    if op in ("block", "block_bwd"):
        H = _log_int(rng, 1, 128, 64)
        experts = rng.random() < 0.8
        k = rng.randint(1, 8) if experts else 1
        T = _log_int(rng, 1, min(65536, (1 << 28) // (H * k)))
        pre = rng.random() < 0.8
        return _pure(_block("", T, H, k, experts, not pre or rng.random() < 0.7,
                            rng.random() < 0.5, pre, rng.choice([1.0, 0.5, 2.0]),
                            rng.choice([0.0, 0.1, 0.5]) if experts else 0.0, op == "block_bwd"))
    E = rng.choice([1, 2, 4, 8, 16, 32, 64, 128])
    K, N = _log_int(rng, 1, 224, 64), _log_int(rng, 1, 224, 64)
    while E * K * N > 1 << 29:
        E //= 2
        if E == 0:
            E, K = 1, max(64, K // 128 * 64)
    rows = _log_int(rng, 1, min(98304, (1 << 41) // (2 * K * N), (1 << 29) // max(K, N)))
    skew = rng.choice([0.0, 0.5, 1.0]) if E <= 16 else rng.choice([0.0, 0.3])
    if op == "product_dw":
        return _pure(_dw("", rows, E, K, N, rng.choice(["fp32", "bf16"]), skew))
    return _pure((_product if op == "product" else _dx)("", rows, E, K, N, rng.random() < 0.6, skew))


def _pure(case):
    return {k: v for k, v in case.items() if k != "name"}


# ----------------------------------------------------------------- inputs ----

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, std=1.0):
    return (std * torch.randn(shape, generator=g, device="cuda")).to(torch.bfloat16)


def _segments(rows, E, skew, g):
    """Rows of each expert, as offsets [E + 1]: a multinomial draw whose
    probabilities fall off as (e + 1)^-skew (some experts may get no row)."""
    p = torch.arange(1, E + 1, device="cuda", dtype=torch.float64) ** -skew
    e = torch.multinomial((p / p.sum()).float(), rows, replacement=True, generator=g)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(e, minlength=E).cumsum(0)
    return off


def _kept(case):
    slots = case["T"] * case["k"]
    return slots - int(slots * case["drop"])


def _dispatch(case, g):
    """dest_row [T, k]: the slots that are kept, expert-major and in token order
    within an expert, as a dispatch over 64 experts lays them out; -1 elsewhere."""
    slots = case["T"] * case["k"]
    expert = torch.randint(0, 64, (slots,), generator=g, device="cuda")
    kept = torch.randperm(slots, generator=g, device="cuda")[:_kept(case)].sort().values
    order = kept[torch.sort(expert[kept], stable=True).indices]
    dest = torch.full((slots,), -1, dtype=torch.int32, device="cuda")
    dest[order] = torch.arange(order.numel(), dtype=torch.int32, device="cuda")
    return dest.view(case["T"], case["k"])


def prepare(case, seed):
    g = _gen(seed)
    dev = dict(device="cuda")
    if case["op"] in ("block", "block_bwd"):
        T, H, k = case["T"], case["H"], case["k"]
        bf16 = dict(dtype=torch.bfloat16, **dev)
        st = {"case": case, "y": _randn(g, T * k, H, std=0.5),
              "dest": _dispatch(case, g) if case["experts"] else None,
              "w": (torch.softmax(torch.randn(T, k, generator=g, **dev), 1).contiguous()
                    if case["experts"] else None),
              "post": (1 + 0.1 * torch.randn(H, generator=g, **dev)) if case["post"] else None,
              "gate": torch.rand(T, generator=g, **dev) if case["gate"] else None,
              "pre": (1 + 0.1 * torch.randn(H, generator=g, **dev)) if case["pre"] else None}
        if case["op"] == "block":
            st["residual"] = _randn(g, T, H)
            st["out"] = torch.empty(T, H, **bf16)
            st["xn"] = torch.empty(T, H, **bf16) if case["pre"] else None
            return st
        st["h"] = _randn(g, T, H, std=1.5)   # the residual stream that the forward wrote
        st["g_out"] = _randn(g, T, H)
        st["g_xn"] = _randn(g, T, H) if case["pre"] else None
        st["g_residual"] = torch.empty(T, H, **bf16)
        st["g_y"] = torch.zeros(T * k, H, **bf16)
        st["g_w"] = torch.empty(T, k, **dev) if case["experts"] else None
        st["g_post"] = torch.empty(H, **dev) if case["post"] else None
        st["g_gate"] = torch.empty(T, **dev) if case["gate"] else None
        st["g_pre"] = torch.empty(H, **dev) if case["pre"] else None
        return st
    rows, E, K, N = case["rows"], case["E"], case["K"], case["N"]
    off = _segments(rows, E, case["skew"], g)
    st = {"case": case, "offsets": off, "longest": int((off[1:] - off[:-1]).max()),
          "status": torch.zeros(1, dtype=torch.int32, **dev), "x": _randn(g, rows, K)}
    if case["op"] == "product_dw":
        st["g"] = _randn(g, rows, N)
        st["dw"] = torch.empty(E, K, N, dtype=torch.float32 if case["dtype"] == "fp32"
                               else torch.bfloat16, **dev)
        return st
    transposed = case["op"] == "product_dx"
    st["w"] = _randn(g, E, *((N, K) if transposed else (K, N)), std=K ** -0.5)
    st["out"] = torch.empty(rows, N, dtype=torch.bfloat16, **dev)
    if transposed:
        st["u"] = _randn(g, rows, N) if case["gelu"] else None
    else:
        st["u"] = torch.empty_like(st["out"]) if case["gelu"] else None
    return st


# ------------------------------------------------------------------- runs ----

def run(state):
    return _OWN[state["case"]["op"]](state) if own else _PLAIN[state["case"]["op"]](state)


def _gelu(u):
    return u / (1 + torch.exp(-1.5957691216057308 * (u + 0.044715 * u * u * u)))


def _gelu_slope(u):
    s = 1 / (1 + torch.exp(-1.5957691216057308 * (u + 0.044715 * u * u * u)))
    return s + u * s * (1 - s) * 1.5957691216057308 * (1 + 0.134145 * u * u)


def _places(st):
    """Expert and place within its segment of every row."""
    off = st["offsets"]
    r = torch.arange(st["case"]["rows"], device=off.device)
    e = torch.bucketize(r, off[1:].long(), right=True)
    return e, r - off[e]


def _padded(x, st, e, pos):
    """bf16 rows as fp32 [E, longest segment, width], zeros behind each segment."""
    a = torch.zeros(st["case"]["E"], st["longest"], x.shape[1], device=x.device)
    a[e, pos] = x.float()
    return a


def _plain_product(st):
    e, pos = _places(st)
    y = torch.bmm(_padded(st["x"], st, e, pos), st["w"].float())[e, pos]
    if not st["case"]["gelu"]:
        return {"out": y.to(torch.bfloat16)}
    return {"out": _gelu(y).to(torch.bfloat16), "u": y.to(torch.bfloat16)}


def _plain_dx(st):
    e, pos = _places(st)
    y = torch.bmm(_padded(st["x"], st, e, pos), st["w"].float().transpose(1, 2))[e, pos]
    if st["case"]["gelu"]:
        y = y * _gelu_slope(st["u"].float())
    return {"out": y.to(torch.bfloat16)}


def _plain_dw(st):
    e, pos = _places(st)
    dw = torch.bmm(_padded(st["x"], st, e, pos).transpose(1, 2), _padded(st["g"], st, e, pos))
    return {"dw": dw.to(st["dw"].dtype)}


def _slots(st):
    """Each token's rows [T, k, H] in fp32 (zeros where the slot was dropped) and weights [T, k]."""
    c = st["case"]
    if not c["experts"]:
        return st["y"].float()[:, None], torch.ones(c["T"], 1, device=st["y"].device), None
    kept = st["dest"] >= 0
    rows = st["y"][st["dest"].clamp(min=0).long()].float()
    return rows * kept[:, :, None], st["w"], kept


def _plain_block(st):
    c = st["case"]
    rows, w, _ = _slots(st)
    n = (w[:, :, None] * rows).sum(1)
    if c["post"]:
        n = n * torch.rsqrt((n * n).mean(1, keepdim=True) + _EPS) * st["post"]
    if c["gate"]:
        n = n * st["gate"][:, None]
    h = c["scale"] * st["residual"].float() + n
    res = {"out": h.to(torch.bfloat16)}
    if c["pre"]:
        res["xn"] = (h * torch.rsqrt((h * h).mean(1, keepdim=True) + _EPS)
                     * st["pre"]).to(torch.bfloat16)
    return res


def _plain_block_bwd(st):
    c = st["case"]
    rows, w, kept = _slots(st)
    res = {}
    g = st["g_out"].float()
    if c["pre"]:
        h, gx = st["h"].float(), st["g_xn"].float()
        r = torch.rsqrt((h * h).mean(1, keepdim=True) + _EPS)
        v = gx * st["pre"]
        g = g + r * (v - h * (r * r) * (v * h).mean(1, keepdim=True))
        res["g_pre"] = (gx * h * r).sum(0)
    res["g_residual"] = (c["scale"] * g).to(torch.bfloat16)
    y = (w[:, :, None] * rows).sum(1)
    r = torch.rsqrt((y * y).mean(1, keepdim=True) + _EPS) if c["post"] else torch.ones_like(w[:, :1])
    n = y * r
    weight = st["post"] if c["post"] else 1.0
    gate = st["gate"][:, None] if c["gate"] else 1.0
    if c["gate"]:
        res["g_gate"] = (g * weight * n).sum(1)
    if c["post"]:
        res["g_post"] = (gate * g * n).sum(0)
    v = gate * g * weight
    if c["post"]:
        v = r * (v - n * (v * n).mean(1, keepdim=True))
    if not c["experts"]:
        return res | {"g_y": v.to(torch.bfloat16)}
    res["g_w"] = (v[:, None] * rows).sum(2)
    g_y = torch.zeros_like(st["y"])
    g_y[st["dest"][kept].long()] = (w[:, :, None] * v[:, None])[kept].to(torch.bfloat16)
    return res | {"g_y": g_y}


def _own_product(st):
    import top_routing_expert_gb300 as moe
    gelu = st["case"]["gelu"]
    moe.moe_expert_gemm(st["x"], st["offsets"], st["w"], st["out"],
                        epilogue="gelu" if gelu else None, pre=st["u"], dev_status=st["status"])
    return {"out": st["out"], "u": st["u"]} if gelu else {"out": st["out"]}


def _own_dx(st):
    import top_routing_expert_gb300 as moe
    moe.moe_expert_gemm(st["x"], st["offsets"], st["w"], st["out"], transposed=True,
                        epilogue="gelu_grad" if st["case"]["gelu"] else None, pre=st["u"],
                        dev_status=st["status"])
    return {"out": st["out"]}


def _own_dw(st):
    import top_routing_expert_gb300 as moe
    moe.moe_expert_wgrad(st["x"], st["g"], st["offsets"], st["dw"], dev_status=st["status"])
    return {"dw": st["dw"]}


def _own_block(st):
    import top_routing_expert_gb300 as moe
    c = st["case"]
    if "cfg" not in st:   # a user's program keeps this from step to step
        st["cfg"] = moe.BlockConfig.make(post_norm=c["post"], residual_scale=c["scale"], eps=_EPS)
    moe.moe_block_norm(st["cfg"], st["residual"], st["y"], st["out"], xn=st["xn"],
                       dest_row=st["dest"], topk_w=st["w"], post_weight=st["post"],
                       gate=st["gate"], pre_weight=st["pre"])
    return {"out": st["out"], "xn": st["xn"]} if c["pre"] else {"out": st["out"]}


def _own_block_bwd(st):
    import top_routing_expert_gb300 as moe
    c = st["case"]
    if "cfg" not in st:   # a user's program keeps these from step to step
        st["cfg"] = moe.BlockConfig.make(post_norm=c["post"], residual_scale=c["scale"], eps=_EPS)
        st["ws"] = moe.BlockWorkspace(c["T"], c["H"])
    moe.moe_block_norm_bwd(st["cfg"], st["h"], st["y"], st["g_out"], st["g_residual"], st["g_y"],
                           grad_xn=st["g_xn"], dest_row=st["dest"], topk_w=st["w"],
                           post_weight=st["post"], gate=st["gate"], pre_weight=st["pre"],
                           grad_topk_w=st["g_w"], grad_post=st["g_post"], grad_gate=st["g_gate"],
                           grad_pre=st["g_pre"], ws=st["ws"])
    names = ["g_residual", "g_y"]
    names += ["g_pre"] if c["pre"] else []
    names += ["g_gate"] if c["gate"] else []
    names += ["g_post"] if c["post"] else []
    names += ["g_w"] if c["experts"] else []
    return {n: st[n] for n in names}


_PLAIN = {"product": _plain_product, "product_dx": _plain_dx, "product_dw": _plain_dw,
          "block": _plain_block, "block_bwd": _plain_block_bwd}
_OWN = {"product": _own_product, "product_dx": _own_dx, "product_dw": _own_dw,
        "block": _own_block, "block_bwd": _own_block_bwd}


# ------------------------------------------------------------------- work ----

def work(case):
    if case["op"] in ("block", "block_bwd"):
        T, H, k, kept = case["T"], case["H"], case["k"], _kept(case)
        vectors = 4 * H * (case["post"] + case["pre"])
        slots = 8 * T * k if case["experts"] else 0
        if case["op"] == "block":
            return {"bytes": 2 * H * (kept + (2 + case["pre"]) * T) + vectors + slots
                    + 4 * T * case["gate"],
                    "flops": H * (2 * kept + T * (2 + 4 * case["post"] + 4 * case["pre"]))}
        return {"bytes": 2 * H * (2 * kept + (2 + 2 * case["pre"]) * T) + 2 * vectors
                + slots + (4 * T * k if case["experts"] else 0) + 8 * T * case["gate"],
                "flops": H * (5 * kept + T * (3 + 8 * case["post"] + 9 * case["pre"]))}
    rows, E, K, N = case["rows"], case["E"], case["K"], case["N"]
    if case["op"] == "product_dw":
        return {"bytes": 2 * rows * (K + N) + E * K * N * (4 if case["dtype"] == "fp32" else 2),
                "flops": 2 * rows * K * N}
    # expected number of experts with a row, under the draw of the segments
    p = [(e + 1) ** -case["skew"] for e in range(E)]
    used = sum(1 - (1 - v / sum(p)) ** rows for v in p)
    return {"bytes": int(2 * rows * K + 2 * used * N * K + (4 if case["gelu"] else 2) * rows * N),
            "flops": 2 * rows * K * N}


# ------------------------------------------------------------------ exact ----

def exact(case, seed):
    """The operators' definitions in 64 bits, written apart from the forms above."""
    st = prepare(case, seed)
    if case["op"] in ("block", "block_bwd"):
        return _exact_block(case, st)
    E, K, N = case["E"], case["K"], case["N"]
    cut = st["offsets"].tolist()
    x = st["x"]
    if case["op"] == "product_dw":
        dw = torch.zeros(E, K, N, dtype=torch.float64, device="cuda")
        for e in range(E):
            lo, hi = cut[e], cut[e + 1]
            dw[e] = x[lo:hi].double().T @ st["g"][lo:hi].double()
        return {"dw": dw}
    y = torch.empty(case["rows"], N, dtype=torch.float64, device="cuda")
    for e in range(E):
        w = st["w"][e].double()
        y[cut[e]:cut[e + 1]] = x[cut[e]:cut[e + 1]].double() @ (w.T if w.shape[0] == N and
                                                               case["op"] == "product_dx" else w)
    if not case["gelu"]:
        return {"out": y}
    z = lambda u: torch.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3))
    if case["op"] == "product":
        return {"out": 0.5 * y * (1 + z(y)), "u": y}
    u = st["u"].double()
    t = z(u)
    inner = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * u ** 2)
    return {"out": y * (0.5 * (1 + t) + 0.5 * u * (1 - t * t) * inner)}


def _norm(v, weight):
    return v / torch.sqrt((v ** 2).sum(1, keepdim=True) / v.shape[1] + _EPS) * weight


def _exact_block(case, st):
    """The forward slot by slot; the gradient by automatic differentiation."""
    d = {n: st[n].double() for n in ("y", "w", "post", "gate", "pre") if st[n] is not None}
    bwd = case["op"] == "block_bwd"
    if bwd:
        d = {n: v.requires_grad_() for n, v in d.items()}
    T, H = case["T"], case["H"]
    if case["experts"]:
        total = torch.zeros(T, H, dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            t = torch.nonzero(st["dest"][:, j] >= 0)[:, 0]
            row = d["y"][st["dest"][t, j].long()]
            total = total.index_add(0, t, d["w"][t, j][:, None] * row)
    else:
        total = d["y"]
    if case["post"]:
        total = _norm(total, d["post"])
    if case["gate"]:
        total = d["gate"][:, None] * total
    if not bwd:
        h = case["scale"] * st["residual"].double() + total
        return {"out": h} | ({"xn": _norm(h, d["pre"])} if case["pre"] else {})
    # the gradient is taken at the stream as it was stored
    h = st["h"].double().requires_grad_()
    g = st["g_out"].double()
    res = {}
    if case["pre"]:
        gh, res["g_pre"] = torch.autograd.grad((_norm(h, d["pre"]) * st["g_xn"].double()).sum(),
                                               (h, d["pre"]))
        g = g + gh
    res["g_residual"] = case["scale"] * g
    names = ["y"] + [n for n in ("w", "post", "gate") if n in d]
    grads = torch.autograd.grad((total * g).sum(), [d[n] for n in names])
    return res | {"g_" + n: v for n, v in zip(names, grads)}
