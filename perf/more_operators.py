"""Operators of a feed-forward block on quantized weights: what is measured, on which sizes, and their
plain forms.

Operands are e4m3 codes with one exponent byte E (value 2**(E - 127)) for each 1 x 128 (activations) or
128 x 128 (weights) block; A and W stand for what they say, with a factor per row:

* route:    logits [T, E]; s = softmax or sigmoid; c = s + bias (c = the logits where there is neither a bias
            nor groups); only the best groups (sum of the `group_top` largest c of each) are looked at; ids:
            the k largest c, the lowest index of equals; weights: s of those, over their sum, times scale;
            order: the assignments t k + j sorted by expert, in their own order; offsets: where each begins;
* linear:   out = act(A W^T + bias) + residual;
* gated:    v = silu(A G^T) * (A U^T), as codes and exponents by 1 x 128 blocks;
* experts:  gated, of the rows that were routed to each expert (token of position p: order[p] // k), in that
            order; or out[order[p]] = row p times the expert's W^T;
* combine:  out[t] = residual[t] + sum_j weights[t, j] y[t k + j].
"""

import math

import torch

own = False

BLOCK = 128       # elements of a scale block
F8 = torch.float8_e4m3fn
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------

def listed():
    return [
        # one token of a decoder with 64 experts: latency
        {"name": "route 1x64", "op": "route", "tokens": 1, "experts": 64, "top_k": 6, "dtype": "bf16", "scores": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "group_top": 1, "renormalize": True, "scale": 1.0},
        # a ragged batch, experts in groups that share a machine, weights as they come out of the softmax
        {"name": "route 333x160", "op": "route", "tokens": 333, "experts": 160, "top_k": 6, "dtype": "f16", "scores": "softmax", "bias": False,
         "groups": 8, "top_groups": 3, "group_top": 1, "renormalize": False, "scale": 16.0},
        # a long prompt, sigmoid scores with a bias that balances the experts' load
        {"name": "route 8192x256", "op": "route", "tokens": 8192, "experts": 256, "top_k": 8, "dtype": "f32", "scores": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_top": 2, "renormalize": True, "scale": 2.5},
        # down projection of one token, added to what went into the block
        {"name": "linear 1x4096x11008", "op": "linear", "m": 1, "n": 4096, "k": 11008, "dtype": "bf16", "bias": False, "act": "none",
         "residual": True},
        # first projection of a plain feed-forward, a short ragged prompt
        {"name": "linear 515x11008x4096", "op": "linear", "m": 515, "n": 11008, "k": 4096, "dtype": "f16", "bias": True, "act": "gelu",
         "residual": False},
        # gate and up projections of a batch of sequences decoding together
        {"name": "gated 24x11008x4096", "op": "gated", "m": 24, "n": 11008, "k": 4096},
        # gate and up projections of a long prompt
        {"name": "gated 4096x11008x4096", "op": "gated", "m": 4096, "n": 11008, "k": 4096},
        # experts of one token: latency
        {"name": "experts gated 1 of 64", "op": "experts_gated", "tokens": 1, "experts": 64, "top_k": 6, "n": 1376, "k": 4096},
        # a decoding batch: nearly every expert is read for a few rows
        {"name": "experts out 40 of 64", "op": "experts_out", "tokens": 40, "experts": 64, "top_k": 6, "n": 4096, "k": 1376},
        # a long prompt over all experts, some of them much busier than others
        {"name": "experts gated 4096 of 64", "op": "experts_gated", "tokens": 4096, "experts": 64, "top_k": 6, "n": 1376, "k": 4096},
        # one token
        {"name": "combine 1x6x4096", "op": "combine", "tokens": 1, "top_k": 6, "d": 4096, "dtype": "bf16", "residual": True},
        # a long prompt
        {"name": "combine 4096x8x4096", "op": "combine", "tokens": 4096, "top_k": 8, "d": 4096, "dtype": "bf16", "residual": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: whole blocks, a multiple of 8, or any number."""
    v = _log(rng, lo, hi)
    step = rng.choice((BLOCK, BLOCK, 8, 1))
    return max(lo, v // step * step)


def draw(rng):
    op = rng.choice(("route", "linear", "gated", "experts_gated", "experts_out", "combine"))
    if op == "route":
        experts = rng.choice((8, 16, 60, 64, 128, 160, 256, 384, 512))
        groups = rng.choice((1, 1, 4, 8) if experts % 8 == 0 else (1, 4))
        top_groups = rng.randint(max(1, groups // 4), groups)
        top_k = rng.randint(1, min(10, experts // groups * top_groups))
        return {"op": op, "tokens": _log(rng, 1, 8192), "experts": experts, "top_k": top_k, "dtype": rng.choice(("bf16", "f16", "f32")),
                "scores": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5, "groups": groups, "top_groups": top_groups,
                "group_top": rng.choice((1, 2)) if experts > groups else 1, "renormalize": rng.random() < 0.7, "scale": rng.choice((1.0, 2.5))}
    if op in ("linear", "gated"):
        while True:
            case = {"op": op, "m": _log(rng, 1, 8192), "n": _width(rng, 128, 11008), "k": _width(rng, 128, 28672)}
            if case["m"] * case["n"] * case["k"] <= 4096 * 11008 * 4096:
                break
        if op == "linear":
            case |= {"dtype": rng.choice(("bf16", "f16")), "bias": rng.random() < 0.5, "act": rng.choice(("none", "relu", "silu", "gelu")),
                     "residual": rng.random() < 0.5}
        return case
    if op == "combine":
        while True:
            case = {"op": op, "tokens": _log(rng, 1, 8192), "top_k": rng.randint(1, 10), "d": _width(rng, 128, 8192),
                    "dtype": rng.choice(("bf16", "f16")), "residual": rng.random() < 0.5}
            if case["tokens"] * case["top_k"] * case["d"] <= 4096 * 8 * 4096:
                return case
    while True:
        experts = rng.choice((8, 16, 32, 64, 128))
        case = {"op": op, "tokens": _log(rng, 1, 4096), "experts": experts, "top_k": rng.randint(1, min(8, experts)),
                "n": _width(rng, 128, 11008 // 4), "k": _width(rng, 128, 4096)}
        if op == "experts_out":
            case["n"], case["k"] = case["k"], case["n"]
        if experts * case["n"] * case["k"] <= 64 * 1376 * 4096 and case["tokens"] * case["top_k"] * case["n"] * case["k"] <= 4096 * 6 * 1376 * 4096:
            return case


def _in_use(case):
    """Experts that some token is routed to, where tokens choose evenly: somewhat fewer where some are preferred."""
    return case["experts"] * (1 - (1 - case["top_k"] / case["experts"]) ** case["tokens"])


def work(case):
    op = case["op"]
    if op == "route":
        t, k, e = case["tokens"], case["top_k"], case["experts"]
        return {"bytes": t * e * (4 if case["dtype"] == "f32" else 2) + 12 * t * k + 4 * (e + 1) + (4 * e if case["bias"] else 0),
                "flops": 4 * t * e}
    if op == "combine":
        t, k, d = case["tokens"], case["top_k"], case["d"]
        return {"bytes": 2 * t * d * (k + (2 if case["residual"] else 1)) + 4 * t * k, "flops": 2 * t * k * d}
    n, k = case["n"], case["k"]
    kb, nb = -(-k // BLOCK), -(-n // BLOCK)
    if op == "linear":
        m = case["m"]
        return {"bytes": (m + n) * k + (m + nb) * kb + 4 * (m + n) + 2 * m * n * (2 if case["residual"] else 1) + (4 * n if case["bias"] else 0),
                "flops": 2 * m * n * k}
    if op == "gated":
        m = case["m"]
        return {"bytes": (m + 2 * n) * k + (m + 2 * nb) * kb + 4 * (m + 2 * n) + m * (n + nb), "flops": 4 * m * n * k}
    rows, used = case["tokens"] * case["top_k"], _in_use(case)
    if op == "experts_gated":
        return {"bytes": case["tokens"] * (k + kb + 4) + 2 * used * (n * k + nb * kb + 4 * n) + rows * (n + nb + 4), "flops": 4 * rows * n * k}
    return {"bytes": rows * (k + kb + 4) + used * (n * k + nb * kb + 4 * n) + 2 * rows * n, "flops": 2 * rows * n * k}


# ---------------------------------------------------------------------------------------
# The number format in elementary operations
# ---------------------------------------------------------------------------------------

def _exponent(amax):
    """ceil(log2(amax / 448)) limited to [-96, 120], as int32."""
    m, x = torch.frexp(amax)  # amax = m * 2**x, m in [0.5, 1); 448 = 0.875 * 2**9
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, -96)).clamp(-96, 120)


def _pow2(e):
    return torch.ldexp(torch.ones((), device=e.device), e)


def _blocks(u):
    """u [rows, d] as [rows, ceil(d / 128), 128], zeros after its end."""
    rows, d = u.shape
    nb = -(-d // BLOCK)
    return torch.nn.functional.pad(u, (0, nb * BLOCK - d)).view(rows, nb, BLOCK)


def _codes(u):
    """(codes [rows, d], exponent bytes [rows, ceil(d / 128)]) of fp32 u by 1 x 128 blocks."""
    v = _blocks(u)
    e = _exponent(v.abs().amax(-1))
    c = (v * _pow2(-e)[..., None]).to(F8)
    return c.view(u.shape[0], -1)[:, :u.shape[1]], (e + 127).to(torch.uint8)


def _values(c, e):
    """fp32 of codes by 1 x 128 blocks."""
    return (_blocks(c.float()) * _pow2(e.to(torch.int32) - 127)[..., None]).view(c.shape[0], -1)[:, :c.shape[1]]


def _weights(w):
    """fp32 of weights (codes, exponents, scale) [..., n, k]."""
    c, e, s = w
    n, k = c.shape[-2:]
    e = _pow2(e.to(torch.int32) - 127).repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k]
    return c.float() * e * s[..., None]


def _padded(c, step=16):
    """The same values in rows whose pitch is a multiple of `step` elements, as codes are kept."""
    out = torch.zeros(*c.shape[:-1], -(-c.shape[-1] // step) * step, dtype=torch.uint8, device=c.device)[..., :c.shape[-1]]
    out.copy_(c.view(torch.uint8))
    return out.view(c.dtype)


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _made_weights(g, *shape):
    """(codes, exponents, scale) as the quantizer leaves 4-bit weights: whole numbers, exponents of one, a step for each row."""
    n, k = shape[-2:]
    c = (2.5 * _randn(g, *shape)).round_().clamp_(-8, 7).to(F8)
    e = torch.full((*shape[:-2], -(-n // BLOCK), -(-k // BLOCK)), 127, dtype=torch.uint8, device="cuda")
    s = (0.4 / math.sqrt(k)) * (0.5 + torch.rand(*shape[:-1], generator=g, device="cuda"))
    return _padded(c), _padded(e, 4), s


def _made_rows(g, rows, d, product=False):
    """(codes, exponents): normed activations with outlier channels, or products of two."""
    x = _randn(g, rows, d)
    if product:
        x *= _randn(g, rows, d)
    x[:, ::97] *= 20.0
    c, e = _codes(x)
    return _padded(c), _padded(e, 4)


def _made_routes(g, case):
    """(expert of each position, offsets, order): tokens choose at random, some experts oftener than others."""
    t, experts, k = case["tokens"], case["experts"], case["top_k"]
    ids = (_randn(g, t, experts) + 0.4 * _randn(g, experts)).topk(k, dim=-1).indices.view(-1)
    e, order = ids.sort(stable=True)
    return e, _begins(ids, experts), order.to(torch.int32)


def _begins(ids, experts):
    """Where each expert's assignments begin among the sorted ones, and where the last ends."""
    count = torch.zeros(experts + 1, dtype=torch.int64, device=ids.device)
    count.scatter_add_(0, ids + 1, torch.ones_like(ids))
    return count.cumsum(0).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    if op == "route":
        t, e = case["tokens"], case["experts"]
        logits = (1.5 * _randn(g, t, e) + 0.3 * _randn(g, e)).to(DTYPES[case["dtype"]])
        return {"op": op, "logits": logits, "bias": 0.1 * _randn(g, e) if case["bias"] else None,
                **{k: case[k] for k in ("top_k", "scores", "groups", "top_groups", "group_top", "renormalize", "scale")}}
    if op == "combine":
        t, k, d = case["tokens"], case["top_k"], case["d"]
        dtype = DTYPES[case["dtype"]]
        weights = torch.softmax(_randn(g, t, k), -1)
        return {"op": op, "y": _randn(g, t * k, d).to(dtype), "weights": weights,
                "residual": (2.0 * _randn(g, t, d)).to(dtype) if case["residual"] else None}
    n, k = case["n"], case["k"]
    if op in ("linear", "gated"):
        m = case["m"]
        a, ae = _made_rows(g, m, k)
        state = {"op": op, "a": a, "ae": ae, "ra": torch.rand(m, generator=g, device="cuda") + 0.5, "w": _made_weights(g, n, k)}
        if op == "gated":
            return state | {"up": _made_weights(g, n, k)}
        dtype = DTYPES[case["dtype"]]
        return state | {"dtype": dtype, "act": None if case["act"] == "none" else case["act"], "bias": _randn(g, n) if case["bias"] else None,
                        "residual": (2.0 * _randn(g, m, n)).to(dtype) if case["residual"] else None}
    expert, offsets, order = _made_routes(g, case)
    experts, top_k = case["experts"], case["top_k"]
    state = {"op": op, "expert": expert, "offsets": offsets, "order": order, "top_k": top_k, "w": _made_weights(g, experts, n, k)}
    if op == "experts_gated":
        a, ae = _made_rows(g, case["tokens"], k)
        return state | {"a": a, "ae": ae, "ra": torch.rand(case["tokens"], generator=g, device="cuda") + 0.5, "up": _made_weights(g, experts, n, k)}
    a, ae = _made_rows(g, case["tokens"] * top_k, k, product=True)
    return state | {"a": a, "ae": ae}


# ---------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------

def run(state):
    if own:
        from post_weight_quantization_03_gb300 import gptq
    op = state["op"]
    if op == "route":
        given = {k: state[k] for k in ("bias", "scores", "groups", "top_groups", "group_top", "renormalize", "scale")}
        ids, weights, offsets, order = (gptq.moe_route if own else _route)(state["logits"], state["top_k"], **given)
        return {"ids": ids, "weights": weights, "offsets": offsets, "order": order}
    if op == "combine":
        return (gptq.moe_combine if own else _combine)(state["y"], state["weights"], residual=state["residual"])
    if op == "linear":
        if own:
            return gptq.fp8_linear(state["a"], state["ae"], state["w"][0], state["w"][1], a_scale=state["ra"], w_scale=state["w"][2],
                                   bias=state["bias"], act=state["act"], residual=state["residual"], out_dtype=state["dtype"])
        return _linear(state)
    if op == "experts_out":
        if own:
            return gptq.fp8_experts(state["a"], state["ae"], state["w"][0], state["w"][1], state["offsets"], state["order"],
                                    w_scale=state["w"][2], out_dtype=torch.bfloat16)
        return _experts_out(state)
    if not own:
        c, e = _codes((_gated if op == "gated" else _experts_gated)(state))
    elif op == "gated":
        c, e = gptq.fp8_gated(state["a"], state["ae"], state["w"], state["up"], a_scale=state["ra"], act="silu")
    else:
        c, e = gptq.fp8_experts_gated(state["a"], state["ae"], state["w"], state["up"], state["offsets"], state["order"], state["top_k"],
                                      a_scale=state["ra"], act="silu")
    return {"codes": c, "exps": e.view(torch.float8_e8m0fnu)}


def _best(x, n):
    """Indices of the n largest along the last axis, largest first, the lowest index of equals."""
    return x.sort(dim=-1, descending=True, stable=True).indices[..., :n]


def _route(logits, top_k, bias, scores, groups, top_groups, group_top, renormalize, scale):
    x = logits.double()  # (choices next to one another may be closer than 32 bits tell)
    t, experts = x.shape
    if scores == "softmax":
        s = torch.exp(x - x.amax(-1, keepdim=True))
        s = s / s.sum(-1, keepdim=True)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    c = x if bias is None and groups == 1 else s if bias is None else s + bias.double()
    if groups > 1:
        of_group = c.view(t, groups, -1)
        value = of_group.sort(dim=-1, descending=True).values[..., :group_top].sum(-1)
        open_ = torch.zeros_like(value).scatter_(-1, _best(value, top_groups), 1.0)
        c = torch.where(open_[..., None] > 0, of_group, -math.inf).view(t, experts)
    ids = _best(c, top_k)
    w = s.gather(-1, ids)
    if renormalize:
        w = w / w.sum(-1, keepdim=True)
    flat = ids.reshape(-1)
    return ids.to(torch.int32), (w * scale).float(), _begins(flat, experts), flat.sort(stable=True).indices.to(torch.int32)


def _act(x, act):
    if act == "relu":
        return x.clamp(min=0.0)
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * 0.5 ** 0.5))
    return x


def _linear(state):
    x = _values(state["a"], state["ae"]) @ _weights(state["w"]).t() * state["ra"][:, None]
    if state["bias"] is not None:
        x = x + state["bias"]
    x = _act(x, state["act"])
    if state["residual"] is not None:
        x = x + state["residual"].float()
    return x.to(state["dtype"])


def _gated(state):
    a = _values(state["a"], state["ae"]) * state["ra"][:, None]
    return _act(a @ _weights(state["w"]).t(), "silu") * (a @ _weights(state["up"]).t())


def _by_expert(state, rows, weights):
    """Each of the `rows`, which are sorted by expert, times its expert's weights: one batched product of the experts in use."""
    e, offsets = state["expert"], state["offsets"].long()
    used, at = e.unique(return_inverse=True)
    rank = torch.arange(len(e), device=e.device) - offsets[e]
    padded = torch.zeros(len(used), int(rank.max()) + 1, rows.shape[1], device=rows.device)
    padded[at, rank] = rows
    return (padded @ _weights([p.view(torch.uint8)[used].view(p.dtype) for p in weights[:2]] + [weights[2][used]]).transpose(1, 2))[at, rank]


def _experts_gated(state):
    a = _values(state["a"], state["ae"]) * state["ra"][:, None]
    rows = a[state["order"].long() // state["top_k"]]
    return _act(_by_expert(state, rows, state["w"]), "silu") * _by_expert(state, rows, state["up"])


def _experts_out(state):
    y = _by_expert(state, _values(state["a"], state["ae"]), state["w"])
    out = torch.empty_like(y)
    out[state["order"].long()] = y
    return out.to(torch.bfloat16)


def _combine(y, weights, residual):
    t, k = weights.shape
    x = (y.float().view(t, k, -1) * weights[..., None]).sum(1)
    if residual is not None:
        x = x + residual.float()
    return x.to(y.dtype)


# ---------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------

def _matrix64(c, e, row_block):
    """fp64 of the codes of a matrix [rows, d], exponents by row_block x 128 blocks."""
    rows, d = c.shape
    of_row, of_col = torch.arange(rows, device=c.device) // row_block, torch.arange(d, device=c.device) // BLOCK
    return c.double() * torch.exp2(e.double() - 127)[of_row][:, of_col]


def _silu64(x):
    return x * torch.sigmoid(x)


def _coded64(v):
    """What codes and exponents of v stand for before they are rounded to 8 bits: elements over their block's scale, the scales."""
    rows, d = v.shape
    nb = -(-d // BLOCK)
    u = torch.zeros(rows, nb * BLOCK, dtype=torch.float64, device=v.device)
    u[:, :d] = v
    u = u.view(rows, nb, BLOCK)
    amax = u.abs().amax(-1)
    scale = torch.exp2(torch.where(amax > 0, torch.ceil(torch.log2(amax / 448.0)), -96.0).clamp(-96, 120))
    return {"codes": (u / scale[..., None]).view(rows, -1)[:, :d], "exps": scale}


def _route64(state):
    x = state["logits"].double()
    t, experts = x.shape
    s = torch.softmax(x, -1) if state["scores"] == "softmax" else torch.sigmoid(x)
    c = x.clone() if state["bias"] is None and state["groups"] == 1 else s + (0.0 if state["bias"] is None else state["bias"].double())
    size = experts // state["groups"]
    if state["groups"] > 1:
        value = c.view(t, -1, size).topk(state["group_top"], dim=-1).values.sum(-1)
        closed = torch.ones_like(value, dtype=torch.bool)
        closed.scatter_(-1, value.topk(state["top_groups"], dim=-1).indices, False)
        c[closed.repeat_interleave(size, -1)] = -math.inf
    ids = []
    for _ in range(state["top_k"]):
        ids.append(c.argmax(-1))
        c.scatter_(-1, ids[-1][:, None], -math.inf)
    ids = torch.stack(ids, -1)
    w = s.gather(-1, ids) * state["scale"]
    if state["renormalize"]:
        w = w / s.gather(-1, ids).sum(-1, keepdim=True)
    return {"ids": None, "weights": w, "offsets": None, "order": None}


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _route64(state)
    if op == "combine":
        y, w = state["y"].double().view(*state["weights"].shape, -1), state["weights"].double()
        out = torch.einsum("tk,tkd->td", w, y)
        return out if state["residual"] is None else out + state["residual"].double()
    a = _matrix64(state["a"], state["ae"], 1)
    if "ra" in state:
        a *= state["ra"].double()[:, None]

    def product(rows, w, i=None):
        c, e, s = w if i is None else [p[i] for p in w]
        return (rows @ _matrix64(c, e, BLOCK).t()) * s.double()

    if op == "linear":
        x = product(a, state["w"])
        if state["bias"] is not None:
            x += state["bias"].double()
        act = state["act"]
        x = _silu64(x) if act == "silu" else torch.nn.functional.gelu(x) if act == "gelu" else torch.relu(x) if act == "relu" else x
        return x if state["residual"] is None else x + state["residual"].double()
    if op == "gated":
        return _coded64(_silu64(product(a, state["w"])) * product(a, state["up"]))
    begins, order = state["offsets"].tolist(), state["order"].long()
    out = torch.zeros(len(order), case["n"], dtype=torch.float64, device=a.device)
    for i, (lo, hi) in enumerate(zip(begins, begins[1:])):
        if lo == hi:
            continue
        if op == "experts_gated":
            rows = a[order[lo:hi] // state["top_k"]]
            out[lo:hi] = _silu64(product(rows, state["w"], i)) * product(rows, state["up"], i)
        else:
            out[order[lo:hi]] = product(a[lo:hi], state["w"], i)
    return _coded64(out) if op == "experts_gated" else out
