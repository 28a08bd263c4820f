"""The 8-bit serving operators: what is measured, on which sizes, and their plain forms.

Number format (all three operators): e4m3 codes with one exponent byte E (value 2**(E - 127)) for
each block.  For a block whose largest magnitude is a, e = ceil(log2(a / 448)) limited to
[-96, 120] (a block of zeros: -96), E = e + 127 and code = e4m3(x * 2**-e).

* norm:      h = x + r;  u = h * w;  rstd = (mean(h * h) + eps) ** -0.5;  codes and exponents of u
             by 1 x 128 blocks, rstd as the row's scale (y = rstd * 2**(E - 127) * code);
* product:   out[m, n] = ra[m] * sum_k 2**(EA[m, k/128] + EW[n/128, k/128] - 254) a[m, k] w[n, k];
* attention: T new tokens of each sequence appended to a cache of 64-token blocks (an exponent
             for each block and head), then causal attention of their queries over the cache.
"""

import math

import torch

own = False

BLOCK = 128       # elements of a scale block of the norm's output and of the product
TOKENS = 64       # tokens of a cache block
EPS = 1e-6
F8 = torch.float8_e4m3fn
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------

def listed():
    return [
        # one token of a 4096-wide decoder: latency
        {"name": "norm 1x4096", "op": "norm", "rows": 1, "d": 4096, "dtype": "bf16", "residual": True},
        # a ragged batch, a width that ends inside a block, the first norm (no residual)
        {"name": "norm 333x5000", "op": "norm", "rows": 333, "d": 5000, "dtype": "f16", "residual": False},
        # a long prompt of the widest model here
        {"name": "norm 8192x8192", "op": "norm", "rows": 8192, "d": 8192, "dtype": "bf16", "residual": True},
        # attention output projection, one token
        {"name": "product 1x4096x4096", "op": "product", "m": 1, "n": 4096, "k": 4096, "dtype": "bf16"},
        # up projection, a batch of sequences decoding together
        {"name": "product 24x11008x4096", "op": "product", "m": 24, "n": 11008, "k": 4096, "dtype": "bf16"},
        # down projection of the widest layer, a full decoding batch
        {"name": "product 128x8192x28672", "op": "product", "m": 128, "n": 8192, "k": 28672, "dtype": "bf16"},
        # down projection of a short prompt, ragged
        {"name": "product 515x4096x11008", "op": "product", "m": 515, "n": 4096, "k": 11008, "dtype": "f16"},
        # up projection of a long prompt
        {"name": "product 8192x11008x4096", "op": "product", "m": 8192, "n": 11008, "k": 4096, "dtype": "bf16"},
        # one sequence, one token, a short history: latency
        {"name": "attention 1x1 of 500", "op": "attention", "seqs": 1, "new": 1, "longest": 500, "heads": 32, "kv_heads": 32,
         "dim": 128, "dtype": "bf16"},
        # a full decoding batch with histories of many lengths, eight queries to a head
        {"name": "attention 48x1 of 8000", "op": "attention", "seqs": 48, "new": 1, "longest": 8000, "heads": 64, "kv_heads": 8,
         "dim": 128, "dtype": "bf16"},
        # a prompt into an empty cache
        {"name": "attention 1x4096 of 4096", "op": "attention", "seqs": 1, "new": 4096, "longest": 4096, "heads": 32, "kv_heads": 8,
         "dim": 128, "dtype": "bf16"},
        # a ragged chunk of two prompts behind long histories, small heads
        {"name": "attention 2x777 of 16000", "op": "attention", "seqs": 2, "new": 777, "longest": 16000, "heads": 32, "kv_heads": 8,
         "dim": 64, "dtype": "f16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: whole blocks, a multiple of 8, or any number."""
    v = _log(rng, lo, hi)
    step = rng.choice((BLOCK, BLOCK, 8, 1))
    return max(lo, v // step * step)


def draw(rng):
    op = rng.choice(("norm", "product", "attention"))
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 8192), "d": _width(rng, 128, 8192), "dtype": rng.choice(("bf16", "f16", "f32")),
                "residual": rng.random() < 0.7}
    if op == "product":
        while True:
            case = {"op": op, "m": _log(rng, 1, 8192), "n": _width(rng, 128, 11008), "k": _width(rng, 128, 28672),
                    "dtype": rng.choice(("bf16", "f16"))}
            if case["m"] * case["n"] * case["k"] <= 8192 * 11008 * 4096:
                return case
    while True:
        kv = rng.choice((1, 2, 4, 8, 8, 32))
        group = rng.choice((1, 2, 3, 4, 7, 8, 16)) if kv < 32 else 1
        new = _log(rng, 1, 8) if rng.random() < 0.5 else _log(rng, 9, 4096)
        case = {"op": op, "seqs": _log(rng, 1, 48), "new": new, "longest": _log(rng, max(64, new), 32768), "heads": kv * group,
                "kv_heads": kv, "dim": rng.choice((64, 128)), "dtype": rng.choice(("bf16", "f16"))}
        w = work(case)
        if w["flops"] <= 1.4e11 and w["bytes"] <= 5.5e8 and case["seqs"] * new * case["heads"] * case["longest"] <= 1.2e9:
            return case


def _lengths(case):
    """Tokens of each sequence, the new ones included: the first has the most, the others between that and half of it."""
    longest, new = case["longest"], case["new"]
    return [max(new, longest - (i * 977) % (longest // 2 + 1)) for i in range(case["seqs"])]


def work(case):
    if case["op"] == "norm":
        n, es = case["rows"] * case["d"], 4 if case["dtype"] == "f32" else 2
        blocks = case["rows"] * -(-case["d"] // BLOCK)
        return {"bytes": n * (es * (3 if case["residual"] else 2) + 1) + blocks + case["rows"] * 4 + case["d"] * es, "flops": 6 * n}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        kb = -(-k // BLOCK)
        return {"bytes": (m + n) * k + (m + -(-n // BLOCK)) * kb + 4 * m + 2 * m * n, "flops": 2 * m * n * k}
    new, d = case["new"], case["dim"]
    seen = sum(_lengths(case))
    pairs = sum(new * length - new * (new - 1) // 2 for length in _lengths(case))
    fresh = case["seqs"] * new
    return {"bytes": 2 * d * case["kv_heads"] * (seen + 2 * fresh) + 2 * 2 * d * case["heads"] * fresh,
            "flops": 4 * d * case["heads"] * pairs}


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


def _value(exps):
    """The values 2**(E - 127) that exponent bytes stand for."""
    return _pow2(exps.to(torch.int32) - 127)


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


def _padded(c, step=16):
    """The same values in rows whose pitch is a multiple of `step` elements, as codes are kept."""
    out = torch.zeros(c.shape[0], -(-c.shape[1] // step) * step, dtype=torch.uint8, device=c.device)[:, :c.shape[1]]
    out.copy_(c.view(torch.uint8))
    return out.view(c.dtype)


# ---------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)

    dtype = DTYPES[case["dtype"]]
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        x = randn(rows, d)
        x[:, ::97] *= 20.0                                   # outlier channels
        w = 1.0 + 0.2 * randn(d)
        return {"op": "norm", "x": x.to(dtype), "r": (2.0 * randn(rows, d)).to(dtype) if case["residual"] else None, "w": w.to(dtype)}
    if case["op"] == "product":
        m, n, k = case["m"], case["n"], case["k"]
        a = randn(m, k)
        a[:, ::97] *= 20.0
        ac, ae = _codes(a)
        w = randn(n, k) * 0.02
        nb, kb = -(-n // BLOCK), -(-k // BLOCK)
        wb = torch.nn.functional.pad(w, (0, kb * BLOCK - k, 0, nb * BLOCK - n)).view(nb, BLOCK, kb, BLOCK)
        e = _exponent(wb.abs().amax((1, 3)))
        wc = (wb * _pow2(-e)[:, None, :, None]).to(F8).view(nb * BLOCK, kb * BLOCK)[:n, :k]
        return {"op": "product", "a": _padded(ac), "ae": _padded(ae, 4), "ra": torch.rand(m, generator=g, device="cuda") + 0.5,
                "w": _padded(wc), "we": _padded((e + 127).to(torch.uint8), 4), "dtype": dtype}
    b, new, d, kv = case["seqs"], case["new"], case["dim"], case["kv_heads"]
    lengths = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    most = -(-case["longest"] // TOKENS)
    pages = torch.randperm(b * most, generator=g, device="cuda").to(torch.int32).view(b, most)

    def filled(outliers):
        v = randn(b * most, kv, TOKENS, d)
        if outliers:
            v[..., ::31] *= 4.0                              # keys have channels that stand out
        e = _exponent(v.abs().amax((2, 3)))
        return (v * _pow2(-e)[..., None, None]).to(F8), (e + 127).to(torch.uint8)

    kc, ke = filled(True)
    vc, ve = filled(False)
    return {"op": "attention", "q": randn(b, new, case["heads"], d).to(dtype), "k": randn(b, new, kv, d).to(dtype),
            "v": randn(b, new, kv, d).to(dtype), "cache": (kc, vc.transpose(2, 3).contiguous(), ke, ve), "table": pages,
            "start": lengths - new, "lengths": lengths}


# ---------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------

def run(state):
    if own:
        from post_weight_quantization_03_gb300 import gptq
    if state["op"] == "norm":
        if own:
            c, e, rstd, h = gptq.rmsnorm_fp8(state["x"], state["w"], residual=state["r"], eps=EPS)
        else:
            c, e, rstd, h = _norm(state["x"], state["w"], state["r"])
        return {"codes": c, "exps": e.view(torch.float8_e8m0fnu), "rstd": rstd, "h": h}
    if state["op"] == "product":
        if own:
            return gptq.fp8_matmul(state["a"], state["ae"], state["w"], state["we"], a_scale=state["ra"], out_dtype=state["dtype"])
        return _product(state["a"], state["ae"], state["w"], state["we"], state["ra"], state["dtype"])
    cache = state["cache"]
    if own:
        gptq.kv8_append(cache, state["k"], state["v"], state["table"], state["start"])
        out = gptq.kv8_attention(state["q"], cache, state["table"], state["lengths"])
    else:
        _append(cache[0], cache[2], state["k"], state["table"], state["start"])
        _append(cache[1].transpose(2, 3), cache[3], state["v"], state["table"], state["start"])
        out = _attention(state["q"], cache, state["table"], state["lengths"])
    return {"out": out, "k": cache[0], "v": cache[1], "k_exps": cache[2].view(torch.float8_e8m0fnu),
            "v_exps": cache[3].view(torch.float8_e8m0fnu)}


def _norm(x, w, r):
    h = x.float() if r is None else x.float() + r.float()
    c, e = _codes(h * w.float())
    return c, e, torch.rsqrt(h.square().mean(-1) + EPS), h.to(x.dtype)


def _product(a, ae, w, we, ra, dtype):
    (m, k), n = a.shape, w.shape[0]
    av = (_blocks(a.float()) * _value(ae)[..., None]).view(m, -1)
    wv = _blocks(w.float()) * _value(we).repeat_interleave(BLOCK, 0)[:n, :, None]
    return (av @ wv.view(n, -1).t() * ra[:, None]).to(dtype)


def _append(codes, exps, x, table, start):
    """x [seqs, new, kv_heads, dim] into codes [blocks, kv_heads, 64, dim] at the tokens from `start` on, in place."""
    new = x.shape[1]
    blk = (start // TOKENS)[:, None] + torch.arange((new + 126) // TOKENS, device=x.device, dtype=torch.int32)
    pos = blk[..., None] * TOKENS + torch.arange(TOKENS, device=x.device, dtype=torch.int32)
    begin = start[:, None, None]
    fresh, old = (pos >= begin) & (pos < begin + new), pos < begin
    page = table.gather(1, blk.clamp(max=table.shape[1] - 1).long()).long()
    seq = torch.arange(x.shape[0], device=x.device)[:, None, None]
    v = x[seq, (pos - begin).clamp(0, new - 1).long()].transpose(2, 3).float()  # [seqs, blocks, kv_heads, 64, dim]
    f, o = fresh[:, :, None, :, None], old[:, :, None, :, None]
    need = _exponent(torch.where(f, v.abs(), 0.0).amax((-2, -1)))
    was = exps[page].to(torch.int32) - 127
    e = torch.where(old.any(-1)[..., None], torch.maximum(was, need), need)
    held = codes[page]                                                          # slots after the new tokens stay as they are
    v = torch.where(f, v * _pow2(-e)[..., None, None], held.float() * torch.where(o, _pow2(was - e)[..., None, None], 1.0))
    there = fresh.any(-1)
    codes[page[there]] = v[there].to(F8)
    exps[page[there]] = (e + 127).to(torch.uint8)[there]


def _attention(query, cache, table, lengths):
    kc, vc, ke, ve = cache
    b, new, heads, d = query.shape
    kv, s = kc.shape[1], table.shape[1] * TOKENS
    page = table.long()
    k = (kc[page].float() * _value(ke[page])[..., None, None]).transpose(1, 2).reshape(b, kv, s, d)
    v = (vc[page].float() * _value(ve[page])[..., None, None]).permute(0, 2, 1, 4, 3).reshape(b, kv, s, d)
    q = query.float().view(b, new, kv, heads // kv, d).permute(0, 2, 3, 1, 4).reshape(b, kv, -1, d)
    x = (q @ k.transpose(2, 3) * d ** -0.5).view(b, kv, -1, new, s)
    last = lengths[:, None] - new + torch.arange(new, device=q.device)  # the last token that a query sees
    x = torch.where((torch.arange(s, device=q.device) <= last[..., None])[:, None, None], x, -math.inf)
    x = torch.exp(x - x.amax(-1, keepdim=True))
    x /= x.sum(-1, keepdim=True)
    out = x.view(b, kv, -1, s) @ v
    return out.view(b, kv, -1, new, d).permute(0, 3, 1, 2, 4).reshape(b, new, heads, d).to(query.dtype)


# ---------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------

def _nearest(x):
    """The e4m3 value next to each x (|x| <= 448; ties to the even one): multiples of 2**(p - 3) where
    2**p <= |x| < 2**(p + 1), of 2**-9 below 2**-6."""
    p = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(p - 3)
    return torch.round(x / step) * step


def _scale64(amax):
    """2**e of blocks with these largest magnitudes."""
    e = torch.ceil(torch.log2(amax / 448.0))
    return torch.exp2(torch.where(amax > 0, e, -96.0).clamp(-96, 120))


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "norm":
        x, w = state["x"].double(), state["w"].double()
        h = x if state["r"] is None else x + state["r"].double()
        rows, d = h.shape
        nb = -(-d // BLOCK)
        u = torch.zeros(rows, nb * BLOCK, dtype=torch.float64, device=h.device)
        u[:, :d] = h * w
        u = u.view(rows, nb, BLOCK)
        scale = _scale64(u.abs().amax(-1))
        codes = _nearest(u / scale[..., None]).view(rows, -1)[:, :d]
        return {"codes": codes, "exps": scale, "rstd": (h.square().sum(-1) / d + EPS) ** -0.5, "h": h}
    if case["op"] == "product":
        m, k = state["a"].shape
        n = state["w"].shape[0]
        of_k = torch.arange(k, device="cuda") // BLOCK
        of_n = torch.arange(n, device="cuda") // BLOCK
        a = state["a"].double() * torch.exp2(state["ae"].double() - 127)[:, of_k]
        w = state["w"].double() * torch.exp2(state["we"].double() - 127)[of_n][:, of_k]
        return state["ra"].double()[:, None] * (a @ w.t())
    q, (kc, vc, ke, ve) = state["q"].double(), state["cache"]
    b, new, heads, d = q.shape
    kv = kc.shape[1]
    group = heads // kv
    k, v, ks, vs = kc.double(), vc.double(), torch.exp2(ke.double() - 127), torch.exp2(ve.double() - 127)
    out = torch.zeros(b, new, heads, d, dtype=torch.float64, device=q.device)
    table, lengths = state["table"].tolist(), state["lengths"].tolist()
    slot = torch.arange(TOKENS, device=q.device)
    for i, length in enumerate(lengths):
        first = length - new
        for blk in range(first // TOKENS, (length - 1) // TOKENS + 1):
            page, t0 = table[i][blk], blk * TOKENS
            lo, hi = max(first, t0), min(length, t0 + TOKENS)
            for codes, scales, x in ((k[page], ks[page], state["k"][i]), (v[page].transpose(1, 2), vs[page], state["v"][i])):
                x = x[lo - first:hi - first].double().transpose(0, 1)                 # [kv_heads, tokens, dim]
                scale = _scale64(x.abs().amax((1, 2)))
                if lo > t0:
                    scale = torch.maximum(scale, scales)
                kept = codes * torch.where(slot < lo - t0, (scales / scale)[:, None], 1.0)[..., None]
                kept[:, lo - t0:hi - t0] = x / scale[:, None, None]
                codes.copy_(_nearest(kept))
                scales.copy_(scale)
        pages = torch.tensor(table[i][:(length - 1) // TOKENS + 1], device=q.device)
        last = first + torch.arange(new, device=q.device)
        seen = torch.arange(len(pages) * TOKENS, device=q.device) <= last[:, None]
        keys = (k[pages] * ks[pages][..., None, None]).transpose(0, 1).reshape(kv, -1, d)
        values = (v[pages] * vs[pages][..., None, None]).permute(1, 0, 3, 2).reshape(kv, -1, d)
        for head in range(heads):
            x = q[i, :, head] @ keys[head // group].t() / math.sqrt(d)
            out[i, :, head] = torch.softmax(x.masked_fill(~seen, -math.inf), -1) @ values[head // group]
    return {"out": out, "k": k, "v": v, "k_exps": ks, "v_exps": vs}
