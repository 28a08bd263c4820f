"""Independent 64-bit definitions of the 8-bit serving operators (NumPy; no library code).

Number format: e4m3 codes with one exponent byte E per block, value ``code * 2**(E - 127)``,
``e = ceil(log2(amax / 448))`` limited to [-96, 120] over the block's finite elements (-96 for
zeros), codes rounded to nearest even, non-finite elements NaN.
"""

from __future__ import annotations

import math

import numpy as np

BLOCK = 128
TOKENS = 64
E_MIN, E_MAX, BIAS = -96, 120, 127
NAN_CODE = 0x7F


def decode_table():
    """The 256 values of e4m3: sign, 4 exponent bits (bias 7), 3 fraction bits; 0x7F NaN."""
    out = np.empty(256)
    for b in range(256):
        s, e, f = b >> 7, b >> 3 & 15, b & 7
        v = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out[b] = math.nan if b & 0x7F == NAN_CODE else -v if s else v
    return out


TABLE = decode_table()


def decode(codes):
    return TABLE[np.asarray(codes, np.uint8)]


def encode(x):
    """Nearest e4m3 code of values with |x| <= 448 (ties to the even code), NaN for the rest."""
    x = np.asarray(x, np.float64)
    pos = TABLE[:NAN_CODE]                       # ascending: code order is value order
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(pos, a), 0, len(pos) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isfinite(x), code, NAN_CODE).astype(np.uint8)


def block_exponent(amax):
    if amax == 0:
        return E_MIN
    m, x = math.frexp(amax)                      # amax = m 2^x;  448 = 0.875 * 2^9
    return min(max(x - 9 + (1 if m > 0.875 else 0), E_MIN), E_MAX)


def _amax(x):
    f = np.abs(x[np.isfinite(x)])
    return float(f.max()) if f.size else 0.0


def quantize(x, row_block=1):
    """(codes, exponent bytes) of a matrix by ``row_block x 128`` blocks."""
    x = np.asarray(x, np.float64)
    rows, d = x.shape
    codes = np.empty((rows, d), np.uint8)
    exps = np.empty((-(-rows // row_block), -(-d // BLOCK)), np.uint8)
    for i in range(exps.shape[0]):
        for j in range(exps.shape[1]):
            at = np.s_[i * row_block:(i + 1) * row_block, j * BLOCK:(j + 1) * BLOCK]
            e = block_exponent(_amax(x[at]))
            exps[i, j] = e + BIAS
            codes[at] = encode(x[at] * 2.0 ** -e)
    return codes, exps


def dequantize(codes, exps, row_block=1):
    s = 2.0 ** (exps.astype(np.float64) - BIAS)
    s = np.repeat(np.repeat(s, row_block, 0), BLOCK, 1)[:codes.shape[0], :codes.shape[1]]
    return decode(codes) * s


def rmsnorm(x, w, r=None, eps=1e-6):
    """(codes, exps, rstd, h) with h and u = h * w taken in fp32 as the format's input is
    defined, the mean of squares in 64 bits."""
    h = np.asarray(x, np.float32)
    if r is not None:
        h = h + np.asarray(r, np.float32)
    with np.errstate(invalid="ignore", over="ignore"):
        u = h * np.asarray(w, np.float32)
    codes, exps = quantize(u)
    return codes, exps, (np.square(h.astype(np.float64)).mean(1) + eps) ** -0.5, h


def matmul(a, ae, w, we, ra=None, rw=None):
    """(product, sum of the magnitudes of its terms)."""
    A, W = dequantize(a, ae), dequantize(w, we, BLOCK)
    f = np.ones((A.shape[0], W.shape[0]))
    if ra is not None:
        f = f * np.asarray(ra, np.float64)[:, None]
    if rw is not None:
        f = f * np.asarray(rw, np.float64)[None]
    return A @ W.T * f, np.abs(A) @ np.abs(W).T * np.abs(f)


def kv_append(cache, k, v, table, start):
    """New tokens [seqs, new, kv, d] into copies of the cache's arrays."""
    kc, vc, ke, ve = (np.array(t) for t in cache)
    n_blocks, kv = ke.shape
    new = k.shape[1]
    for s in range(k.shape[0]):
        st = int(start[s])
        if st < 0 or new == 0:
            continue
        for blk in range(st // TOKENS, (st + new - 1) // TOKENS + 1):
            if blk >= table.shape[1] or not 0 <= table[s, blk] < n_blocks:
                continue
            page, t0 = int(table[s, blk]), blk * TOKENS
            lo, hi = max(st, t0) - t0, min(st + new, t0 + TOKENS) - t0
            for h in range(kv):
                x = k[s, lo + t0 - st:hi + t0 - st, h].astype(np.float64)
                y = v[s, lo + t0 - st:hi + t0 - st, h].astype(np.float64)
                marked = ~np.isfinite(y).all(1)
                for codes, exps, z in ((kc[page, h], ke, x), (vc[page, h].T, ve, y)):
                    e = block_exponent(_amax(z))
                    if lo > 0:
                        was = int(exps[page, h]) - BIAS
                        e = max(e, was)
                        if e > was:
                            codes[:lo] = encode(decode(codes[:lo]) * 2.0 ** (was - e))
                    exps[page, h] = e + BIAS
                    codes[lo:hi] = encode(z * 2.0 ** -e)
                kc[page, h, lo:hi][marked] = NAN_CODE
                vt = vc[page, h].T[lo:hi]
                vt[~np.isfinite(y)] = 0
    return kc, vc, ke, ve


def kv_attention(q, cache, table, lengths, scale=None, causal=True):
    """(out, sum of p |v|, largest sum |q k| scale) in 64 bits."""
    kc, vc, ke, ve = (np.asarray(t) for t in cache)
    n_blocks, kv = ke.shape
    seqs, new, heads, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    terms = 0.0
    for s in range(seqs):
        length = min(max(int(lengths[s]), 0), table.shape[1] * TOKENS)
        nb = -(-length // TOKENS)
        pages = table[s, :nb].astype(np.int64)
        there = (pages >= 0) & (pages < n_blocks)
        pg = np.where(there, pages, 0)
        pos = np.arange(nb * TOKENS)
        base = np.repeat(there, TOKENS) & (pos < length)
        for h in range(kv):
            if nb == 0:
                continue
            K = (decode(kc[pg, h]) * 2.0 ** (ke[pg, h].astype(float) - BIAS)[:, None, None]).reshape(-1, d)
            V = (decode(vc[pg, h]) * 2.0 ** (ve[pg, h].astype(float) - BIAS)[:, None, None])
            V = V.transpose(0, 2, 1).reshape(-1, d)
            for t in range(new):
                see = base & (pos <= length - new + t) if causal else base
                if not see.any():
                    continue
                for g in range(heads // kv):
                    qv = q[s, t, h * (heads // kv) + g].astype(np.float64)
                    x = K[see] @ qv * scale
                    p = np.exp(x - x.max())
                    p /= p.sum()
                    out[s, t, h * (heads // kv) + g] = p @ V[see]
                    mag[s, t, h * (heads // kv) + g] = p @ np.abs(V[see])
                    if np.isfinite(x).all():
                        terms = max(terms, float((np.abs(K[see]) @ np.abs(qv)).max() * abs(scale)))
    return out, mag, terms
