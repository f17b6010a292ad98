"""Plain 64-bit forms of the dense operators (numpy, scipy's erfc), and how far
32-bit arithmetic with one final rounding may be from them."""
from __future__ import annotations

import numpy as np
import torch
from scipy.special import erfc

U32 = 2.0 ** -24                       # half a step of fp32, relative
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
BLOCK = 32


def f64(t):
    """a tensor (any type) as a float64 array"""
    return t.detach().to("cpu").to(torch.float64).numpy()


# ------------------------------------------------------------- activations --

def phi_cdf(z):
    return 0.5 * erfc(-z / np.sqrt(2.0))


def act(z, kind):
    with np.errstate(over="ignore"):
        return {"none": lambda: z, "relu": lambda: np.where(z < 0, 0.0, z),
                "silu": lambda: z / (1 + np.exp(-z)), "gelu": lambda: z * phi_cdf(z)}[kind]()


def act_slope(z, kind):
    with np.errstate(over="ignore"):
        if kind == "relu":
            return np.where(z > 0, 1.0, np.where(z <= 0, 0.0, z))
        if kind == "silu":
            s = 1 / (1 + np.exp(-z))
            return s * (1 + z * (1 - s))
        return phi_cdf(z) + z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)


def slope_terms(z, kind):
    """sum of the magnitudes of the terms that act_slope adds (what a rounding
    of each of them is relative to)"""
    with np.errstate(over="ignore"):
        if kind == "relu":
            return np.ones_like(z)
        if kind == "silu":
            s = 1 / (1 + np.exp(-z))
            return s * (1 + np.abs(z) * (1 - s) + np.abs(z))
        return phi_cdf(z) + np.abs(z) * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)


def act_rel(z, kind):
    """relative error of the activation in 32 bits: 16 roundings' worth for the
    library functions and the few operations around them; erfc and exp of an
    argument x that is itself rounded by 2^-24 are off by (2 x^2) 2^-24 = z^2 2^-24
    more (d log erfc(x) / dx tends to -2 x, with x = z / sqrt 2)"""
    if kind in ("none", "relu"):
        return 0.0 * z
    return (16 + (np.minimum(np.abs(z), 40.0) ** 2 if kind == "gelu" else 0.0)) * U32


# ------------------------------------------------------------------ linear --

def linear(x, w, bias, residual, kind):
    """(out, error scale of z): x, w, ... float64 arrays"""
    z = x @ w
    size = np.abs(x) @ np.abs(w)
    if bias is not None:
        z = z + bias
        size = size + np.abs(bias)
    out = act(z, kind)
    if residual is not None:
        out = out + residual
    return out, z, size


def linear_tol(x, w, bias, residual, kind, out, z, size, dtype):
    """d products and d + 1 additions in 32 bits, each off by at most one step
    (2^-23) of the running magnitude, which sum |x w| bounds; |act'| <= 1.13;
    the activation's own error; residual added with one rounding; rounded once"""
    d = x.shape[1]
    err = 1.13 * (2 * d + 4) * 2.0 ** -23 * size + act_rel(z, kind) * np.abs(act(z, kind))
    if residual is not None:
        err = err + U32 * (np.abs(residual) + np.abs(out))
    return err + HALF[dtype] * (np.abs(out) + err) + TINY[dtype]


# -------------------------------------------------------- 8-bit checkpoint --

def e4m3_values():
    """the 256 codes' values, from the format: sign, 4 exponent bits (bias 7), 3 fraction bits"""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = np.nan if c & 127 == 127 else (-a if c & 128 else a)
    return v


E4M3 = e4m3_values()


def scale_exponents(z):
    """[T, nb] e of each block of 32 columns: least e with max finite |z| <= 448 2^e"""
    T, f = z.shape
    nb = -(-f // BLOCK)
    a = np.zeros((T, nb * BLOCK))
    with np.errstate(invalid="ignore"):
        a[:, :f] = np.where(np.isfinite(z), np.abs(z), 0.0)
    M = a.reshape(T, nb, BLOCK).max(axis=2)
    m, k = np.frexp(M)
    e = np.where(m <= 0.875, k - 9, k - 8)
    return np.where(M == 0, -110, np.clip(e, -110, 120)).astype(np.int64)


def encode(z):
    """(codes uint8 [T, f], scale bytes uint8 [T, nb]): nearest value, ties to the even code"""
    e = scale_exponents(z)
    s = np.repeat(e, BLOCK, axis=1)[:, : z.shape[1]]
    q = np.ldexp(np.where(np.isfinite(z), z, 0.0), -s)
    a = np.abs(q)
    _, k = np.frexp(a)
    step = np.ldexp(1.0, np.maximum(k - 1, -6) - 3)
    r = np.rint(a / step) * step  # numpy's rint: ties to even
    pos = E4M3[:127]
    code = np.searchsorted(pos, r)
    assert np.array_equal(pos[code], r)
    code = code | np.where(np.signbit(z), 128, 0)
    code = np.where(np.isfinite(z), code, 0x7F)
    return code.astype(np.uint8), (e + 127).astype(np.uint8)


def decode(codes, scales):
    e = scales.astype(np.int64) - 127
    return np.ldexp(E4M3[codes], np.repeat(e, BLOCK, axis=1)[:, : codes.shape[1]])


# ------------------------------------------------------------------ router --

def softmax(logits):
    """(p, lse): NaN and -inf logits are absent; rows of only such have p = 0, lse = 0"""
    v = np.where(np.isnan(logits), -np.inf, logits)
    m = v.max(axis=1, keepdims=True)
    none = np.isneginf(m)[:, 0]
    ex = np.exp(v - np.where(np.isneginf(m), 0.0, m))
    s = ex.sum(axis=1, keepdims=True)
    p = np.where(none[:, None], 0.0, ex / np.where(s == 0, 1, s))
    with np.errstate(divide="ignore"):
        return p, np.where(none, 0.0, m[:, 0] + np.log(s[:, 0]))


def counts(ids, E):
    ok = (ids >= 0) & (ids < E)
    c = np.bincount(ids[ok], minlength=E)[:E]
    return np.concatenate([c, [ok.any(axis=1).sum(), c.sum()]]).astype(np.int64)


def balance(logits, ids):
    """(loss [2], cnt, prob)"""
    E = logits.shape[1]
    c = counts(ids, E)
    live = ((ids >= 0) & (ids < E)).any(axis=1)
    p, lse = softmax(logits)
    nt, na = max(c[E], 1), max(c[E + 1], 1)
    prob = p[live].sum(axis=0) / nt
    return np.array([E * (c[:E] / na * prob).sum(), (lse[live] ** 2).sum() / nt]), c, prob


def route_backward(logits, ids, w, dw, cnt, dloss):
    """(dlogits, scale of its rounding errors); w, dw or dloss may be None"""
    T, E = logits.shape
    ok = (ids >= 0) & (ids < E)
    live = ok.any(axis=1)
    p, lse = softmax(logits)
    out, size = np.zeros((T, E)), np.zeros((T, E))
    if dloss is not None:
        nt, na = max(cnt[E], 1), max(cnt[E + 1], 1)
        f = cnt[:E] / na
        gb, gz = dloss[0] * E / nt, dloss[1] * 2 / nt
        fp = (f * p).sum(axis=1, keepdims=True)
        out = live[:, None] * p * (gb * (f - fp) + gz * lse[:, None])
        size = live[:, None] * p * (abs(gb) * (f + fp) + abs(gz) * np.abs(lse[:, None]))
    if dw is not None:
        a = np.where(ok, w * dw, 0.0)
        wk = np.where(ok, w, 0.0)
        pick = a - wk * a.sum(axis=1, keepdims=True)
        psize = np.abs(a) + wk * np.abs(a).sum(axis=1, keepdims=True)
        for k in range(ids.shape[1]):
            r = np.nonzero(ok[:, k])[0]
            np.add.at(out, (r, ids[r, k]), pick[r, k])
            np.add.at(size, (r, ids[r, k]), psize[r, k])
    return out, size
