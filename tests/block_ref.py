"""Plain 64-bit forms of the operators around the routed layer's block (numpy):
routing by scores, norms with gate and residual, 4-bit weights; and how far 32-bit
arithmetic with one final rounding may be from them."""
from __future__ import annotations

import numpy as np

from dense_ref import HALF, TINY, U32, f64

NINF = -np.inf
__all__ = ["HALF", "TINY", "U32", "f64"]


# ------------------------------------------------------- routing by scores --

def log_scores(logits, kind):
    """log of each expert's score; -inf where the expert is absent (NaN, -inf)"""
    v = np.where(logits > NINF, logits, NINF).astype(np.float64)
    if kind == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(v > NINF, -np.logaddexp(0.0, -v), NINF)
    top = v.max(axis=1, keepdims=True)
    if np.isposinf(top).any():  # shared evenly among the infinite ones
        v = np.where(np.isposinf(top), np.where(np.isposinf(v), 0.0, NINF), v)
        top = v.max(axis=1, keepdims=True)
    d = v - np.where(np.isneginf(top), 0.0, top)
    total = np.exp(d).sum(axis=1, keepdims=True)  # 0: nobody is there
    return d - np.log(np.where(total > 0, total, 1.0))


def route(logits, K, bias=None, score="softmax", groups=1, keep=None, group_top=1, renorm=True,
          scale=1.0):
    """(ids [T, K], w [T, K], the smallest gap between different choices that could have
    been made, relative to what is compared). Without a bias experts go by their logits,
    of which the score is a rising function."""
    T, E = logits.shape
    n, keep = E // groups, groups if keep is None else keep
    ls = log_scores(logits, score)
    c = np.exp(ls) + (0.0 if bias is None else np.where(np.isnan(bias), NINF, bias))
    there = (logits > NINF) & (True if bias is None else (bias > NINF)[None, :])
    c = np.where(there, c, NINF)
    ids, w = np.full((T, K), -1), np.zeros((T, K))
    gap = np.inf

    big = 0.0 if bias is None else np.abs(bias[np.isfinite(bias)]).max()

    def apart(v):
        nonlocal gap
        v = v[np.isfinite(v)]
        d, size = -np.diff(v), np.maximum(np.abs(v[:-1]), np.abs(v[1:]))
        if (d > 0).any():
            gap = min(gap, (d / np.maximum(size, big))[d > 0].min())

    for t in range(T):
        worth = np.full(groups, NINF)
        for g in range(groups):
            best = np.sort(c[t, g * n:(g + 1) * n])[::-1][:group_top]
            if there[t, g * n:(g + 1) * n].any():
                worth[g] = best[best > NINF].sum()
        order = np.argsort(-worth, kind="stable")
        if groups > 1:
            apart(worth[order])
        mine = np.full(E, NINF)
        key = c if bias is not None else np.where(there, logits, NINF)
        for g in order[:keep]:
            mine[g * n:(g + 1) * n] = key[t, g * n:(g + 1) * n]
        pick = np.argsort(-mine, kind="stable")[:K + 1]
        if bias is not None:
            apart(mine[pick])
        pick = [e for e in pick[:K] if mine[e] > NINF]
        ids[t, :len(pick)] = pick
        if not pick:
            continue
        s = ls[t, pick]
        if renorm:
            s = s - s.max()
            s = s - np.log(np.exp(s).sum())
        w[t, :len(pick)] = scale * np.exp(s)
    return ids, w, gap


def route_tolerance(logits, ids, w, score):
    """fp32: the exponentials' arguments (off by half a step of themselves, which are at
    most the spread of the logits that carry weight), their sum over the experts, and a
    division or two"""
    v = np.where(np.isfinite(logits), logits, 0.0).astype(np.float64)
    pick = np.take_along_axis(v, np.clip(ids, 0, None), axis=1)
    far = np.abs(pick) if score == "sigmoid" else np.abs(v.max(axis=1, keepdims=True) - pick)
    spread = np.maximum(far, np.abs(pick.max(axis=1, keepdims=True) - pick))
    return np.abs(w) * (40 + 3 * spread) * U32 + 2.0 ** -120


def route_backward(logits, ids, dw, score="softmax", renorm=True, scale=1.0, add=None):
    """(dlogits, sum of the magnitudes of its terms)"""
    T, E = logits.shape
    ok = (ids >= 0) & (ids < E)
    at = np.where(ok, ids, 0)
    ok &= np.take_along_axis(logits, at, axis=1) > NINF
    ls = log_scores(logits, score)
    ll = np.where(ok, np.take_along_axis(ls, at, axis=1), NINF)
    u = np.where(ok, scale * np.where(ok, dw, 0.0), 0.0)
    if renorm:
        top = ll.max(axis=1, keepdims=True)
        part = np.exp(ll - np.where(np.isneginf(top), 0.0, top))
        part /= np.maximum(part.sum(axis=1, keepdims=True), 1e-300)
        g = part * (u - (part * u).sum(axis=1, keepdims=True))
        size = part * (np.abs(u) + (part * np.abs(u)).sum(axis=1, keepdims=True))
    else:
        s = np.exp(ll)
        g, size = s * u, s * np.abs(u)
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    slope = 1.0
    if score == "sigmoid":
        with np.errstate(over="ignore", invalid="ignore"):
            slope = np.take_along_axis(np.exp(np.where(logits > NINF, -np.logaddexp(0.0, logits.astype(np.float64)), 0.0)), at, axis=1)
    for k in range(ids.shape[1]):
        r = np.nonzero(ok[:, k])[0]
        f = slope if np.isscalar(slope) else slope[r, k]
        np.add.at(out, (r, ids[r, k]), (g[r, k] * f))
        np.add.at(mag, (r, ids[r, k]), (size[r, k] * f))
    if score == "softmax" and not renorm:
        p = np.exp(ls)
        out -= p * g.sum(axis=1, keepdims=True)
        mag += p * size.sum(axis=1, keepdims=True)
    if add is not None:
        out, mag = out + add, mag + np.abs(add)
    return out, mag


def backward_tolerance(logits, mag, out, dtype):
    v = np.where(np.isfinite(logits), logits, 0.0).astype(np.float64)
    spread = np.minimum(np.abs(v).max(axis=1, keepdims=True) * 2, 200.0)
    return mag * (64 + 8 * spread) * U32 + np.abs(out) * HALF[dtype] + TINY[dtype] + 2.0 ** -120


# ------------------------------------------------------------------- norms --

def spread_gate(gate, kind, T, d):
    if gate is None:
        return np.ones((1, 1))
    return gate.reshape({"token": (T, 1), "channel": (1, d), "full": (T, d)}[kind])


def inverse_rms(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def norm(r, y=None, w_post=None, gate=None, kind="none", w_pre=None, alpha=1.0, eps=1e-6):
    """dict of z, h, stats (and n, the normalised y)"""
    T, d = r.shape
    iy = iz = np.zeros((T, 1))
    z, n = r, None
    if y is not None:
        n = y
        if w_post is not None:
            iy = inverse_rms(y, eps)
            n = y * iy * w_post
        z = r + alpha * spread_gate(gate, kind, T, d) * n
    got = {"z": z, "n": n}
    if w_pre is not None:
        iz = inverse_rms(z, eps)
        got["h"] = z * iz * w_pre
    got["stats"] = np.concatenate([iy, iz], axis=1)
    return got


def norm_tolerance(want, r, gate, kind, w_pre, alpha):
    """fp32 errors of z, h, stats before the outputs' own rounding. A sum of d squares
    is at most d / 64 additions long in one lane, then joined."""
    T, d = r.shape
    rel = (d / 64 + 32) * U32
    moved = np.zeros_like(r)
    if want["n"] is not None:
        moved = np.abs(alpha * spread_gate(gate, kind, T, d) * want["n"]) * (rel + 8 * U32)
        moved = moved + np.abs(want["z"]) * U32 + 2.0 ** -126
    tol = {"z": moved, "stats": np.abs(want["stats"]) * rel}
    z = np.abs(want["z"])
    if w_pre is not None:
        with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
            off = np.nan_to_num((z * moved).sum(axis=1, keepdims=True)
                                / (z * z).sum(axis=1, keepdims=True), nan=0.0)
        iz = want["stats"][:, 1:]
        tol["h"] = np.abs(want["h"]) * (rel + off + 4 * U32) + np.abs(w_pre) * iz * moved
        tol["stats"] = tol["stats"] + want["stats"] * np.concatenate([0 * off, off], axis=1)
    return tol


def norm_backward(z, stats, dz=None, dh=None, y=None, w_post=None, gate=None, kind="none",
                  w_pre=None, alpha=1.0):
    """(dict of gradients, dict of the sums of the magnitudes of their terms)"""
    T, d = z.shape
    iy, iz = stats[:, :1], stats[:, 1:]
    got, mag = {}, {}
    dr = np.zeros((T, d)) if dz is None else dz.copy()
    size = np.abs(dr)
    if w_pre is not None:
        zn = z * iz
        g = dh * w_pre
        dr = dr + iz * (g - zn * (g * zn).mean(axis=1, keepdims=True))
        size = size + iz * (np.abs(g) + np.abs(zn) * np.abs(g * zn).mean(axis=1, keepdims=True))
        got["dw_pre"], mag["dw_pre"] = (dh * zn).sum(axis=0), np.abs(dh * zn).sum(axis=0)
    got["dr"], mag["dr"] = dr, size
    if y is None:
        return got, mag
    gv = spread_gate(gate, kind, T, d)
    yn = y * iy
    n = yn * w_post if w_post is not None else y
    if gate is not None:
        axis = {"token": 1, "channel": 0, "full": None}[kind]
        a, b = alpha * dr * n, np.abs(alpha * size * n)
        got["dgate"] = a if axis is None else a.sum(axis=axis)
        mag["dgate"] = b if axis is None else b.sum(axis=axis)
    q, qs = alpha * gv * dr, np.abs(alpha * gv) * size
    if w_post is None:
        got["dy"], mag["dy"] = q, qs
        return got, mag
    got["dw_post"], mag["dw_post"] = (q * yn).sum(axis=0), (qs * np.abs(yn)).sum(axis=0)
    g, gs = q * w_post, qs * np.abs(w_post)
    got["dy"] = iy * (g - yn * (g * yn).mean(axis=1, keepdims=True))
    mag["dy"] = iy * (gs + np.abs(yn) * (gs * np.abs(yn)).mean(axis=1, keepdims=True))
    return got, mag


def norm_backward_tolerance(mag, T, d, name, dtype, want):
    """every term carries at most two row sums (d / 64 additions in a lane each) and some
    roundings; the column sums at most T additions more, however they are cut"""
    rel = 2 * (d / 64 + 48) * U32
    if name in ("dw_pre", "dw_post") or (name == "dgate" and mag.ndim == 1):
        rel += max(T, d / 64) * U32
    return mag * rel + np.abs(want) * HALF[dtype] + TINY[dtype] + 2.0 ** -120


# ----------------------------------------------------------- 4-bit weights --

VALUES = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def mx4_encode(w):
    """(codes uint8 [E, Kd, N], scale bytes uint8 [E, ceil(Kd / 32), N]) of float64 w"""
    E, Kd, N = w.shape
    nb = -(-Kd // 32)
    a = np.zeros((E, nb * 32, N))
    a[:, :Kd] = w
    b = a.reshape(E, nb, 32, N)
    odd = ~np.isfinite(b).all(axis=2)
    M = np.where(np.isfinite(b), np.abs(b), 0.0).max(axis=2)
    m, k = np.frexp(M)
    e = np.where(M == 0, -110, np.clip(np.where(m <= 0.75, k - 3, k - 2), -110, 120))
    with np.errstate(invalid="ignore"):
        t = np.minimum(np.ldexp(np.abs(np.nan_to_num(b, posinf=0, neginf=0)), -e[:, :, None]), 6.0)
    step = np.where(t < 2, 0.5, np.where(t < 4, 1.0, 2.0))
    v = np.rint(t / step) * step  # ties to even multiples, which are the even codes
    codes = np.searchsorted(VALUES, v) | np.where(np.signbit(b), 8, 0)
    codes = codes.reshape(E, nb * 32, N)[:, :Kd]
    return codes.astype(np.uint8), np.where(odd, 255, e + 127).astype(np.uint8)


def mx4_values(codes, scales):
    """what codes and scale bytes stand for"""
    v = np.where(codes & 8, -1.0, 1.0) * VALUES[codes & 7]
    s = np.repeat(scales.astype(np.int64), 32, axis=1)[:, :codes.shape[1]]
    return np.where(s == 255, np.nan, np.ldexp(v, s - 127))


def mx4_places(Kd, N, down):
    """byte of each weight's code and scale in an expert's packed bytes, and their number"""
    m = 2 if down else 1
    nst, groups = -(-Kd // 32), -(-N // (256 * m))
    k, n = np.arange(Kd)[:, None], np.arange(N)[None, :]
    group, rest = n // (256 * m), n % (256 * m)
    slice_, stream, col = rest // (64 * m), rest % (64 * m) // 64, n % 64
    tile = ((group * nst + k // 32) * 4 + slice_) * m + stream
    lane = 16 * (k % 32 // 8) + col // 4
    code = tile * 1088 + lane * 16 + (col % 4) * 4 + (k % 8) // 2
    return code, tile * 1088 + 1024 + col, groups * nst * 4 * m * 1088


def mx4_unpack(packed, E, Kd, N, down):
    """(codes, scale bytes) of packed bytes [E * bytes]"""
    code, scale, size = mx4_places(Kd, N, down)
    p = packed.reshape(E, size)
    half = (np.arange(Kd) % 2)[:, None] * 4
    return (p[:, code] >> half) & 15, p[:, scale][:, ::32]
