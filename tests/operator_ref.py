"""Plain 64-bit forms of the general gates, their gradient, the combine's gradient and the 4-bit
experts, written from the formulas in include/lc_moe.h with numpy. They share no code with the
library."""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24   # half a step of fp32, relative
U16 = 2.0 ** -8    # half a step of bf16, relative


def scores(z, score):
    z = np.asarray(z, np.float64)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-z))
    m = z.max(axis=1, keepdims=True)
    e = np.exp(z - np.where(np.isinf(m), 0.0, m))
    S = e.sum(axis=1, keepdims=True)
    return e / np.where(S > 0, S, 1.0)


def picks(s, bias, K, groups=1, top_groups=1, group_rank=1):
    """K picks per token by repeated maximum: groups first, then keys; equal values to the lower index."""
    T, E = s.shape
    key = s if bias is None else s + np.asarray(bias, np.float64)
    size = E // groups
    out = np.empty((T, K), np.int32)
    for t in range(T):
        stay = range(groups)
        if top_groups < groups:
            best = [sum(sorted(key[t, g * size:(g + 1) * size], reverse=True)[:group_rank]) for g in range(groups)]
            stay = sorted(range(groups), key=lambda g: (-best[g], g))[:top_groups]
        cand = [i for g in sorted(stay) for i in range(g * size, (g + 1) * size)]
        cand = np.array(cand)
        order = np.lexsort((cand, -key[t, cand]))
        out[t] = cand[order[:K]]
    return out


def gates(z, s, idx, score, renorm, scale):
    """Gates of the picks. Renormalised gates whose scores all underflow are taken from the logits:
    s is e^z times a common factor there."""
    p = np.take_along_axis(s, idx.astype(np.int64), 1)
    if renorm:
        zc = np.take_along_axis(np.asarray(z, np.float64), idx.astype(np.int64), 1)
        tot = p.sum(1, keepdims=True)
        low = zc.max(1, keepdims=True)
        e = np.exp(zc - np.where(np.isinf(low), 0.0, low))
        eq = e.sum(1, keepdims=True)
        soft = np.where(eq > 0, e / np.where(eq > 0, eq, 1.0), 0.0)
        p = np.where(tot > 1e-280, p / np.where(tot > 0, tot, 1.0), soft)
    return scale * p


def gate_backward(z, idx, dgate, score, renorm, scale):
    """(dz, bound): the gradient, and a bound on the sizes its fp32 evaluation adds up."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    s = scores(z, score)
    at = np.arange(T)[:, None]
    ok = (idx >= 0) & (idx < E)
    i = np.where(ok, idx, 0)
    ps = np.where(ok, s[at, i], 0.0)
    dg = np.where(ok, scale * np.asarray(dgate, np.float64), 0.0)
    dz, bound = np.zeros((T, E)), np.zeros((T, E))
    if renorm:
        tot = ps.sum(1, keepdims=True)
        p = np.where(tot > 0, ps / np.where(tot > 0, tot, 1.0), 0.0)
        f = 1.0 - ps if score == "sigmoid" else np.ones_like(ps)
        mean, amean = (p * dg).sum(1, keepdims=True), (p * np.abs(dg)).sum(1, keepdims=True)
        np.add.at(dz, (at, i), p * f * (dg - mean))
        np.add.at(bound, (at, i), p * f * (np.abs(dg) + amean))
    elif score == "sigmoid":
        np.add.at(dz, (at, i), dg * ps * (1 - ps))
        np.add.at(bound, (at, i), np.abs(dg) * ps * (1 - ps))
    else:
        D, aD = (ps * dg).sum(1, keepdims=True), (ps * np.abs(dg)).sum(1, keepdims=True)
        np.add.at(dz, (at, i), ps * dg)
        np.add.at(bound, (at, i), ps * np.abs(dg))
        dz -= s * D
        bound += s * aD
    return dz, bound


def w4_unpack(codes, scale, rows, cols, group):
    """[rows, cols] float64 from one matrix's codes (bytes) and scales (float64 [rows/16, cols/group, 16])."""
    words = np.ascontiguousarray(codes).reshape(-1).view("<u4")
    r, c = np.meshgrid(np.arange(rows), np.arange(cols), indexing="ij")
    byte = ((r // 16) * (cols // 64) + c // 64) * 512 + 16 * (4 * (r % 8) + (c % 32) // 8) \
        + 4 * (2 * ((c % 64) // 32) + (r % 16) // 8)
    p = (c % 8) // 2 + 4 * (c % 2)
    q = (words[byte // 4] >> (4 * p).astype(np.uint32)) & 15
    return (q.astype(np.float64) - 8) * scale[r // 16, c // group, 2 * (r % 8) + (r % 16) // 8]


def w4_quantize(w, group):
    """(q in -7..7, scale) of float64 [rows, cols] by the header's rule; scales rounded to bf16."""
    rows, cols = w.shape
    a = np.abs(w).reshape(rows, cols // group, group).max(2)
    s = (a / 7.0).astype(np.float32)
    b = s.view(np.uint32).astype(np.uint64)
    b = ((b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16).astype(np.uint32)
    s = b.view(np.float32).astype(np.float64)
    s = np.where(s == 0, 1.0, s)
    q = np.rint(w / np.repeat(s, group, axis=1))
    return np.clip(q, -7, 7), s
