"""The operators around int8 experts in 64 bits (numpy), for the tests: scored
routing, int8 products, the int8-activation FFN and the block norms, each from its
formula, and the bounds of what fp32 arithmetic may add to them."""
from __future__ import annotations

import numpy as np

LOWEST = np.finfo(np.float32).min
U32 = 2.0 ** -24  # half a step of fp32, relative
UBF = 2.0 ** -8   # of bf16


def route(logits, k, bias=None, score="softmax", n_group=1, topk_group=1, group_top=1, renorm=True, scale=1.0):
    """ids [T, k], w [T, k] (fp64)."""
    T, E = logits.shape
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        l = logits[t].astype(np.float64)
        live = logits[t] > LOWEST
        s = np.zeros(E)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s[live] = 1.0 / (1.0 + np.exp(-l[live]))
        elif live.any():
            m = l[live].max()
            with np.errstate(invalid="ignore"):  # inf - inf, where l == m
                s[live] = np.exp(np.where(l[live] == m, 0.0, l[live] - m))
            s /= s.sum()
        c = s if bias is None else s + bias.astype(np.float64)
        if bias is not None:
            live = live & (bias > LOWEST)
        allowed = live.copy()
        if n_group > 1:
            size = E // n_group
            rank = []
            for g in range(n_group):
                best = sorted(c[g * size:(g + 1) * size][live[g * size:(g + 1) * size]], reverse=True)[:group_top]
                if best:
                    rank.append((-sum(best), g))
            kept = [g for _, g in sorted(rank)[:topk_group]]
            allowed &= np.isin(np.arange(E) // size, kept)
        cand = [e for e in range(E) if allowed[e]]
        top = sorted(cand, key=lambda e: (-c[e], e))[:k]
        ids[t, :len(top)] = top
        w[t, :len(top)] = s[top]
        if renorm:
            z = w[t].sum()
            w[t] = w[t] / z if z > 0 else 0.0
    return ids, w * scale


def codes(v):
    """int8 codes and scale of each row (ties to even)."""
    s = np.abs(v).max(-1, initial=0.0) / 127.0
    q = np.rint(np.divide(v, s[..., None], out=np.zeros_like(v), where=s[..., None] > 0))
    return np.clip(q, -127, 127), s


def linear(xq, sx, wq, sw):
    acc = xq.astype(np.int64) @ wq.astype(np.int64).T
    return acc * sx.astype(np.float64)[:, None] * sw.astype(np.float64)


def gelu_tanh(a):
    return 0.5 * a * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (a + 0.044715 * a ** 3)))


def ffn_row(xq, sx, q13, s13, q2, s2):
    """One route: (row [H], tolerance [H]).  xq [H] codes, the expert's codes and scales.

    The fp32 error of h_i: its sums are exact integers (one rounding each to fp32 and
    two per scale, for g and for u: 6 roundings of half a step), gelu's argument and
    tanhf (2 steps by CUDA's table) and the products after it: 16 half steps of |g u|
    cover them, gelu being at most |g| (its cancellation at negative g is an absolute
    error of the size of a step of |g|).  A code of h is then h / sh with that error
    over sh, plus 127 times sh's own relative error (16 + 1 half steps); where the exact
    quotient is nearer to a half than that, either code is right, and the row may be
    off by one code step there.  The sum over the codes is exact; 4 half steps cover
    its rounding and the scales."""
    I = q2.shape[1]
    acc = q13.astype(np.int64) @ xq.astype(np.int64)
    g = acc * float(sx) * s13.astype(np.float64)
    a, u = g[:I], g[I:]
    h = gelu_tanh(a) * u
    q, sh = codes(h[None])
    q, sh = q[0], sh[0]
    row = (q2.astype(np.float64) @ q) * sh * s2.astype(np.float64)
    tol = 4 * U32 * np.abs(row)
    if sh > 0:
        slack = 16 * U32 * np.abs(a * u) / sh + 127 * 17 * U32
        r = np.abs(h / sh)
        near = np.abs(r - np.floor(r) - 0.5) <= slack
        tol = tol + 17 * U32 * np.abs(row) + (np.abs(q2.astype(np.float64)) @ near) * sh * np.abs(s2.astype(np.float64))
    return row, tol


def combine(rows, route_pos, w):
    """z [T, H] and sum |w r| (for the bound of its fp32 sum)."""
    T, k = w.shape
    z = np.zeros((T, rows.shape[1]))
    mag = np.zeros_like(z)
    for t in range(T):
        for j in range(k):
            p = route_pos[t * k + j]
            if 0 <= p < rows.shape[0]:
                z[t] += float(w[t, j]) * rows[p].astype(np.float64)
                mag[t] += np.abs(float(w[t, j]) * rows[p].astype(np.float64))
    return z, mag


def norm_error(H):
    """Relative error of r = rsqrt(mean + eps) in fp32, in units of U32: a sum of
    squares over at most 16 values of a thread, 5 lane steps and 32 warps is off by at
    most 16 + 5 + 32 half steps, one for the mean, one for eps, halved by the root, and
    one step of the root itself."""
    return (min(H, 16) + 5 + 32 + 2) / 2 + 2


def after_block(z, mag, residual, post_w, gate_h, gate_t, eps, offset, rs, bs):
    """y [T, H] and its tolerance before the rounding to bf16.  z carries up to 33
    half steps of `mag` from its own fp32 sum (k <= 32 products); the error of a sum of squares follows it."""
    H = z.shape[1]
    rz = 33 * U32 * mag
    n = 6.0
    if post_w is not None:
        r = 1.0 / np.sqrt((z * z).mean(1, keepdims=True) + eps)
        gain = r * np.abs(offset + post_w.astype(np.float64))
        dz = np.sqrt((rz * rz).mean(1, keepdims=True)) * r  # relative error that z's own error leaves in r
        zn = z * r * (offset + post_w.astype(np.float64))
        n += norm_error(H)
        rz = rz * gain + np.abs(zn) * dz
    else:
        zn = z
    f = bs * (1.0 if gate_t is None else gate_t.astype(np.float64)[:, None]) * \
        (1.0 if gate_h is None else gate_h.astype(np.float64))
    y = rs * residual + f * zn
    tol = np.abs(f) * rz + U32 * (n * np.abs(f * zn) + 3 * np.abs(rs * residual) + np.abs(y))
    return y, tol


def norm(x, weight, eps, offset):
    """n [T, H] and its relative fp32 error (in absolute terms)."""
    n = x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * (offset + weight.astype(np.float64))
    return n, (norm_error(x.shape[1]) + 3) * U32
