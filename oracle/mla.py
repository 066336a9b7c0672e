"""Latent attention, stated plainly (test infrastructure; see the package docstring), in f64 NumPy.

A token's cache row is f16(norm(x[:rank]) * w | rot(x[rank:], p)). Head h of a query q has score
(Wk_h^T q[:hd] . c + q[hd:] . r) * scale with a row (c | r) and value Wv_h c; ``w[h]`` holds the hd rows of Wk_h, then
those of Wv_h. :func:`attention` makes keys and values of every head (the definition); :func:`absorbed` multiplies the
weights into the query and into the sum, and is pinned equal to it.

Both give an elementwise bound, every rounding at its worst; it grows with the rank and the context past the answer itself.
:func:`attention_spread` and :func:`absorbed_spread` give the variance that independent roundings leave instead, from the steps of f16 at
the very numbers that are rounded, and :func:`off` says how many times that an answer is away.
"""
from __future__ import annotations

import numpy as np

ROPE = 64
U = 2.0 ** -11          # half a step of f16, relative
TINY = 2.0 ** -25       # half a step of its subnormals
E = 2.0 ** -23          # one f32 addition, however its unit rounds


def rotate(x, cos, sin):
    """Pairs (j, j + 32) of the last axis turned by the angles of the tables' rows."""
    h = x.shape[-1] // 2
    return np.concatenate([x[..., :h] * cos - x[..., h:] * sin, x[..., h:] * cos + x[..., :h] * sin], -1)


def append(kv, norm_w, cos, sin, eps, rank):
    """Cache rows in f64 (not rounded); cos, sin [n, 32] of the rows' positions."""
    x = kv.astype(np.float64)
    c = x[:, :rank] / np.sqrt(np.mean(x[:, :rank] ** 2, -1, keepdims=True) + eps) * norm_w.astype(np.float64)
    return np.concatenate([c, rotate(x[:, rank:], cos.astype(np.float64), sin.astype(np.float64))], -1)


def queries(q, cos, sin, hd):
    x = q.astype(np.float64)
    return np.concatenate([x[..., :hd], rotate(x[..., hd:], cos.astype(np.float64)[:, None], sin.astype(np.float64)[:, None])], -1)


def _weights(x):
    with np.errstate(invalid="ignore"):
        p = np.exp(x - x.max(-1, keepdims=True))
        return p / p.sum(-1, keepdims=True)


def keys_values(rows, w, h, hd):
    c = rows[:, :-ROPE].astype(np.float64)
    k = np.concatenate([c @ w[h, :hd].astype(np.float64).T, rows[:, -ROPE:].astype(np.float64)], -1)
    return k, c @ w[h, hd:].astype(np.float64).T


def attention(q, rows, w, scale, before=None):
    """q [n, heads, hd + 64] over rows [L, rank + 64] -> out [n, heads, hd] and a bound of the error of a kernel that
    makes keys and values as f16, weighs them with f16 weights and rounds the output to f16. Query i sees rows 0 .. before + i
    (all of them where before is None). A weight is kept relative to a reference that makes a row's largest 2^-1 or more, so that half
    a step of f16's subnormals is 2 TINY of the largest at most."""
    q = q.astype(np.float64)
    n, heads, width = q.shape
    hd, L = width - ROPE, len(rows)
    seen = np.ones((n, L), bool) if before is None else np.arange(L)[None] <= before + np.arange(n)[:, None]
    out, bound = np.zeros((n, heads, hd)), np.zeros((n, heads, hd))
    for h in range(heads):
        k, v = keys_values(rows, w, h, hd)
        p = _weights(np.where(seen, q[:, h] @ k.T * scale, -np.inf))
        out[:, h] = p @ v
        size = np.abs(q[:, h]) @ np.abs(k).T * scale
        # products made as f16 (their own sums in f32), then a sum of hd + 64 products, the weight's exponent
        delta = np.max(np.where(seen, size * (U + (len(rows[0]) + width) * E) + 8 * E, 0), -1, keepdims=True)
        av = np.abs(v) * (1 + U)
        bound[:, h] = ((2 * delta + 2 * U + (len(rows[0]) + L) * E) * (p @ av) + U * np.abs(out[:, h]) + TINY
                       + 2 * TINY * p.max(-1, keepdims=True) * (seen @ av))
    return out, bound


def absorbed(q, rows, w, scale):
    """The single-token form: q [heads, hd + 64] -> out [heads, hd] and a bound of the error of a kernel that rounds the
    absorbed query, the weights, the sum over the rows and the output to f16. (The kernels keep the sum, and up to 32 heads the query, as two
    f16 numbers: the bound allows for one.)"""
    q = q.astype(np.float64)
    heads, hd, L = q.shape[0], q.shape[1] - ROPE, len(rows)
    rows = rows.astype(np.float64)
    c, w = rows[:, :-ROPE], w.astype(np.float64)
    R = c.shape[1]
    qc = np.einsum("hd,hdr->hr", q[:, :hd], w[:, :hd])
    dq = U * np.abs(qc) + TINY + hd * E * np.einsum("hd,hdr->hr", np.abs(q[:, :hd]), np.abs(w[:, :hd]))
    full = np.concatenate([qc, q[:, hd:]], -1)
    p = _weights(full @ rows.T * scale)
    o = p @ c
    out = np.einsum("hr,hdr->hd", o, w[:, hd:])
    delta = scale * np.max(dq @ np.abs(c).T + (R + ROPE) * E * (np.abs(full) @ np.abs(rows).T), -1, keepdims=True) + 8 * E
    do = ((2 * delta + U + 2 * L * E) * (p @ np.abs(c)) + U * np.abs(o) + TINY
          + TINY * p.max(-1, keepdims=True) * np.abs(c).sum(0))
    bound = np.einsum("hr,hdr->hd", do + R * E * np.abs(o), np.abs(w[:, hd:])) + U * np.abs(out) + TINY
    return out, bound


# ---------------------------------------------------------------- what independent roundings add up to
# A rounding is off by something between half a step down and half a step up: step^2 / 12 on average. A weight of the softmax is rounded relative to
# a reference that is not known here; over mantissas of all sizes alike its step^2 is 2^-20 of its square times 3 / (8 ln 2).
WEIGHT = 3 / (8 * np.log(2)) * 2.0 ** -20 / 12


def rounding(x):
    """The variance of rounding x to f16."""
    _, e = np.frexp(x)
    return 2.0 ** (2 * np.maximum(e - 11, -24)) / 12


def attention_spread(q, rows, w, scale, before):
    """:func:`attention`'s answer and the variance of its error: keys and values as f16, f16 weights, the output as f16."""
    q = q.astype(np.float64)
    n, heads, width = q.shape
    hd, L = width - ROPE, len(rows)
    seen = np.arange(L)[None] <= before + np.arange(n)[:, None]
    out, var = np.zeros((n, heads, hd)), np.zeros((n, heads, hd))
    for h in range(heads):
        k, v = keys_values(rows, w, h, hd)
        p = _weights(np.where(seen, q[:, h] @ k.T * scale, -np.inf))
        o = out[:, h] = p @ v
        score = scale ** 2 * q[:, h, :hd] ** 2 @ rounding(k[:, :hd]).T           # (the rotated part is f16 already)
        s2 = p * p * score
        var[:, h] = (s2 @ v ** 2 - 2 * o * (s2 @ v) + s2.sum(-1, keepdims=True) * o ** 2 + (p * p) @ (rounding(v) + WEIGHT * v ** 2)
                     + rounding(o))
    return out, var


def absorbed_spread(q, rows, w, scale, pair):
    """:func:`absorbed`'s answer and the variance of its error: f16 weights, the output as f16, and (not `pair`) the absorbed query as one f16
    number; as two, and the sum over the rows as two, they are exact beside the rest."""
    q = q.astype(np.float64)
    heads, hd = q.shape[0], q.shape[1] - ROPE
    rows, w = rows.astype(np.float64), w.astype(np.float64)
    c = rows[:, :-ROPE]
    qc = np.einsum("hd,hdr->hr", q[:, :hd], w[:, :hd])
    p = _weights(np.concatenate([qc, q[:, hd:]], -1) @ rows.T * scale)
    o = p @ c
    out = np.einsum("hr,hdr->hd", o, w[:, hd:])
    var = rounding(out)
    for h in range(heads):
        v = c @ w[h, hd:].T
        var[h] += WEIGHT * (p[h] ** 2 @ v ** 2)
        if not pair:        # one error for all rows: it moves the answer by the values' covariance with the latents
            m = scale * ((p[h][:, None] * (v - out[h])).T @ c)
            var[h] += m ** 2 @ rounding(qc[h])
    return out, var


def off(got, want, var):
    """How many times the spread an answer is away: the root mean square of its error over the last two axes (heads and values), and the
    largest head's."""
    e = (got.astype(np.float64) - want) ** 2
    e, var = e.reshape(-1, *e.shape[-2:]), var.reshape(-1, *e.shape[-2:])
    return float(np.sqrt(e.mean() / var.mean())), float(np.sqrt(np.max(e.mean(-1) / var.mean(-1))))
