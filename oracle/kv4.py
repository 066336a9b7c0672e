"""The 4-bit KV pool, stated plainly (test infrastructure; see the package docstring): the row
quantiser, the record layout and the attention over records, in f64 NumPy.

A row is cut into blocks of 32. A block keeps m = f16(min x), d = f16((max x - min x) / 15) and
codes c = clamp(rint((x - m) / d), 0, 15) (0 where d = 0), each rounded once from its exact value to
nearest even; a zero minimum is stored as +0. Decoded: d c + m.
"""
from __future__ import annotations

import numpy as np

QK = 32
TOKENS = 16


def record_bytes(hd: int) -> int:
    return 20 * hd


def quantize(rows):
    """Rows [n, dim] (f32 or f16 values) -> codes u8 [n, dim], scales f16 and minima f16 [n, dim / 32]."""
    x = np.asarray(rows).astype(np.float64)
    if not np.all(np.isfinite(x)):
        raise ValueError("kv4: rows must be finite")
    n, dim = x.shape
    x = x.reshape(n, dim // QK, QK)
    low, high = x.min(-1), x.max(-1)
    with np.errstate(over="ignore"):
        m = (low.astype(np.float16) + np.float16(0)).astype(np.float16)
        d = ((high - low) / 15.0).astype(np.float16)
    if not (np.all(np.isfinite(m)) and np.all(np.isfinite(d))):
        raise ValueError("kv4: a block scale or minimum overflows f16")
    md, dd = m.astype(np.float64)[..., None], d.astype(np.float64)[..., None]
    c = np.where(dd > 0, np.clip(np.rint((x - md) / np.where(dd > 0, dd, 1.0)), 0, 15), 0)
    return c.astype(np.uint8).reshape(n, dim), d, m


def dequantize(codes, d, m):
    n, dim = codes.shape
    c = codes.astype(np.float64).reshape(n, dim // QK, QK)
    return (c * d.astype(np.float64)[..., None] + m.astype(np.float64)[..., None]).reshape(n, dim)


def place(records, blocks, slots, head, kq, vq, hd):
    """Write quantised rows (codes, d, m) of K and V into ``records`` u8 [num_blocks, n_kv, 20 hd]."""
    nb = hd // QK
    for r, (blk, s) in enumerate(zip(blocks, slots)):
        rec = records[blk, head]
        word = rec.view(np.float16)
        for b in range(nb):
            word[8 * hd + s * nb + b] = kq[1][r, b]
            word[8 * hd + hd // 2 + s * nb + b] = kq[2][r, b]
            at = 9 * hd + 4 * nb * (s % 4) + 2 * nb * (s // 8) + 2 * b + (s // 4) % 2
            word[at] = vq[1][r, b]
            word[at + hd // 2] = vq[2][r, b]
            for j in range(4):
                for i in range(4):
                    lo, hi = kq[0][r, 32 * b + 4 * j + i], kq[0][r, 32 * b + 4 * j + i + 16]
                    rec[s * (hd // 2) + 4 * (nb * j + b) + i] = lo | (hi << 4)
            for w in range(8):
                u = w ^ (4 * ((s >> 1) & 1)) if hd == 128 else w
                e = [int(vq[0][r, 32 * b + w + 8 * q]) for q in range(4)]
                at = 8 * hd + s * (hd // 2) + 2 * (nb * u + b)
                rec[at] = e[0] | (e[1] << 4)
                rec[at + 1] = e[2] | (e[3] << 4)


def rows_of(records, blocks, slots, hd):
    """Decode the K and V rows of (block, slot) pairs: f64 [n, n_kv, hd] each."""
    nb = hd // QK
    e = np.arange(hd)
    b, i = e // 32, e % 32
    n_kv = records.shape[1]
    blk = np.asarray(blocks, np.int64)[:, None, None]
    s = np.asarray(slots, np.int64)[:, None, None]
    g = np.arange(n_kv)[None, :, None]
    word = records.view(np.float16).astype(np.float64)
    kc = records[blk, g, s * (hd // 2) + 4 * (nb * (i % 16 // 4) + b) + i % 4] >> (4 * (i // 16)).astype(np.uint8) & 15
    u = (i % 8) ^ (4 * (s >> 1 & 1)) if hd == 128 else i % 8 + 0 * s
    vc = records[blk, g, 8 * hd + s * (hd // 2) + 2 * (nb * u + b) + i // 16] >> (4 * (i // 8 % 2)).astype(np.uint8) & 15
    vw = 9 * hd + 4 * nb * (s % 4) + 2 * nb * (s // 8) + 2 * b + (s // 4) % 2
    kw = 8 * hd + s * nb + b
    return (kc * word[blk, g, kw] + word[blk, g, kw + hd // 2], vc * word[blk, g, vw] + word[blk, g, vw + hd // 2])


def paged_attention(q, records, block_tables, lens, scale):
    """softmax(scale q K^T) V per sequence over its first ``lens[b]`` tokens; rows of length 0 are NaN."""
    q = np.asarray(q, np.float64)
    B, H, hd = q.shape
    n_kv = records.shape[1]
    out = np.full((B, H, hd), np.nan)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        t = np.arange(n)
        k, v = rows_of(records, np.asarray(block_tables)[b][t // TOKENS], t % TOKENS, hd)
        for h in range(H):
            g = h // (H // n_kv)
            x = k[:, g] @ q[b, h] * scale
            p = np.exp(x - x.max())
            out[b, h] = p @ v[:, g] / p.sum()
    return out
