"""Pins of the spread that independent roundings leave in latent attention: an evaluation that rounds where the kernels do lies at it, and
answers that are wrong in one place lie far off, at lengths where the elementwise bounds let them pass."""
import numpy as np
import pytest

from oracle import mla

WHOLE, HEAD = 1.25, 2.5     # what the GPU tests allow of a whole answer and of its worst head


def case(n, heads, hd, rank, L, seed=0):
    g = np.random.default_rng(seed)
    return ((1.5 * g.standard_normal((n, heads, hd + 64))).astype(np.float16), g.standard_normal((L, rank + 64)).astype(np.float16),
            (g.standard_normal((heads, 2 * hd, rank)) / np.sqrt(rank)).astype(np.float16), 1 / np.sqrt(hd + 64))


def half(x):
    return x.astype(np.float16).astype(np.float64)


def absorbed(q, rows, w, scale, query_pair=True, sum_pair=True, keep=None, rotated=True, flat=False):
    """The single-token form with its roundings; `keep`: the rows it looks at."""
    q, rows, w = q.astype(np.float64), rows.astype(np.float64), w.astype(np.float64)
    rows = rows if keep is None else rows[keep]
    hd, c = q.shape[1] - mla.ROPE, rows[:, :-mla.ROPE]
    exact = np.einsum("hd,hdr->hr", q[:, :hd], w[:, :hd])
    qc = half(exact) + (half(exact - half(exact)) if query_pair else 0)
    x = (qc @ c.T + rotated * (q[:, hd:] @ rows[:, -mla.ROPE:].T)) * scale / np.log(2) * (not flat)
    p = 2.0 ** (x - x.max(-1, keepdims=True) + 6.3)
    o = half(p) @ c / p.sum(-1, keepdims=True)
    o = half(o) + (half(o - half(o)) if sum_pair else 0)
    return np.einsum("hr,hdr->hd", o, w[:, hd:]).astype(np.float16)


def expanded(q, rows, w, scale, before):
    q = q.astype(np.float64)
    n, heads, width = q.shape
    out, seen = np.zeros((n, heads, width - mla.ROPE)), np.arange(len(rows))[None] <= before + np.arange(n)[:, None]
    for h in range(heads):
        k, v = mla.keys_values(rows, w, h, width - mla.ROPE)
        x = np.where(seen, q[:, h] @ half(k).T * scale / np.log(2), -np.inf)
        p = 2.0 ** (x - x.max(-1, keepdims=True) + 6.3)
        out[:, h] = half(p) @ half(v) / p.sum(-1, keepdims=True)
    return out.astype(np.float16)


def test_answers_are_the_definition():
    q, rows, w, scale = case(3, 4, 64, 256, 40)
    a, b = mla.attention_spread(q, rows, w, scale, 37)[0], mla.attention(q, rows, w, scale, before=37)[0]
    np.testing.assert_allclose(a, b, rtol=1e-12, atol=1e-13)
    for pair in (False, True):
        np.testing.assert_allclose(mla.absorbed_spread(q[1], rows[:39], w, scale, pair)[0], b[1], rtol=1e-10, atol=1e-12)


def test_rounding_is_the_variance_of_f16():
    x = np.random.default_rng(0).standard_normal(200000) * np.exp2(np.random.default_rng(1).integers(-30, 15, 200000).astype(np.float64))
    for lo, hi in ((2.0 ** -13, 6e4), (2.0 ** -20, 2.0 ** -15)):
        y = x[(np.abs(x) > lo) & (np.abs(x) < hi)]
        assert abs(np.mean((half(y) - y) ** 2 / mla.rounding(y)) - 1) < 0.02
    p = np.exp2(-8 * np.random.default_rng(2).random(200000))
    assert abs(np.mean((half(p) - p) ** 2 / p ** 2) / mla.WEIGHT - 1) < 0.02


@pytest.mark.parametrize("hd,rank,L", [(128, 512, 64), (64, 256, 700), (128, 512, 2048), (128, 512, 12000)])
def test_absorbed(hd, rank, L):
    q, rows, w, scale = case(1, 8, hd, rank, L, seed=L)
    q, rows = q[0], rows
    pair, single = mla.absorbed_spread(q, rows, w, scale, True), mla.absorbed_spread(q, rows, w, scale, False)

    def size(got, to=pair):
        return mla.off(got, *to)

    for got, to in ((absorbed(q, rows, w, scale), pair), (absorbed(q, rows, w, scale, query_pair=False), single)):
        whole, head = size(got, to)
        assert whole < WHOLE and head < HEAD, (whole, head)
    # the low halves of the query and of the sum are seen, too
    if L >= 700:
        assert size(absorbed(q, rows, w, scale, query_pair=False))[0] > WHOLE
        assert size(absorbed(q, rows, w, scale, sum_pair=False))[0] > WHOLE
    tile = np.arange(L) // 64
    right = absorbed(q, rows, w, scale)
    wrong = dict(zeros=np.zeros_like(right), flat=absorbed(q, rows, w, scale, flat=True), unrotated=absorbed(q, rows, w, scale, rotated=False),
                 reversed=right[::-1], half=absorbed(q, rows, w, scale, keep=np.arange(L) < L // 2), one=absorbed(q, rows, w, scale, keep=np.arange(L) != L // 2))
    if L > 64:
        wrong |= {f"tile {t}": absorbed(q, rows, w, scale, keep=tile != t) for t in (0, tile[-1] // 2, tile[-1])}
        twice = np.concatenate([np.arange(L), np.flatnonzero(tile == tile[-1] // 2)])
        wrong["a tile twice"] = absorbed(q, rows, w, scale, keep=twice)
    for name, got in wrong.items():
        assert size(got, single)[0] > 2 * WHOLE, name


@pytest.mark.parametrize("n,heads,hd,rank,before", [(40, 3, 128, 512, 500), (64, 2, 64, 512, 2500), (100, 2, 64, 256, 0)])
def test_expanded(n, heads, hd, rank, before):
    q, rows, w, scale = case(n, heads, hd, rank, before + n, seed=n)
    to = mla.attention_spread(q, rows, w, scale, before)
    whole, head = mla.off(expanded(q, rows, w, scale, before), *to)
    assert whole < WHOLE and head < HEAD, (whole, head)
    wrong = [expanded(q, rows, w, scale, before + 1)]
    if before:
        wrong += [expanded(q, rows, w, scale, before - 1), expanded(q, rows[64:], w, scale, before - 64)]
    for got in wrong:
        assert mla.off(got, *to)[0] > 2 * WHOLE
