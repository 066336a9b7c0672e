"""Pins of the latent attention oracle."""
import numpy as np
import pytest

from oracle import mla


def case(n, heads, hd, rank, L, seed=0):
    g = np.random.default_rng(seed)
    return (g.standard_normal((n, heads, hd + 64)), g.standard_normal((L, rank + 64)),
            g.standard_normal((heads, 2 * hd, rank)) / np.sqrt(rank))


@pytest.mark.parametrize("heads,hd,rank,L", [(1, 64, 256, 1), (3, 64, 256, 17), (5, 128, 512, 40)])
def test_absorbed_is_the_definition(heads, hd, rank, L):
    q, rows, w = case(1, heads, hd, rank, L)
    a, _ = mla.attention(q, rows, w, 0.07)
    b, _ = mla.absorbed(q[0], rows, w, 0.07)
    np.testing.assert_allclose(a[0], b, rtol=1e-11, atol=1e-12)


def test_brute_force():
    q, rows, w = case(2, 2, 64, 256, 5)
    out, _ = mla.attention(q, rows, w, 0.1, before=3)
    for i in range(2):
        for h in range(2):
            s = []
            for t in range(3 + i + 1):
                k = [sum(w[h, d, r] * rows[t, r] for r in range(256)) for d in range(64)]
                s.append(0.1 * (sum(q[i, h, d] * k[d] for d in range(64)) + sum(q[i, h, 64 + j] * rows[t, 256 + j] for j in range(64))))
            e = [np.exp(x - max(s)) for x in s]
            for d in (0, 17, 63):
                v = [sum(w[h, 64 + d, r] * rows[t, r] for r in range(256)) for t in range(len(e))]
                assert abs(out[i, h, d] - sum(a * b for a, b in zip(e, v)) / sum(e)) < 1e-12


def test_one_key_gives_its_value_and_a_zero_query_the_mean():
    q, rows, w = case(1, 2, 64, 256, 9)
    out, _ = mla.absorbed(q[0], rows[:1], w, 0.1)
    np.testing.assert_allclose(out, w[:, 64:] @ rows[0, :256], rtol=1e-12)
    out, _ = mla.absorbed(np.zeros_like(q[0]), rows, w, 0.1)
    np.testing.assert_allclose(out, (w[:, 64:] @ rows[:, :256].T).mean(-1), rtol=1e-10, atol=1e-12)


def test_rows():
    x = np.full((2, 256 + 64), 3.0)
    ones, zeros = np.ones((2, 32)), np.zeros((2, 32))
    row = mla.append(x, np.full(256, 2.0), ones, zeros, 0.0, 256)
    assert np.all(row[:, :256] == 2.0) and np.all(row[:, 256:] == 3.0)
    turned = mla.append(x, np.ones(256), zeros, ones, 0.0, 256)
    assert np.all(turned[:, 256:288] == -3.0) and np.all(turned[:, 288:] == 3.0)
    q = mla.queries(np.ones((2, 4, 128)), zeros, ones, 64)
    assert np.all(q[..., :64] == 1) and np.all(q[..., 64:96] == -1) and np.all(q[..., 96:] == 1)


@pytest.mark.parametrize("defect", ["values first", "unrotated part first", "late key", "no scale"])
def test_defects_are_seen(defect):
    q, rows, w = case(3, 2, 64, 256, 12, seed=1)
    want, bound = mla.attention(q, rows, w, 0.1, before=9)
    if defect == "values first":
        got, _ = mla.attention(q, rows, np.concatenate([w[:, 64:], w[:, :64]], 1), 0.1, before=9)
    elif defect == "unrotated part first":
        got, _ = mla.attention(q, np.concatenate([rows[:, 256:], rows[:, :256]], 1), w, 0.1, before=9)
    elif defect == "late key":
        got, _ = mla.attention(q, rows, w, 0.1, before=8)
    else:
        got, _ = mla.attention(q, rows, w, 1.0, before=9)
    assert np.any(np.abs(got - want) > bound)
