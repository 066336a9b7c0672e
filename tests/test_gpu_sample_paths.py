"""The sampler where its search takes another course: rows spread over 16 CTAs, borders in a crowd of equal
or nearly equal logits (more candidates than the lists hold), fewer tokens than top-k asks for. The
tolerances are those of test_gpu_sample.py, whose check this uses."""
import numpy as np
import pytest

from gpu_util import lib

from test_gpu_sample import check, logits_of

pytestmark = pytest.mark.gpu

SETS = {"none": {}, "top-k 50": dict(k=50), "top-k 128": dict(k=128, p=0.97), "top-k 129": dict(k=129, p=0.97),
        "top-k 700": dict(k=700, p=0.9, m=0.001), "top-p 0.9": dict(p=0.9), "top-p 0.2": dict(p=0.2, t=1.5),
        "min-p": dict(m=0.05), "top-p and min-p": dict(p=0.995, m=1e-4)}


def args_of(name, B):
    return {a: np.full(B, v) for a, v in SETS[name].items()}


@pytest.mark.parametrize("batch", [1, 4, 5])
@pytest.mark.parametrize("vocab", [65536, 65537, 151936, 360448])
def test_few_long_rows(batch, vocab):
    ql = lib()
    rng = np.random.default_rng(vocab + batch)
    x = logits_of(rng, batch, vocab)
    for name in SETS:
        check(ql, x, rng.random(batch), **args_of(name, batch), sure=0)


@pytest.mark.parametrize("name", [n for n in SETS if n != "none"])
@pytest.mark.parametrize("batch", [2, 24])
def test_borders_in_a_crowd_of_equal_logits(batch, name):
    """A fifth of the row is its largest logit, another tenth shares one value below it. The 700 kept by top-k 700 are
    equal, and 0.9 of them (as f32: 629.99998) is nearer to 630 tokens than 630 eps(V) = 1.2e-4, so none of its rows
    counts as certain. Top-p 0.995 falls where a token weighs about e^-3, and eps(V) = 1.9e-7 of the row's weight (over 20000
    tokens of e^2.5 and as much again: 3e5) is 0.06: about as much, so whether a row is certain there is chance."""
    ql = lib()
    rng = np.random.default_rng(batch)
    V = 100003
    x = np.minimum(rng.standard_normal((batch, V)), 0.84).astype(np.float32) * 3
    x[:, ::10] = np.float32(1.25)
    check(ql, x, rng.random(batch), **args_of(name, batch), sure=0 if name in ("top-k 700", "top-p and min-p") else 0.5)


@pytest.mark.parametrize("name", [n for n in SETS if n != "none"])
def test_nearly_flat_rows(name):
    """At a temperature of 40 all logits lie within a few bins of the first histogram."""
    ql = lib()
    rng = np.random.default_rng(5)
    x = logits_of(rng, 12, 70001)
    check(ql, x, rng.random(12), **{**args_of(name, 12), "t": np.full(12, 40.0)}, sure=0.5)


@pytest.mark.parametrize("vocab", [40, 5000, 70001])
def test_fewer_tokens_than_top_k(vocab):
    ql = lib()
    rng = np.random.default_rng(vocab)
    x = np.full((10, vocab), -np.inf, np.float32)
    for r in range(10):
        at = rng.choice(vocab, 1 + 4 * r, replace=False)
        x[r, at] = rng.standard_normal(at.size).astype(np.float32)
    for k in (30, 128, 4000):
        check(ql, x, rng.random(10), k=np.full(10, k), p=np.full(10, 0.95))
        check(ql, x, rng.random(10), k=np.full(10, k))


@pytest.mark.parametrize("top_k", [None, 3, 300])
def test_more_rows_than_a_grid_dimension_of_16_bits(top_k):
    """Row by row the same as a call of those rows alone, and the arg max where the temperature is 0."""
    import torch
    from gpu_util import dev
    ql = lib()
    rng = np.random.default_rng(9)
    B, V = 70001, 41
    x = dev(logits_of(rng, B, V))
    t = dev((np.arange(B) % 3).astype(np.float32))
    u = dev(rng.random(B).astype(np.float32))
    k = None if top_k is None else torch.full((B,), top_k, dtype=torch.int32, device="cuda")
    tokens = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    ql.ql_sample(x, u, tokens, temperature=t, top_k=k)
    ql.ql_check_device_error()
    assert torch.equal(tokens[::3].long(), x[::3].argmax(1))
    assert bool(((tokens >= 0) & (tokens < V)).all())
    for a in (0, 33333, B - 5):
        part = torch.full((5,), -7, dtype=torch.int32, device="cuda")
        ql.ql_sample(x[a:a + 5], u[a:a + 5], part, temperature=t[a:a + 5], top_k=None if k is None else k[a:a + 5])
        assert torch.equal(part, tokens[a:a + 5])
