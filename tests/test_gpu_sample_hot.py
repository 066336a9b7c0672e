"""Temperatures up to the end of f32, and rows whose largest logit is near its lowest value: every token that is not masked
weighs nearly the same, and a masked one (-inf, NaN) weighs nothing, as in any other row.

Above a temperature of about 1e36 the second part of 64 log2(e) / T is a subnormal f32 number, off by 2^-150 at most; times
a logit of up to 2^128, in 64ths of an octave (ln 2 / 64 = 0.0108 of the weight): 2^-22 * 0.0108 = 2.6e-9, 2^-28.5 of a weight, on
top of the other temperatures' 2^-29: EPS = 2 (2^-28.5 + 2^-29 + V 2^-40).
"""
import numpy as np
import pytest

from gpu_util import lib

from test_gpu_sample import logits_of
from test_gpu_sample_sets import check_all

pytestmark = pytest.mark.gpu

HOT = [1e37, 2e37, 1e38, 3e38, float(np.finfo(np.float32).max)]
SETS = {"none": {}, "min-p": dict(m=0.3), "top-k 3": dict(k=3), "top-k 128": dict(k=128, p=0.9), "top-k 500": dict(k=500),
        "top-p": dict(p=0.7), "top-p and min-p": dict(p=0.9, m=0.4), "top-p tiny": dict(p=1e-9)}


def hot_eps(V):
    return 2 * (2.0 ** -28.5 + 2.0 ** -29 + V * 2.0 ** -40)


@pytest.mark.parametrize("name", sorted(SETS))
@pytest.mark.parametrize("vocab", [5, 777, 4001, 70001])
@pytest.mark.parametrize("half", [False, True])
def test_masked_tokens_are_never_drawn(name, vocab, half):
    ql = lib()
    rng = np.random.default_rng(vocab + half)
    B = 2 * len(HOT)
    x = logits_of(rng, B, vocab, np.float16 if half else np.float32)
    for r in range(B):
        left = rng.choice(vocab, max(1, min(vocab // 2, (2, 40, 3000)[r % 3])), replace=False)   # few, some, many tokens left
        keep = x[r, left].copy()
        x[r] = -np.inf
        x[r, 1::2] = np.nan
        x[r, left] = keep
    u = np.minimum((np.arange(B) + rng.random(B)) / B, 0.9999999)
    f = {a: np.full(B, v) for a, v in SETS[name].items()}
    check_all(ql, x, u, t=np.repeat(HOT, 2), e=hot_eps(vocab), **f)


@pytest.mark.parametrize("name", sorted(SETS))
def test_logits_of_the_temperature_s_size(name):
    """Logits up to the ends of f32, whose weights differ at these temperatures."""
    ql = lib()
    rng = np.random.default_rng(7)
    B, V = 2 * len(HOT), 5003
    x = (rng.uniform(-1, 1, (B, V)) * 3.4e38).astype(np.float32)
    x[:, ::7] = -np.inf
    x[::2, 3] = np.finfo(np.float32).max
    x[1::2, 4] = -np.finfo(np.float32).max
    f = {a: np.full(B, v) for a, v in SETS[name].items()}
    check_all(ql, x, rng.random(B), t=np.repeat(HOT, 2), e=hot_eps(V), **f)


@pytest.mark.parametrize("name", sorted(SETS))
def test_rows_whose_largest_logit_is_near_the_lowest_value(name):
    ql = lib()
    rng = np.random.default_rng(8)
    low = np.finfo(np.float32).min
    temps = [1.0, 1e30, 1e34, 1e35, 1e36, 1e38]
    B, V = 2 * len(temps), 5003
    x = np.full((B, V), -np.inf, np.float32)
    x[:, ::3] = np.nan
    for r in range(B):
        left = rng.choice(V, (2, 900)[r % 2], replace=False)
        x[r, left] = low
        x[r, left[::2]] = np.float32(-3.4028e38)
    f = {a: np.full(B, v) for a, v in SETS[name].items()}
    check_all(ql, x, rng.random(B), t=np.repeat(temps, 2), e=hot_eps(V), **f)
