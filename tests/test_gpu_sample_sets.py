"""Every drawn token is one that the tolerance allows: no row is left out because a border is near.

A share of the kept weight is off by EPS at most, so the top-p border is that of a p between p (1 - EPS) and p (1 + EPS), and
the token lies, in index order, between the first that the definition gives for u - EPS and the last for u + EPS, over
those borders; it is one of the tokens kept at p (1 + EPS). Its probability is its weight over a kept weight between those
of the two borders, within EPS and one f32 rounding.
"""
import numpy as np
import pytest

from oracle import sample as osample

from gpu_util import lib, dev

from test_gpu_sample import draw, eps, logits_of
from test_gpu_sample_paths import SETS, args_of

pytestmark = pytest.mark.gpu


def allowed(row, u, e, temperature, top_k, top_p, min_p):
    """(tokens kept at most, first and last place among them, weights, least and largest kept weight)."""
    ends, sums = [], []
    index = w = None
    for p in {top_p, min(1.0, top_p * (1 - e)), min(1.0, top_p * (1 + e))}:
        at, weights = osample.kept(row, temperature, top_k, p, min_p)
        if index is None or len(at) > len(index):
            index, w = at, weights
        total = np.cumsum(weights)
        sums.append(total[-1])
        for x in (u - e, u + e):
            ends.append(int(at[min(int(np.searchsorted(total, max(x, 0.0) * total[-1], side="right")), len(at) - 1)]))
    return index, min(ends), max(ends), w, min(sums), max(sums)


def check_all(ql, x, u, t=None, k=None, p=None, m=None, e=None):
    x = np.asarray(x)
    B, V = x.shape
    e = eps(V) if e is None else e
    u = np.asarray(u, np.float32)
    f = [None if a is None else np.asarray(a, d) for a, d in ((t, np.float32), (k, np.int32), (p, np.float32), (m, np.float32))]
    tokens, probs = draw(ql, dev(x), dev(u), *[None if a is None else dev(a) for a in f])
    ql.ql_check_device_error()
    tokens, probs = tokens.cpu().numpy(), probs.cpu().numpy()
    single = 0
    for r in range(B):
        args = dict(temperature=1.0 if t is None else float(f[0][r]), top_k=0 if k is None else int(f[1][r]),
                    top_p=1.0 if p is None else float(f[2][r]), min_p=0.0 if m is None else float(f[3][r]))
        index, lo, hi, w, low, high = allowed(x[r], float(u[r]), e, **args)
        tok = int(tokens[r])
        at = int(np.searchsorted(index, tok))
        assert at < len(index) and index[at] == tok and lo <= tok <= hi, (r, args, float(u[r]), tok, lo, hi)
        least, most = w[at] / high, w[at] / low
        assert least - e - 2.0 ** -24 * least <= probs[r] <= most + e + 2.0 ** -24 * most, (r, args, float(probs[r]), least, most)
        single += lo == hi
    return single


@pytest.mark.parametrize("batch", [1, 4, 5])
@pytest.mark.parametrize("vocab", [65536, 65537, 151936, 360448])
def test_few_long_rows(batch, vocab):
    ql = lib()
    rng = np.random.default_rng(2 * vocab + batch)
    x = logits_of(rng, batch, vocab)
    for name in SETS:
        check_all(ql, x, rng.random(batch), **args_of(name, batch))


@pytest.mark.parametrize("name", [n for n in SETS if n != "none"])
@pytest.mark.parametrize("batch", [2, 24])
def test_borders_in_a_crowd_of_equal_logits(batch, name):
    """As in test_gpu_sample_paths.py, with a share of 0.9003 in top-k 700, which is no whole number of its equal tokens."""
    ql = lib()
    rng = np.random.default_rng(100 + batch)
    V = 100003
    x = np.minimum(rng.standard_normal((batch, V)), 0.84).astype(np.float32) * 3
    x[:, ::10] = np.float32(1.25)
    f = args_of(name, batch)
    if name == "top-k 700":
        f["p"] = np.full(batch, 0.9003)
    check_all(ql, x, rng.random(batch), **f)


def test_the_check_refuses_wrong_tokens():
    """A token beside the drawn one, one outside the kept ones and one that was never written are outside the allowed."""
    rng = np.random.default_rng(1)
    x = logits_of(rng, 20, 5000)
    for r in range(20):
        index, lo, hi, *_ = allowed(x[r], 0.37, eps(5000), 1.0, 300, 0.9, 0.0)
        assert lo == hi and len(index) < 300 and lo in index and -7 not in index


@pytest.mark.parametrize("vocab", [65536, 151936])
def test_rows_without_top_p_are_certain(vocab):
    ql = lib()
    rng = np.random.default_rng(vocab + 1)
    x = logits_of(rng, 4, vocab)
    sure = total = 0
    for name in SETS:
        if "p" in SETS[name]:
            continue
        sure += check_all(ql, x, (np.arange(4) + rng.random(4)) / 4.001, **args_of(name, 4))
        total += 4
    assert sure >= 0.9 * total
