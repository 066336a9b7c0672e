"""Rows whose border lies among logits that are almost equal: the first tokens of the order are then found by dividing
the distances down to one value of their scale (24 T / 2^23), the keys of that value, and the indices of one key. Steps are in
units of that scale, so that a value of it holds none, one or several of the tokens around the border."""
import numpy as np
import pytest

from gpu_util import lib

from test_gpu_sample import logits_of
from test_gpu_sample_sets import check_all

pytestmark = pytest.mark.gpu

UNIT = 24.0 / 2 ** 23


def near_ties(rng, B, V, step, behind):
    """Logits 1 - (0, step, 2 step, ...) UNIT in any order (each an f32 number: rounded to 2^-24), the last ones far behind."""
    x = 1.0 - UNIT * np.repeat((step * np.arange(V))[None], B, 0)
    x[:, behind:] = -3.0 - rng.random((B, V - behind))
    return rng.permuted(x, axis=1).astype(np.float32)


@pytest.mark.parametrize("step", [0.02, 0.3, 0.9, 1.0, 1.7, 40.0])
@pytest.mark.parametrize("vocab,behind", [(300, 200), (1126, 1000), (2825, 282), (21372, 140), (72581, 72000)])
def test_borders_among_near_ties(vocab, behind, step):
    ql = lib()
    rng = np.random.default_rng(vocab + int(100 * step))
    B = 9
    x = near_ties(rng, B, vocab, step, behind)
    for k in (100, 126, 127, 128, 129, 200):
        check_all(ql, x, rng.random(B), k=np.full(B, k))
    check_all(ql, x, rng.random(B), k=np.full(B, 128), p=np.full(B, 0.9), m=np.full(B, 1e-3))
    check_all(ql, x, rng.random(B), k=np.full(B, 127), t=np.geomspace(0.01, 1e4, B))
    check_all(ql, x, rng.random(B), p=np.full(B, 0.3))


@pytest.mark.parametrize("temperature", [4.6, 40.0, 1e3, 1e6])
@pytest.mark.parametrize("masked", [0.0, 0.9])
def test_flat_rows_with_a_top_k_of_about_the_list(temperature, masked):
    ql = lib()
    rng = np.random.default_rng(int(temperature))
    for B, V in ((138, 2825), (3, 7329), (4, 72581), (31, 67100)):
        x = logits_of(rng, B, V, size=0.01)
        x[:, rng.random(V) < masked] = -np.inf
        x[:, 0] = 0.5
        for k in (50, 127, 128):
            check_all(ql, x, rng.random(B), k=np.full(B, k), t=np.full(B, temperature))
