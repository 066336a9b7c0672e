"""The token sampler on the GPU (``ql_sample``) against ``oracle.sample`` in f64.

Weights are 40-bit fixed-point numbers with a relative error below 2^-29 before that rounding (the
exponent's two roundings in 64ths of an octave, the series and two integer products, 2^-31 or so
each), so a share of the kept weight is off by at most EPS(V) = 2 (2^-29 + V 2^-40): the token has to
be the oracle's wherever u is farther than that from a border of its share and the top-p border does
not move when p does by that much. Probabilities are one f32 rounding and EPS from the oracle's.
"""
import math

import numpy as np
import pytest
import torch

from oracle import sample as osample

from gpu_util import lib, dev

pytestmark = pytest.mark.gpu


def eps(vocab):
    return 2 * (2.0 ** -29 + vocab * 2.0 ** -40)


def draw(ql, logits, u, t=None, k=None, p=None, m=None, active=None, stream=None):
    B = logits.shape[0]
    tokens = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    probs = torch.full((B,), -7.0, device="cuda")
    ql.ql_sample(logits, u, tokens, temperature=t, top_k=k, top_p=p, min_p=m, probs=probs, active=active, stream=stream)
    return tokens, probs


def check(ql, x, u, t=None, k=None, p=None, m=None, logits=None, sure=0.9):
    """x: [B, V] numpy as the device holds it; the filters are numpy [B] or None. `sure`: the least share of rows that
    the borders leave certain."""
    x = np.asarray(x)
    B, V = x.shape
    u = np.asarray(u, np.float32)
    f = [None if a is None else np.asarray(a, d) for a, d in ((t, np.float32), (k, np.int32), (p, np.float32), (m, np.float32))]
    d = [None if a is None else dev(a) for a in f]
    tokens, probs = draw(ql, dev(x) if logits is None else logits, dev(u), *d)
    ql.ql_check_device_error()
    tokens, probs = tokens.cpu().numpy(), probs.cpu().numpy()
    certain = 0
    for r in range(B):
        args = dict(temperature=1.0 if t is None else float(f[0][r]), top_k=0 if k is None else int(f[1][r]),
                    top_p=1.0 if p is None else float(f[2][r]), min_p=0.0 if m is None else float(f[3][r]))
        tok, prob, gap = osample.sample(x[r], float(u[r]), **args)
        if args["temperature"] > 0 and args["top_p"] < 1:
            near = [len(osample.kept(x[r], **{**args, "top_p": min(args["top_p"] * q, 1.0)})[0]) for q in (1 - eps(V), 1 + eps(V))]
            if near[0] != near[1]:
                continue
        if gap <= eps(V):
            continue
        certain += 1
        assert tokens[r] == tok, (r, args, float(u[r]), int(tokens[r]), tok, gap)
        assert abs(float(probs[r]) - prob) <= 2.0 ** -24 * prob + eps(V), (r, probs[r], prob)
    assert certain >= sure * B, certain
    return tokens


def logits_of(rng, B, V, dtype=np.float32, size=2.5):
    x = rng.standard_normal((B, V)) * size
    x[:, rng.integers(0, V, 4)] += 3
    return x.astype(dtype)


FILTERS = {
    "none": {},
    "temperature": dict(t=0.7),
    "hot": dict(t=40.0),
    "cold": dict(t=0.02),
    "top-k 1": dict(k=1),
    "top-k 50": dict(k=50),
    "top-k all": dict(k=10 ** 9),
    "top-p 0.9": dict(p=0.9),
    "top-p 0.3": dict(p=0.3, t=1.3),
    "top-p tiny": dict(p=1e-9),
    "min-p 0.1": dict(m=0.1, t=0.8),
    "min-p 1": dict(m=1.0),
    "all": dict(t=0.9, k=40, p=0.95, m=0.02),
    "k and p": dict(k=700, p=0.8, t=1.5),
}


@pytest.mark.parametrize("name", sorted(FILTERS))
@pytest.mark.parametrize("vocab", [1, 2, 31, 257, 1000, 8193, 33001])
@pytest.mark.parametrize("half", [False, True])
def test_filters_and_sizes(name, vocab, half):
    ql = lib()
    rng = np.random.default_rng(vocab * 2 + half)
    B = 24
    x = logits_of(rng, B, vocab, np.float16 if half else np.float32)
    u = (np.arange(B) + rng.random(B)) / B
    f = {a: np.full(B, v) for a, v in FILTERS[name].items()}
    check(ql, x, np.minimum(u, 0.9999999), **f)


@pytest.mark.parametrize("vocab", [151936, 360448])
@pytest.mark.parametrize("name", ["none", "top-p 0.9", "top-k 50", "all", "min-p 0.1"])
def test_large_vocabularies(vocab, name):
    ql = lib()
    rng = np.random.default_rng(vocab)
    x = logits_of(rng, 5, vocab)
    f = {a: np.full(5, v) for a, v in FILTERS[name].items()}
    check(ql, x, rng.random(5), sure=0.5, **f)


def test_rows_with_filters_of_their_own_and_strided_rows():
    ql = lib()
    rng = np.random.default_rng(3)
    B, V = 40, 5003
    for dtype in (np.float32, np.float16):
        for pad, off in ((0, 0), (1, 0), (3, 1), (2, 3)):
            x = logits_of(rng, B, V, dtype)
            wide = torch.full((B * (V + pad) + off,), 50.0, dtype=torch.float32 if dtype == np.float32 else torch.float16, device="cuda")
            view = wide[off:].view(B, V + pad)[:, :V]
            view.copy_(dev(x))
            check(ql, x, rng.random(B), t=rng.choice([0.0, 0.5, 1.0, 2.0], B), k=rng.choice([0, 1, 7, 900, 6000], B),
                  p=rng.choice([1.0, 0.5, 0.99, 2.0], B), m=rng.choice([0.0, 0.01, 0.5], B), logits=view, sure=0.8)


def test_ties_go_to_the_lowest_index():
    ql = lib()
    V = 3001
    x = np.zeros((6, V), np.float32)
    x[:, ::2] = -0.0                                    # a zero is a zero
    u = np.array([0.0, 0.1, 0.5, 0.77, 0.9999, 0.3], np.float32)
    got = check(ql, x, u, sure=0.5)
    got = check(ql, x, u, k=np.full(6, 10), sure=0.5)
    assert got.max() < 10
    got = check(ql, x, u, p=np.full(6, 0.25), sure=0.5)
    assert got.max() <= V // 4
    got = check(ql, x, u, t=np.zeros(6))
    assert not got.any()
    # groups of ties, the border inside a group
    rng = np.random.default_rng(4)
    x = rng.integers(0, 5, (30, V)).astype(np.float32)
    check(ql, x, rng.random(30), k=rng.integers(1, V, 30))
    check(ql, x, rng.random(30), p=0.02 + 0.9 * rng.random(30))
    check(ql, (x * 100).astype(np.float16), rng.random(30), k=rng.integers(1, V, 30))


def test_masked_rows():
    ql = lib()
    rng = np.random.default_rng(5)
    V = 777
    inf = np.inf
    x = logits_of(rng, 12, V)
    x[0] = -inf                                          # nothing left
    x[1] = np.nan
    x[2, :] = -inf
    x[2, 400] = -5.0                                     # one token left
    x[3, ::2] = np.nan
    x[4, 1::2] = -inf
    x[5, :] = np.finfo(np.float32).min                    # a mask of the lowest value that leaves nothing else
    x[6, :700] = np.finfo(np.float32).min
    x[7, 10] = inf                                        # counts as the largest finite value
    x[8, 10] = x[8, 20] = inf
    x[9] = 3e38
    x[9, 5] = -3e38
    x[10] = -inf
    x[10, 3] = np.finfo(np.float32).min
    u = np.full(12, 0.6, np.float32)
    for f in ({}, dict(k=np.full(12, 3)), dict(p=np.full(12, 0.7)), dict(m=np.full(12, 0.2)), dict(t=np.full(12, 1e-30)),
              dict(t=np.full(12, 1e30)), dict(t=np.zeros(12)), dict(k=np.full(12, 500), p=np.full(12, 0.9), m=np.full(12, 0.01))):
        got = check(ql, x, u, **f)
        assert got[0] == -1 and got[1] == -1 and got[2] == 400 and got[7] == 10 and got[10] == 3


def test_large_logits_and_small_temperatures():
    ql = lib()
    rng = np.random.default_rng(6)
    x = logits_of(rng, 16, 4001)
    scale = np.logspace(0, 30, 16)[:, None]
    y = (x * scale).astype(np.float32)
    t = scale[:, 0].astype(np.float32)
    check(ql, y, rng.random(16), t=t)
    check(ql, y, rng.random(16), t=t, p=np.full(16, 0.9), m=np.full(16, 0.01))
    check(ql, (x / scale).astype(np.float32), rng.random(16), t=(1 / t).astype(np.float32))
    check(ql, (x + 1e4).astype(np.float32), rng.random(16), k=np.full(16, 100))
    check(ql, (x - 3e6).astype(np.float32), rng.random(16), p=np.full(16, 0.9))


def test_shares_of_a_row_follow_its_weights():
    """One row, u on a grid: the tokens drawn are the running sum's, one after the other."""
    ql = lib()
    rng = np.random.default_rng(7)
    V, B = 900, 4096
    row = logits_of(rng, 1, V)
    u = ((np.arange(B) + 0.5) / B).astype(np.float32)
    got = check(ql, np.repeat(row, B, 0), u, p=np.full(B, 0.95))
    assert np.all(np.diff(got) >= 0)


def test_bad_arguments_of_a_row_are_recorded():
    ql = lib()
    rng = np.random.default_rng(8)
    x = dev(logits_of(rng, 3, 100))
    u = dev(np.full(3, 0.5, np.float32))
    one = np.ones(3, np.float32)
    for name, bad in (("t", -1.0), ("t", np.nan), ("t", np.inf), ("p", np.nan), ("m", np.nan), ("u", -0.1), ("u", 1.0), ("u", np.nan)):
        a = one.copy() * 0.5
        a[1] = bad
        f = {} if name == "u" else {name: dev(a)}
        tokens, probs = draw(ql, x, dev(a) if name == "u" else u, **f)
        with pytest.raises(ql.QLError) as e:
            ql.ql_check_device_error()
        assert e.value.status == ql.QL_EDEVICE
        assert int(tokens[1]) == -1 and float(probs[1]) == 0 and int(tokens[0]) >= 0 and int(tokens[2]) >= 0


def test_inactive_rows_keep_their_token():
    ql = lib()
    rng = np.random.default_rng(9)
    x = logits_of(rng, 6, 400)
    act = dev(np.array([1, 0, 1, 0, 0, 1], np.int32))
    tokens, probs = draw(ql, dev(x), dev(np.full(6, 0.4, np.float32)), active=act)
    for r in range(6):
        if act[r]:
            assert int(tokens[r]) == osample.sample(x[r], float(np.float32(0.4)))[0]
        else:
            assert int(tokens[r]) == -7 and float(probs[r]) == -7


def test_streams_and_captured_graphs():
    ql = lib()
    rng = np.random.default_rng(10)
    x = dev(logits_of(rng, 20, 60013))
    u = dev(rng.random(20).astype(np.float32))
    p = dev(np.full(20, 0.9, np.float32))
    want = draw(ql, x, u, p=p)
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            got.append(draw(ql, x, u, p=p, stream=s))
    torch.cuda.synchronize()
    for t, q in got:
        assert torch.equal(t, want[0]) and torch.equal(q, want[1])
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    tokens = torch.zeros(20, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        ql.ql_sample(x, u, tokens, top_p=p)
    for _ in range(2):
        u2 = torch.rand(20, device="cuda")
        u.copy_(u2)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(tokens, draw(ql, x, u, p=p)[0])
