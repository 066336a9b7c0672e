"""Pins of the 4-bit KV oracle and of the sampling oracle (no GPU), and the library's refusals."""
import math

import numpy as np
import pytest

from oracle import kv4, sample as osample


@pytest.fixture(scope="module")
def ql():
    from quantized_transformer_decode_ql_gb300 import build
    build.build()
    import quantized_transformer_decode_ql_gb300 as q
    return q


def test_block_by_hand():
    # min -1, max 2: d = 0.2 in f16 (0.199951171875), codes of a ramp over 15 steps are 0..15
    d = float(np.float16(0.2))
    x = np.concatenate([np.float32(-1) + np.float32(0.2) * np.arange(16, dtype=np.float32), np.full(16, -1, np.float32)])
    c, dd, m = kv4.quantize(x[None])
    assert float(dd[0, 0]) == d and float(m[0, 0]) == -1.0
    assert list(c[0, :16]) == list(range(16)) and not c[0, 16:].any()
    y = kv4.dequantize(c, dd, m)
    assert y[0, 3] == -1 + 3 * d


def test_ties_go_to_even_and_a_constant_block_is_its_minimum():
    x = np.zeros(32, np.float32)
    x[:4] = [0.0, 15.0, 2.5, 3.5]
    c, d, m = kv4.quantize(x[None])
    assert float(d[0, 0]) == 1.0 and list(c[0, :4]) == [0, 15, 2, 4]
    c, d, m = kv4.quantize(np.full((1, 32), -3.25, np.float32))
    assert not c.any() and float(d[0, 0]) == 0 and float(m[0, 0]) == -3.25
    c, d, m = kv4.quantize(np.full((1, 32), -0.0, np.float32))
    assert m.view(np.uint16)[0, 0] == 0


def test_error_bound():
    rng = np.random.default_rng(0)
    for s in (1e-3, 1.0, 300.0):
        x = (rng.standard_normal((50, 128)) * s).astype(np.float32)
        c, d, m = kv4.quantize(x)
        # half a step, plus what rounding m and d to f16 takes off the ends of the range
        ends = np.abs(x).reshape(50, 4, 32).max(-1) * 2.0 ** -11 + 15 * d.astype(np.float64) * 2.0 ** -11 + 2.0 ** -20
        bound = np.repeat(d.astype(np.float64) / 2 + 2 * ends, 32, axis=1)
        assert np.all(np.abs(kv4.dequantize(c, d, m) - x) <= bound)


@pytest.mark.parametrize("hd", [64, 128])
def test_layout_holds_every_field_once(hd):
    rng = np.random.default_rng(hd)
    n_kv, blocks = 2, 3
    rec = np.zeros((blocks, n_kv, kv4.record_bytes(hd)), np.uint8)
    k = rng.standard_normal((blocks * 16, n_kv, hd)).astype(np.float32)
    v = rng.standard_normal((blocks * 16, n_kv, hd)).astype(np.float32)
    t = np.arange(blocks * 16)
    for g in range(n_kv):
        kv4.place(rec, t // 16, t % 16, g, kv4.quantize(k[:, g]), kv4.quantize(v[:, g]), hd)
    kk, vv = kv4.rows_of(rec, t // 16, t % 16, hd)
    for g in range(n_kv):
        assert np.array_equal(kk[:, g], kv4.dequantize(*kv4.quantize(k[:, g])))
        assert np.array_equal(vv[:, g], kv4.dequantize(*kv4.quantize(v[:, g])))


def test_attention_of_one_token_is_its_value():
    rng = np.random.default_rng(1)
    rec = np.zeros((2, 1, kv4.record_bytes(64)), np.uint8)
    k, v = (rng.standard_normal((1, 64)).astype(np.float32) for _ in range(2))
    kv4.place(rec, [1], [0], 0, kv4.quantize(k), kv4.quantize(v), 64)
    out = kv4.paged_attention(rng.standard_normal((1, 3, 64)), rec, [[1, 0]], [1], 0.125)
    assert np.allclose(out[0], kv4.dequantize(*kv4.quantize(v)), rtol=0, atol=1e-15)


def test_sampling_by_hand():
    l = np.log(np.array([1.0, 4.0, 2.0, 1.0]))
    assert osample.sample(l, 0.0)[0] == 0 and osample.sample(l, 0.124)[0] == 0
    assert osample.sample(l, 0.126)[0] == 1 and osample.sample(l, 0.9)[0] == 3
    assert list(osample.kept(l, top_k=3)[0]) == [0, 1, 2]        # the tie goes to the lowest index
    assert list(osample.kept(l, top_p=0.5)[0]) == [1]
    assert list(osample.kept(l, top_p=0.501)[0]) == [1, 2]
    assert list(osample.kept(l, top_k=2, top_p=0.67)[0]) == [1, 2]   # 4 / 6 of the two kept is short of 0.67
    assert list(osample.kept(l, min_p=0.49)[0]) == [1, 2] and list(osample.kept(l, min_p=1.0)[0]) == [1]
    assert osample.sample(l, 0.5, temperature=0)[:2] == (1, 1.0)
    assert osample.sample(np.full(3, -np.inf), 0.5)[:2] == (-1, 0.0)
    p = osample.sample(l, 0.3, temperature=0.5)
    assert p[0] == 1 and abs(p[1] - 16 / 22) < 1e-12


def test_refusals_without_gpu(ql):
    L, E = ql.lib(), ql.QL_EINVAL
    assert ql.ql_kv4_record_bytes(128) == 2560 and ql.ql_kv4_record_bytes(64) == 1280 and ql.ql_kv4_record_bytes(96) == 0

    def write(k=4096, v=8192, dtype=0, ks=256, vs=256, slots=64, n=3, n_kv=2, hd=128, pool=1024, blocks=4):
        return L.ql_kv4_write(k, v, dtype, ks, vs, slots, n, n_kv, hd, pool, blocks, None)

    def read(k=4096, v=8192, dtype=0, ks=256, vs=256, slots=64, n=3, n_kv=2, hd=128, pool=1024, blocks=4):
        return L.ql_kv4_read(pool, slots, n, n_kv, hd, blocks, k, v, dtype, ks, vs, None)

    for f in (write, read):
        for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(pool=None), dict(dtype=2), dict(hd=96), dict(n=-1),
                    dict(n_kv=0), dict(blocks=0), dict(k=4098), dict(v=8200), dict(pool=1028), dict(slots=65),
                    dict(ks=255), dict(vs=128), dict(ks=258), dict(dtype=1, ks=260), dict(n=1 << 60)):
            assert f(**bad) == E, bad
        assert f(n=0, k=None, v=None, slots=None, pool=None) == 0     # nothing to do

    def attn(q=64, pool=1024, bt=64, lens=64, batch=2, h=8, kv=2, hd=128, bs=16, maxb=4, blocks=9, out=64, ws=64, wb=1 << 40):
        return L.ql_paged_attn_decode_kv4(q, pool, bt, lens, batch, h, kv, hd, bs, maxb, blocks, 0.1, out, ws, wb, None)

    for bad in (dict(q=None), dict(pool=None), dict(bt=None), dict(lens=None), dict(out=None), dict(ws=None), dict(batch=0),
                dict(batch=70000), dict(h=7), dict(h=0), dict(kv=0), dict(hd=96), dict(bs=32), dict(maxb=0), dict(blocks=0),
                dict(q=66), dict(pool=1032), dict(out=65), dict(ws=72), dict(wb=0)):
        assert attn(**bad) == E, bad
    for bad in ((0, 8, 2, 128, 4), (1, 7, 2, 128, 4), (1, 8, 2, 96, 4), (1, 8, 2, 128, 0)):
        assert ql.ql_paged_attn_kv4_workspace_bytes(*bad) == 0

    def draw(lg=64, dtype=0, stride=100, batch=2, vocab=100, t=None, k=None, p=None, m=None, u=64, act=None, tok=64, pr=None):
        return L.ql_sample(lg, dtype, stride, batch, vocab, t, k, p, m, u, act, tok, pr, None)

    for bad in (dict(lg=None), dict(u=None), dict(tok=None), dict(dtype=3), dict(batch=0), dict(vocab=0), dict(vocab=360449),
                dict(stride=99), dict(lg=66), dict(dtype=1, lg=65), dict(t=2), dict(k=2), dict(p=1), dict(m=3), dict(u=66),
                dict(act=2), dict(tok=66), dict(pr=2)):
        assert draw(**bad) == E, bad


def test_wrappers_refuse_tensors_that_do_not_fit(ql):
    import torch
    k = torch.zeros((3, 2, 64))
    slots = torch.zeros(3, dtype=torch.int64)
    pool = torch.zeros((2, 2, 1280), dtype=torch.uint8)
    for kk, vv in ((k, k.half()), (k.double(), k.double()), (k[:2], k), (k.transpose(1, 2), k)):
        with pytest.raises(ql.QLError) as e:
            ql.ql_kv4_write(kk, vv, slots, 2, 64, pool, 2)
        assert e.value.status == ql.QL_EINVAL
    with pytest.raises(ql.QLError):
        ql.ql_sample(torch.zeros((2, 10)).t(), torch.zeros(10), torch.zeros(10, dtype=torch.int32))
    with pytest.raises(ql.QLError):
        ql.ql_sample(torch.zeros((2, 10), dtype=torch.float64), torch.zeros(2), torch.zeros(2, dtype=torch.int32))
