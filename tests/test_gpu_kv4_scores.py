"""Scores of the 4-bit attention whose weight lies in the minima: m times a sum of q that is small beside the head's
largest |q|; and value scales near the end of f16.

A score is scale sum_b (d_b sum_i q_i c_i + m_b Q_b), Q_b = sum_i q_i of block b. Q_b enters as two f16 numbers at a scale
that brings the head's largest |q| to 2^9 .. 2^10: off by 2^-22 |Q_b|, or by the spacing there, 2^-25 of 2^9 (2^-34 of the
largest |q|), at most. Everything else is an f32 sum of at most 32 + 4 terms whose steps truncate at worst, 2^-23 of
what has been added up, none above A = sum_b (15 d_b + |m_b|) sum_i |q_i|:
    e = |scale| max_t (sum_b |m_b| (2^-22 |Q_b| + 2^-34 max |q|) + 36 2^-23 A).
e moves every weight by a factor of 1 + e, in the numerator and in the denominator; the exponential, its argument and the
weights' two parts add 2^-20; the output is rounded to f16:
    |o - o_ref| <= 2^-11 |o_ref| + 2^-25 + (2 e + 2^-20) max |v|.
"""
import numpy as np
import pytest

from oracle import kv4

from gpu_util import lib, dev
from test_gpu_kv4 import attend, random_records

pytestmark = pytest.mark.gpu


def key_blocks(rec, hd):
    """d and m of the keys of consecutive blocks: [tokens, n_kv, nb] each."""
    nb = hd // 32
    w = rec.view(np.float16).astype(np.float64)
    take = lambda at: w[..., at:at + 16 * nb].reshape(*rec.shape[:2], 16, nb).transpose(0, 2, 1, 3).reshape(-1, rec.shape[1], nb)  # noqa: E731
    return take(8 * hd), take(8 * hd + hd // 2)


def check(got, q, rec, n, scale):
    B, H, hd = q.shape
    n_kv, nb = rec.shape[1], hd // 32
    bt = np.arange(rec.shape[0], dtype=np.int32)[None]
    want = kv4.paged_attention(q, rec, np.repeat(bt, B, 0), [n] * B, scale)
    d, m = (np.repeat(x[:n], H // n_kv, 1) for x in key_blocks(rec, hd))                     # [n, H, nb]
    _, v = kv4.rows_of(rec, bt[0][np.arange(n) // 16], np.arange(n) % 16, hd)
    worst = 0.0
    for b in range(B):
        x = q[b].astype(np.float64).reshape(H, nb, 32)
        Q, size, top = np.abs(x.sum(-1)), np.abs(x).sum(-1), np.abs(x).max((-1, -2))[:, None]
        e = abs(scale) * (np.abs(m) * (2.0 ** -22 * Q + 2.0 ** -34 * top) + 36 * 2.0 ** -23 * (15 * d + np.abs(m)) * size).sum(-1).max(0)
        bound = 2.0 ** -11 * np.abs(want[b]) + 2.0 ** -25 + ((2 * e + 2.0 ** -20) * np.abs(v).max())[:, None]
        worst = max(worst, float((np.abs(got[b].astype(np.float64) - want[b]) / bound).max()))
    assert worst <= 1, worst


@pytest.mark.parametrize("heads,n_kv,hd", [(8, 2, 128), (8, 1, 128), (4, 2, 64), (8, 1, 64)])
@pytest.mark.parametrize("largest", [64.0, 60000.0, 2.0 ** -6])
def test_small_sums_of_q_beside_a_large_element(heads, n_kv, hd, largest):
    """One element of q is large and meets keys of 0; the others are 2^-13 of it, all of one sign, and meet blocks whose
    keys are their minimum alone (one value 32 times)."""
    ql = lib()
    rng = np.random.default_rng(heads + hd)
    n, nb = 150, hd // 32
    rec = random_records(rng, 10, n_kv, hd)
    w = rec.view(np.float16)
    w[..., 8 * hd:8 * hd + hd // 2] = 0.0                                       # d of the keys
    m = 1000.0 * rng.standard_normal((10, n_kv, 16, nb))
    m[..., 0] = 0.0
    w[..., 8 * hd + hd // 2:9 * hd] = m.reshape(10, n_kv, -1)
    q = largest * 2.0 ** -13 * (1 + 0.2 * rng.standard_normal((2, heads, hd)))
    q[..., 5] = largest
    q = q.astype(np.float16)
    scale = 1.5 / (1000.0 * 32 * largest * 2.0 ** -13)                          # scores of order one
    bt = np.repeat(np.arange(10, dtype=np.int32)[None], 2, 0)
    got = attend(ql, dev(q), dev(rec), dev(bt), dev(np.array([n, n], np.int32)), scale)
    ql.ql_check_device_error()
    check(got.cpu().numpy(), q, rec, n, scale)


@pytest.mark.parametrize("size", [16000.0, 33000.0, 40000.0, 60000.0, 65504.0])
@pytest.mark.parametrize("rise", [4.0, 5.5, 5.97, 6.5])
@pytest.mark.parametrize("heads,n_kv", [(4, 1), (8, 1)])
def test_value_scales_near_the_end_of_f16(heads, n_kv, rise, size):
    """Codes 0 and 1 of a scale of up to 65504, and weights that rise by `rise` binades from a warp's first tile to its
    second: outputs are finite f16 numbers."""
    ql = lib()
    hd, blocks = 128, 24
    rng = np.random.default_rng(int(size))
    rec = np.zeros((blocks, n_kv, 20 * hd), np.uint8)
    w = rec.view(np.float16)
    rec[..., 8 * hd:16 * hd] = rng.integers(0, 2, (blocks, n_kv, 8 * hd)) * 0x10 + rng.integers(0, 2, (blocks, n_kv, 8 * hd))
    w[..., 9 * hd:9 * hd + hd // 2] = size                                      # d of the values; m = 0
    for blk in range(blocks):                                                   # keys: m alone, the same in all blocks of a row
        w[blk, :, 8 * hd + hd // 2:9 * hd] = rise * (blk // 8)
    q = np.full((1, heads, hd), 1.0 / 128, np.float16)
    n = blocks * 16 - 3
    bt = np.arange(blocks, dtype=np.int32)[None]
    scale = float(np.log(2.0))                                                  # a key of x: 2^x
    got = attend(ql, dev(q), dev(rec), dev(bt), dev(np.array([n], np.int32)), scale).cpu().numpy()
    ql.ql_check_device_error()
    assert np.all(np.isfinite(got))
    check(got, q, rec, n, scale)
