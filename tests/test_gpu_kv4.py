"""The 4-bit KV pool on the GPU (``ql_kv4_write``, ``ql_kv4_read``, ``ql_paged_attn_decode_kv4``)
against ``oracle.kv4`` in f64.

* Written bytes equal the oracle's; slots nobody addresses keep theirs. Values read back equal
  d c + m rounded once.
* Attention: an output is one f16 rounding (2^-11 of it, 2^-25 in the subnormal range) from the sum
  of values by weights p. A score is an f32 sum of at most 16 rounded terms, none above
  A = scale max_t sum_b (15 d + |m|) sum_i |q_i|, so its error is below 16 2^-23 A (the tensor
  cores may truncate: a whole step each), which moves every weight by that factor twice (numerator
  and denominator); exp2, its argument and the weights' two f16 parts add 2^-20 at most:
  |o - o_ref| <= 2^-11 |o_ref| + 2^-25 + (32 2^-23 A + 2^-20) max |v|.
"""
import math

import numpy as np
import pytest
import torch

from oracle import kv4

from gpu_util import lib, dev

pytestmark = pytest.mark.gpu


def random_records(rng, blocks, n_kv, hd, size=1.0):
    rec = rng.integers(0, 256, (blocks, n_kv, 20 * hd), dtype=np.uint8)
    w = rec.view(np.float16)
    n = hd // 2
    for k in (0, 2):
        d = 0.27 * size * (1 + 0.2 * rng.standard_normal((blocks, n_kv, n))).clip(0.3, 3)
        w[..., 8 * hd + k * n:8 * hd + (k + 1) * n] = d
        w[..., 8 * hd + (k + 1) * n:8 * hd + (k + 2) * n] = -7.5 * d + 0.5 * size * rng.standard_normal(d.shape)
    return rec


def tables(rng, lens, maxb, spare=3):
    need = [-(-int(n) // 16) for n in lens]
    blocks = sum(need) + spare
    ids = rng.permutation(blocks)
    bt = np.full((len(lens), maxb), -1, np.int32)      # entries past the context are never read
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = ids[at:at + n]
        at += n
    return bt, blocks


def attend(ql, q, rec, bt, lens, scale, out=None, ws=None, stream=None):
    B, H, hd = q.shape
    n_kv, maxb = rec.shape[1], bt.shape[1]
    out = torch.full((B, H, hd), 7.0, dtype=torch.float16, device="cuda") if out is None else out
    if ws is None:
        ws = torch.zeros(ql.ql_paged_attn_kv4_workspace_bytes(B, H, n_kv, hd, maxb), dtype=torch.uint8, device="cuda")
    ql.ql_paged_attn_decode_kv4(q, rec, bt, lens, B, H, n_kv, hd, 16, maxb, rec.shape[0], scale, out, ws, stream)
    return out


def check(got, q, rec, bt, lens, scale):
    want = kv4.paged_attention(q, rec, bt, lens, scale)
    hd = q.shape[2]
    for b, n in enumerate(lens):
        if n == 0:
            assert np.all(got[b] == 7.0)
            continue
        used = rec[bt[b, :-(-int(n) // 16)]].view(np.float16).astype(np.float64)
        d, m = np.abs(used[..., 8 * hd:8 * hd + hd // 2]).max(), np.abs(used[..., 8 * hd + hd // 2:9 * hd]).max()
        A = abs(scale) * (15 * d + m) * np.abs(q[b].astype(np.float64)).sum(-1).max()
        v = 15 * used[..., 9 * hd:9 * hd + hd // 2].max() + np.abs(used[..., 9 * hd + hd // 2:]).max()
        bound = 2.0 ** -11 * np.abs(want[b]) + 2.0 ** -25 + (32 * 2.0 ** -23 * A + 2.0 ** -20) * v
        err = np.abs(got[b].astype(np.float64) - want[b])
        assert np.all(err <= bound), (b, int(n), float((err / bound).max()))


# ---------------------------------------------------------------- write and read
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("half", [False, True])
def test_written_bytes_equal_the_oracle(hd, half):
    ql = lib()
    n_kv, blocks, n = 3, 9, 77
    rng = np.random.default_rng(hd + half)
    k = rng.standard_normal((n, n_kv, hd)).astype(np.float32)
    v = (rng.standard_normal((n, n_kv, hd)) * np.logspace(-5, 3, n)[:, None, None]).astype(np.float32)
    k[3] = 0.0
    v[3] = -0.0
    k[4, :, :32] = np.arange(32) % 16 + 0.5 * (np.arange(32) > 20)     # exact ties with a step of one
    k[4, :, 0], k[4, :, 1] = 0.0, 15.0
    v[5] = 1000.0 + rng.integers(0, 3, (n_kv, hd))                      # the minimum's rounding is most of the range
    k[6] = 1e-7 * rng.standard_normal((n_kv, hd))                       # scales below the least f16
    k[7] *= 20000.0 / np.abs(k[7]).max()
    if half:
        k, v = (np.clip(x, -60000, 60000).astype(np.float16) for x in (k, v))
    slots = rng.permutation(blocks * 16)[:n].astype(np.int64)
    slots[10] = slots[11] = -1                                          # padded rows
    pool = torch.full((blocks, n_kv, 20 * hd), 0xA5, dtype=torch.uint8, device="cuda")
    ql.ql_kv4_write(dev(k), dev(v), dev(slots), n_kv, hd, pool, blocks)
    ql.ql_check_device_error()
    want = np.full((blocks, n_kv, 20 * hd), 0xA5, np.uint8)
    live = slots >= 0
    for g in range(n_kv):
        kv4.place(want, slots[live] // 16, slots[live] % 16, g, kv4.quantize(k[live, g]), kv4.quantize(v[live, g]), hd)
    assert np.array_equal(pool.cpu().numpy(), want)
    # and back, into rows that are strided; padded rows stay as they were
    for dt, nt in ((torch.float32, np.float32), (torch.float16, np.float16)):
        wide = torch.full((n, 2 * n_kv * hd + 16), 7.0, dtype=dt, device="cuda")
        ko, vo = wide[:, :n_kv * hd], wide[:, n_kv * hd:2 * n_kv * hd]
        ql.ql_kv4_read(pool, dev(slots), n_kv, hd, blocks, ko, vo)
        ql.ql_check_device_error()
        kr, vr = kv4.rows_of(want, slots[live] // 16, slots[live] % 16, hd)
        got = wide.cpu().numpy()
        assert np.array_equal(got[live, :n_kv * hd], kr.reshape(live.sum(), -1).astype(nt))
        assert np.array_equal(got[live, n_kv * hd:2 * n_kv * hd], vr.reshape(live.sum(), -1).astype(nt))
        assert np.all(got[~live] == 7.0) and np.all(got[:, 2 * n_kv * hd:] == 7.0)


def test_every_border_of_codes_and_scales_rounds_as_defined():
    """f16 rows whose codes lie on and next to borders, and ranges on and next to f16 borders of the scale."""
    ql = lib()
    hd, n = 64, 4096
    rng = np.random.default_rng(5)
    k = (rng.integers(-4096, 4097, (n, 1, hd)) / 64.0).astype(np.float32)
    v = np.zeros((n, 1, hd), np.float32)
    step = (1024 + rng.integers(0, 1024, (n, 1, 1))) * 2.0 ** -12        # a scale of 11 bits
    v[:] = (np.round(rng.random((n, 1, hd)) * 30) / 2 * step)            # codes at k and k + 1/2
    v[..., 0], v[..., 1], v[..., 32], v[..., 33] = 0.0, (15 * step)[..., 0], 0.0, (15 * step)[..., 0]
    # half an f16 step more: the scale itself is a tie; and one f32 ulp to either side of it
    odd = np.arange(n) % 4
    v[odd == 1, 0, 1] = (15 * (step + 2.0 ** -13))[odd == 1, 0, 0]
    v[odd == 2, 0, 1] = np.nextafter((15 * (step + 2.0 ** -13))[odd == 2, 0, 0].astype(np.float32), np.float32(0))
    v[odd == 3, 0, 1] = np.nextafter((15 * (step + 2.0 ** -13))[odd == 3, 0, 0].astype(np.float32), np.float32(99))
    slots = np.arange(n, dtype=np.int64)
    pool = torch.zeros((n // 16, 1, 20 * hd), dtype=torch.uint8, device="cuda")
    ql.ql_kv4_write(dev(k), dev(v), dev(slots), 1, hd, pool, n // 16)
    want = np.zeros((n // 16, 1, 20 * hd), np.uint8)
    kv4.place(want, slots // 16, slots % 16, 0, kv4.quantize(k[:, 0]), kv4.quantize(v[:, 0]), hd)
    assert np.array_equal(pool.cpu().numpy(), want)


def test_bad_slots_and_values_are_recorded():
    ql = lib()
    hd, n_kv, blocks = 64, 2, 2
    k = torch.ones((2, n_kv, hd), device="cuda")
    for bad in (2 * 16 + 3, -2, 1 << 60):
        pool = torch.zeros((blocks, n_kv, 20 * hd), dtype=torch.uint8, device="cuda")
        ql.ql_kv4_write(k, k, dev(np.array([5, bad], np.int64)), n_kv, hd, pool, blocks)
        with pytest.raises(ql.QLError) as e:
            ql.ql_check_device_error()
        assert e.value.status == ql.QL_EDEVICE and not pool[1].any()
        out = torch.full((2, n_kv, hd), 7.0, device="cuda")
        ql.ql_kv4_read(pool, dev(np.array([5, bad], np.int64)), n_kv, hd, blocks, out, out.clone())
        with pytest.raises(ql.QLError):
            ql.ql_check_device_error()
        assert bool((out[0] == 1).all()) and bool((out[1] == 7).all())
    for x in (float("nan"), float("inf"), -float("inf"), 1e6):
        k2 = k.clone()
        k2[1, 1, 33] = x
        pool = torch.zeros((blocks, n_kv, 20 * hd), dtype=torch.uint8, device="cuda")
        ql.ql_kv4_write(k2, k, dev(np.array([5, 6], np.int64)), n_kv, hd, pool, blocks)
        with pytest.raises(ql.QLError):
            ql.ql_check_device_error()
        out = torch.zeros((1, n_kv, hd), device="cuda")
        ql.ql_kv4_read(pool, dev(np.array([5], np.int64)), n_kv, hd, blocks, out, out.clone())
        assert bool((out == 1).all())
    empty = torch.zeros(0, dtype=torch.int64, device="cuda")
    ql.ql_kv4_write(k[:0], k[:0], empty, n_kv, hd, pool, blocks)
    ql.ql_kv4_read(pool, empty, n_kv, hd, blocks, k[:0], k[:0])
    ql.ql_check_device_error()


def test_offsets_past_32_bits():
    ql = lib()
    hd, n_kv = 128, 8
    blocks = (1 << 32) // (n_kv * 20 * hd) + 40             # 4.3 GB of records
    pool = torch.zeros((blocks, n_kv, 20 * hd), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(2)
    n = 33
    k, v = (rng.standard_normal((n, n_kv, hd)).astype(np.float32) for _ in range(2))
    at = np.concatenate([np.arange(17) + (blocks - 3) * 16, np.arange(16) + 5 * 16]).astype(np.int64)
    ql.ql_kv4_write(dev(k), dev(v), dev(at), n_kv, hd, pool, blocks)
    ko, vo = (torch.zeros((n, n_kv, hd), device="cuda") for _ in range(2))
    ql.ql_kv4_read(pool, dev(at), n_kv, hd, blocks, ko, vo)
    for g in range(n_kv):
        assert np.array_equal(ko[:, g].cpu().numpy(), kv4.dequantize(*kv4.quantize(k[:, g])).astype(np.float32))
        assert np.array_equal(vo[:, g].cpu().numpy(), kv4.dequantize(*kv4.quantize(v[:, g])).astype(np.float32))
    bt = np.array([[blocks - 3, blocks - 2]], np.int32)
    q = rng.standard_normal((1, 16, hd)).astype(np.float16)
    got = attend(ql, dev(q), pool, dev(bt), dev(np.array([17], np.int32)), 0.09)
    ql.ql_check_device_error()
    near = pool[blocks - 3:blocks - 1].cpu().numpy()
    check(got.cpu().numpy(), q, near, bt - (blocks - 3), [17], 0.09)


# ---------------------------------------------------------------- attention
SHAPES = [(8, 2, 128), (4, 4, 128), (8, 1, 128), (3, 1, 128), (12, 12, 64), (6, 2, 64), (8, 1, 64), (16, 1, 128),
          (20, 2, 64), (5, 5, 128)]


@pytest.mark.parametrize("heads,n_kv,hd", SHAPES)
def test_attention_small_lengths(heads, n_kv, hd):
    ql = lib()
    rng = np.random.default_rng(heads * 1000 + hd)
    lens = np.array([1, 2, 15, 16, 17, 0, 31, 33, 64, 127, 129, 300], np.int32)
    bt, blocks = tables(rng, lens, 20)
    rec = random_records(rng, blocks, n_kv, hd)
    q = rng.standard_normal((len(lens), heads, hd)).astype(np.float16)
    got = attend(ql, dev(q), dev(rec), dev(bt), dev(lens), 1 / math.sqrt(hd))
    ql.ql_check_device_error()
    check(got.cpu().numpy(), q, rec, bt, lens, 1 / math.sqrt(hd))


@pytest.mark.parametrize("heads,n_kv,hd", [(8, 2, 128), (4, 4, 64), (16, 2, 128)])
def test_attention_long_contexts_split_over_the_gpu(heads, n_kv, hd):
    ql = lib()
    rng = np.random.default_rng(7)
    lens = np.array([5000, 1, 20011], np.int32)
    bt, blocks = tables(rng, lens, 1300)
    rec = random_records(rng, blocks, n_kv, hd)
    q = rng.standard_normal((3, heads, hd)).astype(np.float16)
    got = attend(ql, dev(q), dev(rec), dev(bt), dev(lens), 1 / math.sqrt(hd))
    check(got.cpu().numpy(), q, rec, bt, lens, 1 / math.sqrt(hd))


@pytest.mark.parametrize("heads,hd", [(8, 128), (32, 128), (8, 64)])
def test_attention_with_many_tiles_per_warp(heads, hd):
    """More tiles than a warp's ring has stages, borders of sequences among them."""
    ql = lib()
    rng = np.random.default_rng(heads + hd)
    lens = np.array([31007, 1234, 16010], np.int32)
    bt, blocks = tables(rng, lens, 2000)
    rec = random_records(rng, blocks, 4, hd)
    q = rng.standard_normal((3, heads, hd)).astype(np.float16)
    got = attend(ql, dev(q), dev(rec), dev(bt), dev(lens), 1 / math.sqrt(hd))
    ql.ql_check_device_error()
    check(got.cpu().numpy(), q, rec, bt, lens, 1 / math.sqrt(hd))


def test_attention_many_short_sequences():
    ql = lib()
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 90, 700).astype(np.int32)
    bt, blocks = tables(rng, lens, 6)
    rec = random_records(rng, blocks, 2, 64)
    q = rng.standard_normal((700, 8, 64)).astype(np.float16)
    got = attend(ql, dev(q), dev(rec), dev(bt), dev(lens), 0.125)
    check(got.cpu().numpy(), q, rec, bt, lens, 0.125)


@pytest.mark.parametrize("size,qsize,scale", [(1e-3, 1e-3, 1.0), (500.0, 1.0, 0.01), (3000.0, 0.05, 0.001), (1.0, 60.0, 0.09),
                                              (1.0, 1.0, 0.0), (1.0, 1.0, -0.1), (1.0, 2.0 ** -20, 30.0)])
def test_attention_of_small_and_large_values(size, qsize, scale):
    ql = lib()
    rng = np.random.default_rng(9)
    lens = np.array([40, 333], np.int32)
    bt, blocks = tables(rng, lens, 32)
    rec = random_records(rng, blocks, 2, 128, size)
    q = (rng.standard_normal((2, 8, 128)) * qsize).astype(np.float16)
    got = attend(ql, dev(q), dev(rec), dev(bt), dev(lens), scale)
    check(got.cpu().numpy(), q, rec, bt, lens, scale)


def test_scores_that_rise_and_fall_along_the_context():
    """A running maximum that moves at every block, and one that is set by the first key."""
    ql = lib()
    rng = np.random.default_rng(10)
    hd, n = 128, 900
    for slope in (0.3, -0.3):
        lens = np.array([n], np.int32)
        bt, blocks = tables(rng, lens, 60)
        rec = np.zeros((blocks, 1, 20 * hd), np.uint8)
        k = 0.2 * rng.standard_normal((n, hd)).astype(np.float32)
        k[:, :] += (slope * np.arange(n) / hd * 2)[:, None].astype(np.float32)
        v = rng.standard_normal((n, hd)).astype(np.float32)
        t = np.arange(n)
        kv4.place(rec, bt[0][t // 16], t % 16, 0, kv4.quantize(k), kv4.quantize(v), hd)
        q = np.ones((1, 4, hd), np.float16)
        q[:, 1:] = rng.standard_normal((1, 3, hd))
        got = attend(ql, dev(q), dev(rec), dev(bt), dev(lens), 0.5)
        check(got.cpu().numpy(), q, rec, bt, lens, 0.5)


def test_stale_bytes_behind_the_context_do_not_count():
    """Slots past the length hold NaN and infinite scales: what a reused block may hold."""
    ql = lib()
    rng = np.random.default_rng(11)
    for hd in (64, 128):
        lens = np.array([1, 17, 30, 5], np.int32)
        bt, blocks = tables(rng, lens, 4)
        rec = random_records(rng, blocks, 2, hd)
        q = rng.standard_normal((4, 8, hd)).astype(np.float16)
        want = rec.copy()
        nb = hd // 32
        for b, n in enumerate(lens):
            blk = bt[b, (n - 1) // 16]
            w = rec[blk].view(np.float16)
            for s in range((n - 1) % 16 + 1, 16):
                for i in range(nb):
                    at = 9 * hd + 4 * nb * (s % 4) + 2 * nb * (s // 8) + 2 * i + (s // 4) % 2
                    w[:, 8 * hd + s * nb + i] = np.nan
                    w[:, 8 * hd + hd // 2 + s * nb + i] = np.inf
                    w[:, at] = np.inf if s & 1 else np.nan
                    w[:, at + hd // 2] = np.nan
        got = attend(ql, dev(q), dev(rec), dev(bt), dev(lens), 0.1)
        check(got.cpu().numpy(), q, want, bt, lens, 0.1)


def test_bad_lengths_and_blocks_are_recorded():
    ql = lib()
    rng = np.random.default_rng(12)
    lens = np.array([40, 50, 64], np.int32)
    bt, blocks = tables(rng, lens, 4)
    rec = random_records(rng, blocks, 2, 128)
    q = rng.standard_normal((3, 8, 128)).astype(np.float16)
    for bad in (65, -1):
        l2 = lens.copy()
        l2[1] = bad
        got = attend(ql, dev(q), dev(rec), dev(bt), dev(l2), 0.1)
        with pytest.raises(ql.QLError) as e:
            ql.ql_check_device_error()
        assert e.value.status == ql.QL_EDEVICE
        l2[1] = 0                                   # left as it was
        check(got.cpu().numpy(), q, rec, bt, l2, 0.1)
    for bad in (blocks, -1):
        b2 = bt.copy()
        b2[1, 1] = bad                              # tokens 16..31 are left out
        got = attend(ql, dev(q), dev(rec), dev(b2), dev(lens), 0.1).cpu().numpy()
        with pytest.raises(ql.QLError):
            ql.ql_check_device_error()
        one = np.array([[bt[1, 0], bt[1, 2], bt[1, 3], 0]], np.int32)
        check(got[1:2], q[1:2], rec, one, [34], 0.1)
        check(got[::2], q[::2], rec, bt[::2], lens[::2], 0.1)


def test_one_workspace_serves_calls_of_other_shapes_and_graphs():
    ql = lib()
    rng = np.random.default_rng(13)
    ws = torch.zeros(ql.ql_paged_attn_kv4_workspace_bytes(4, 16, 2, 128, 400), dtype=torch.uint8, device="cuda")
    calls = []
    for heads, n_kv, hd, lens in ((16, 2, 128, [6000, 1, 700, 0]), (4, 4, 64, [3000, 90]), (8, 1, 128, [6400])):
        lens = np.array(lens, np.int32)
        bt, blocks = tables(rng, lens, 400)
        rec = random_records(rng, blocks, n_kv, hd)
        q = rng.standard_normal((len(lens), heads, hd)).astype(np.float16)
        assert ql.ql_paged_attn_kv4_workspace_bytes(len(lens), heads, n_kv, hd, 400) <= ws.numel()
        calls.append((dev(q), dev(rec), dev(bt), dev(lens), q, rec, bt, lens))
    for _ in range(2):
        for c in calls:
            got = attend(ql, *c[:4], 0.1, ws=ws)
            check(got.cpu().numpy(), *c[4:], 0.1)
    # two captured graphs that share the workspace, replayed in turn on one stream
    s = torch.cuda.Stream()
    graphs = []
    for c in calls[:2]:
        out = torch.full(c[0].shape, 7.0, dtype=torch.float16, device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            attend(ql, *c[:4], 0.1, out=out, ws=ws)
        graphs.append((g, out, c))
    first = []
    for round_ in range(3):
        for g, out, c in graphs:
            out.fill_(7.0)
            with torch.cuda.stream(s):
                s.wait_stream(torch.cuda.current_stream())
                g.replay()
            s.synchronize()
            check(out.cpu().numpy(), *c[4:], 0.1)
            first.append(out.clone())
    assert torch.equal(first[0], first[2]) and torch.equal(first[1], first[5])
    ql.ql_check_device_error()


def test_two_streams_with_workspaces_of_their_own():
    ql = lib()
    rng = np.random.default_rng(14)
    lens = np.array([9000, 300], np.int32)
    bt, blocks = tables(rng, lens, 600)
    rec = random_records(rng, blocks, 4, 128)
    q = rng.standard_normal((2, 16, 128)).astype(np.float16)
    a = [dev(q), dev(rec), dev(bt), dev(lens)]
    want = attend(ql, *a, 0.1)
    torch.cuda.synchronize()
    outs = []
    for _ in range(4):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            outs.append(attend(ql, *a, 0.1, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    check(want.cpu().numpy(), q, rec, bt, lens, 0.1)
