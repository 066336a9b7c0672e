"""Latent attention on the GPU against the f64 oracle: the rows' append, the single-token form, the prompt chunk, and
the three together. Tolerances are the oracle's bounds: half a step for every rounding to f16 and a step of f32 for every
addition (``oracle/mla.py``)."""
import math

import numpy as np
import pytest
import torch

from gpu_util import dev, lib
from oracle import mla

pytestmark = pytest.mark.gpu

EPS = 1e-6


def tables(max_position, theta=1e6):
    c, s = np.empty((max_position, 32), np.float32), np.empty((max_position, 32), np.float32)
    lib().ql_rope_tables(c, s, theta)
    return c, s


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("n,heads,hd,rank,f16,strided", [
    (1, 1, 128, 512, False, False), (1, 32, 128, 512, True, False), (2, 5, 64, 256, False, True), (17, 40, 64, 512, True, True),
    (33, 7, 128, 256, False, True), (300, 3, 128, 512, False, False), (5, 130, 64, 256, True, False)])
def test_append(n, heads, hd, rank, f16, strided):
    ql = lib()
    g = np.random.default_rng(n * heads)
    dt = np.float16 if f16 else np.float32
    extra = 64 if strided else 0
    q = (g.standard_normal((n, heads * (hd + 64) + extra)) * 3).astype(dt)
    kv = (g.standard_normal((n, rank + 64 + extra)) * np.exp(g.standard_normal((n, 1)) * 2)).astype(dt)
    w = (1 + 0.1 * g.standard_normal(rank)).astype(np.float32)
    cos, sin = tables(700)
    blocks = n // 16 + 4
    pos = g.integers(0, 700, n).astype(np.int32)
    slots = g.permutation(blocks * 16)[:n].astype(np.int64)
    if n > 4:
        slots[2] = -1
    row = rank + 64
    pool = torch.full((blocks, 16, row), 7.0, dtype=torch.float16, device="cuda")
    q_out = torch.full((n, heads, hd + 64), 9.0, dtype=torch.float16, device="cuda")
    qd, kd = dev(q), dev(kv)
    ql.ql_mla_append(qd[:, extra:].unflatten(1, (heads, hd + 64)), kd[:, extra:], dev(w), dev(cos), dev(sin), dev(pos), dev(slots), EPS,
                     heads, hd, rank, 64, q_out, pool, blocks, 700)
    torch.cuda.synchronize()
    ql.ql_check_device_error()
    want = mla.append(kv[:, extra:], w, cos[pos], sin[pos], EPS, rank)
    wq = mla.queries(q[:, extra:].reshape(n, heads, hd + 64), cos[pos], sin[pos], hd)
    got, gq = pool.cpu().numpy().astype(np.float64).reshape(-1, row), q_out.cpu().numpy().astype(np.float64)
    live = slots >= 0
    # half a step of f16; the norm's sum, root and products (rank + 8 roundings of f32 at most), the rotation's two products
    size = np.abs(want)
    x = np.abs(kv[:, extra:].astype(np.float64))
    turn = np.concatenate([x[:, rank:rank + 32] + x[:, rank + 32:]] * 2, -1)
    tol = mla.U * size + mla.TINY
    tol[:, :rank] += (rank + 8) * mla.E * size[:, :rank]
    tol[:, rank:] += 3 * mla.E * turn
    assert np.all(np.abs(got[slots[live]] - want[live]) <= tol[live])
    qx = np.abs(q[:, extra:].reshape(n, heads, hd + 64).astype(np.float64))
    qt = mla.U * np.abs(wq) + mla.TINY
    qt[..., hd:] += 3 * mla.E * np.concatenate([qx[..., hd:hd + 32] + qx[..., hd + 32:]] * 2, -1)
    assert np.all(np.abs(gq - wq)[live] <= qt[live])
    assert np.all(gq[~live] == 9.0)
    rest = np.setdiff1d(np.arange(blocks * 16), slots[live])
    assert np.all(got[rest] == 7.0)


def test_append_without_queries_and_no_rows():
    ql = lib()
    cos, sin = (dev(x) for x in tables(64))
    kv = torch.randn((3, 320), device="cuda")
    pool = torch.zeros((2, 16, 320), dtype=torch.float16, device="cuda")
    args = (torch.ones(256, device="cuda"), cos, sin)
    pos, slots = torch.tensor([0, 1, 63], dtype=torch.int32, device="cuda"), torch.tensor([31, 0, 5], device="cuda")
    ql.ql_mla_append(None, kv, *args, pos, slots, EPS, 4, 64, 256, 64, None, pool, 2, 64)
    assert int((pool.abs().sum(-1) > 0).sum()) == 3
    before = pool.clone()
    ql.ql_mla_append(None, kv[:0], *args, pos[:0], slots[:0], EPS, 4, 64, 256, 64, None, pool, 2, 64)
    assert torch.equal(pool, before)


@pytest.mark.parametrize("what", ["slot", "negative slot", "position", "negative position", "value", "nan", "squares"])
def test_append_bad_rows_are_recorded(what):
    ql = lib()
    cos, sin = (dev(x) for x in tables(64))
    kv = torch.randn((3, 320), device="cuda")
    q = torch.randn((3, 2, 128), device="cuda")
    pool = torch.zeros((2, 16, 320), dtype=torch.float16, device="cuda")
    q_out = torch.full((3, 2, 128), 9.0, dtype=torch.float16, device="cuda")
    pos, slots = torch.tensor([0, 1, 63], dtype=torch.int32, device="cuda"), torch.tensor([31, 0, 5], device="cuda")
    if what.endswith("slot"):
        slots[1] = 32 if what == "slot" else -2
    elif what.endswith("position"):
        pos[1] = 64 if what == "position" else -1
    else:
        kv[1, 7 if what == "squares" else 300] = 1e5 if what == "value" else 1e25 if what == "squares" else math.nan
    ql.ql_mla_append(q, kv, torch.ones(256, device="cuda"), cos, sin, pos, slots, EPS, 2, 64, 256, 64, q_out, pool, 2, 64)
    with pytest.raises(ql.QLError) as e:
        ql.ql_check_device_error()
    assert e.value.status == ql.QL_EDEVICE
    wrote = what in ("value", "nan", "squares")
    assert int((pool.abs().sum(-1) != 0).sum()) == (3 if wrote else 2)
    assert bool((q_out[1] == 9).all()) == (not wrote) and not bool((q_out[0] == 9).any())


# ---------------------------------------------------------------- inputs of the attention
def latent_case(lens, heads, hd, rank, rows=None, seed=0, size=1.5, extra_blocks=3, stale=None):
    """A paged cache whose blocks are scattered, with `stale` behind every sequence's end, and queries."""
    g = np.random.default_rng(seed)
    need = [(n + 15) // 16 for n in lens]
    maxb = max(max(need), 1)
    blocks = sum(need) + extra_blocks
    ids = g.permutation(blocks)
    pool = g.standard_normal((blocks, 16, rank + 64)).astype(np.float16)
    table = np.full((len(lens), maxb), -7, np.int32)      # entries that no key needs are never looked at
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
        if stale is not None and lens[b] % 16:
            pool[table[b, k - 1], lens[b] % 16:] = stale
    if stale is not None:
        pool[ids[at:]] = stale
    rows = len(lens) if rows is None else rows
    q = (size * g.standard_normal((rows, heads, hd + 64))).astype(np.float16)
    w = (g.standard_normal((heads, 2 * hd, rank)) / math.sqrt(rank)).astype(np.float16)
    return dict(pool=pool, table=table, q=q, w=w, lens=np.array(lens, np.int32), maxb=maxb, blocks=blocks, heads=heads, hd=hd, rank=rank,
                scale=1 / math.sqrt(hd + 64))


def rows_of(c, b, n):
    return c["pool"][c["table"][b, :(n + 15) // 16]].reshape(-1, c["rank"] + 64)[:n]


def decode(c, workspace=None, out=None, **over):
    ql = lib()
    c = {**c, **over}
    B = len(c["lens"])
    if workspace is None:
        workspace = torch.full((ql.ql_mla_decode_workspace_bytes(B, c["heads"], c["hd"], c["rank"], c["maxb"]),), 0xff, dtype=torch.uint8,
                               device="cuda")
    if out is None:
        out = torch.full((B, c["heads"], c["hd"]), 5.0, dtype=torch.float16, device="cuda")
    ql.ql_mla_attn_decode(dev(c["q"]), dev(c["w"]), dev(c["pool"]), dev(c["table"]), dev(c["lens"]), B, c["heads"], c["hd"], c["rank"], 64,
                          16, c["maxb"], c["blocks"], c["scale"], out, workspace)
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(np.float64)


def check_decode(c, got, skip=()):
    for b, n in enumerate(c["lens"]):
        if b in skip:
            continue
        if n == 0:
            assert np.all(got[b] == 5.0), b
            continue
        want, bound = mla.absorbed(c["q"][b], rows_of(c, b, n), c["w"], c["scale"])
        assert np.all(np.abs(got[b] - want) <= bound), (b, n, float(np.max(np.abs(got[b] - want) / bound)))


DECODE = [([1], 1, 64, 256), ([1], 32, 128, 512), ([16, 15, 17], 4, 64, 512), ([63, 64, 65, 0, 1, 128], 3, 128, 256),
          ([2048], 32, 128, 512), ([0, 0, 700, 0], 20, 64, 256), ([1000, 3, 129, 640], 33, 64, 512), ([200, 90], 64, 128, 512),
          ([333, 1, 77], 65, 64, 256), ([129], 96, 128, 512), ([40, 5], 1024, 64, 256), ([70, 4000], 100, 64, 512), ([12000], 8, 128, 512), ([500] * 40, 2, 64, 256)]


@pytest.mark.parametrize("lens,heads,hd,rank", DECODE)
def test_decode(lens, heads, hd, rank):
    c = latent_case(lens, heads, hd, rank, seed=len(lens) + heads, stale=np.nan)
    check_decode(c, decode(c))
    lib().ql_check_device_error()


@pytest.mark.parametrize("rank", [256, 512])
def test_decode_many_short_sequences(rank):
    lens = list(np.random.default_rng(5).integers(0, 70, 700))
    c = latent_case(lens, 3, 64, rank, stale=np.inf)
    check_decode(c, decode(c))


def test_decode_a_full_sequence_among_5000_empty_ones():
    """More sequences than a CTA has threads, most of them idle or of one token."""
    lens = np.zeros(5000, np.int64)
    lens[::371] = 1
    lens[4321] = 3000
    c = latent_case(list(lens), 2, 64, 256, seed=8, stale=np.nan)
    got = decode(c)
    assert np.all(got[lens == 0] == 5.0)
    check_decode(c, got, skip=set(np.flatnonzero(lens == 0)))


@pytest.mark.parametrize("order", ["rising", "falling", "one", "small", "large"])
def test_decode_scores(order):
    """Scores that rise along the context (each tile's largest far above the last one's), fall, hold one key that
    outweighs all, are nearly equal, or span hundreds."""
    c = latent_case([900, 333], 6, 128, 512, seed=3)
    pool, q = c["pool"], c["q"]
    if order in ("rising", "falling"):
        q[..., 128:] = 0
        q[..., 128] = 4.0
        for b, n in enumerate(c["lens"]):
            for t in range(n):
                pool[c["table"][b, t // 16], t % 16, 512] = (t if order == "rising" else n - t) * 0.5
    elif order == "one":
        for b, n in enumerate(c["lens"]):
            pool[c["table"][b, (n // 2) // 16], (n // 2) % 16, 512:] = np.sign(q[b, 0, 128:]) * 12
    elif order == "small":
        q *= np.float16(2.0 ** -10)
    else:
        q *= np.float16(20)
    check_decode(c, decode(c))


def test_decode_bad_blocks_and_lengths():
    ql = lib()
    c = latent_case([100, 300, 90, 50, 64], 5, 64, 256, seed=9)
    table = c["table"].copy()
    table[0, 2] = -1
    table[0, 6] = c["blocks"]
    table[1, :] = 1 << 30
    lens = c["lens"].copy()
    lens[2], lens[3] = c["maxb"] * 16 + 1, -4
    got = decode(c, table=table, lens=lens)
    with pytest.raises(ql.QLError) as e:
        ql.ql_check_device_error()
    assert e.value.status == ql.QL_EDEVICE
    assert np.all(got[1] == 0) and np.all(got[2:4] == 5.0)
    rows = rows_of(c, 0, 100)
    keep = np.concatenate([np.arange(0, 32), np.arange(48, 96)])
    want, bound = mla.absorbed(c["q"][0], rows[keep], c["w"], c["scale"])
    assert np.all(np.abs(got[0] - want) <= bound)
    want, bound = mla.absorbed(c["q"][4], rows_of(c, 4, 64), c["w"], c["scale"])
    assert np.all(np.abs(got[4] - want) <= bound)


def test_decode_absorbed_query_beyond_f16_is_recorded():
    ql = lib()
    c = latent_case([40, 30], 2, 64, 256)
    c["q"][0, 1, :64] = 0
    c["q"][1, 1, :64] = 6e4
    c["w"][1, :64, 7] = 6e4
    got = decode(c)
    with pytest.raises(ql.QLError):
        ql.ql_check_device_error()
    check_decode(c, got, skip=(1,))


def test_decode_one_workspace_for_calls_of_other_shapes_and_graphs():
    ql = lib()
    big = latent_case([700, 20, 300], 33, 128, 512, seed=1)
    small = latent_case([90, 5], 4, 64, 256, seed=2)
    ws = torch.full((ql.ql_mla_decode_workspace_bytes(3, 33, 128, 512, big["maxb"]),), 0xff, dtype=torch.uint8, device="cuda")
    for c in (big, small, big, small):
        check_decode(c, decode(c, workspace=ws))
    # a captured call serves other lengths, tables and queries at its replay
    a = {k: dev(big[k]) for k in ("q", "w", "pool", "table", "lens")}
    out = torch.full((3, 33, 128), 5.0, dtype=torch.float16, device="cuda")

    def call():
        ql.ql_mla_attn_decode(a["q"], a["w"], a["pool"], a["table"], a["lens"], 3, 33, 128, 512, 64, 16, big["maxb"], big["blocks"],
                              big["scale"], out, ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    torch.cuda.synchronize()
    other = {**big, "lens": np.array([3, 0, 290], np.int32), "q": big["q"][::-1].copy()}
    a["lens"].copy_(torch.from_numpy(other["lens"]))
    a["q"].copy_(torch.from_numpy(other["q"]))
    out.fill_(5.0)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    check_decode(other, out.cpu().numpy().astype(np.float64))
    first = out.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)      # the same bits from run to run


def test_decode_two_streams():
    ql = lib()
    cases = [latent_case([900, 30], 16, 64, 512, seed=1), latent_case([400, 77], 16, 64, 512, seed=2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    held, outs = [], []
    for c in cases:
        held.append([dev(c[k]) for k in ("q", "w", "pool", "table", "lens")]
                    + [torch.empty(ql.ql_mla_decode_workspace_bytes(2, 16, 64, 512, c["maxb"]), dtype=torch.uint8, device="cuda")])
        outs.append(torch.zeros((2, 16, 64), dtype=torch.float16, device="cuda"))
    torch.cuda.synchronize()
    for _ in range(5):
        for c, h, o, s in zip(cases, held, outs, streams):
            ql.ql_mla_attn_decode(*h[:5], 2, 16, 64, 512, 64, 16, c["maxb"], c["blocks"], c["scale"], o, h[5], stream=s)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        check_decode(c, o.cpu().numpy().astype(np.float64))


def test_decode_offsets_past_32_bits():
    """Blocks whose rows start beyond 2^32 bytes and 2^31 numbers of the pool."""
    ql = lib()
    heads, hd, rank, n = 3, 64, 512, 50
    blocks = (1 << 32) // (16 * 576) + 5
    c = latent_case([n], heads, hd, rank, seed=4)
    pool = torch.empty((blocks, 16, 576), dtype=torch.float16, device="cuda")
    ids = [blocks - 1, 3, blocks - 2, (1 << 31) // (16 * 576) + 1]
    for i, b in enumerate(ids):
        pool[b] = dev(c["pool"][c["table"][0, i]])
    out = torch.full((1, heads, hd), 5.0, dtype=torch.float16, device="cuda")
    ws = torch.empty(ql.ql_mla_decode_workspace_bytes(1, heads, hd, rank, 4), dtype=torch.uint8, device="cuda")
    ql.ql_mla_attn_decode(dev(c["q"]), dev(c["w"]), pool, torch.tensor([ids], dtype=torch.int32, device="cuda"), dev(c["lens"]), 1, heads, hd,
                          rank, 64, 16, 4, blocks, c["scale"], out, ws)
    torch.cuda.synchronize()
    check_decode(c, out.cpu().numpy().astype(np.float64))


# ---------------------------------------------------------------- chunk
def chunk(c, n, before, out=None, table=None, position=None):
    ql = lib()
    ws = torch.full((ql.ql_mla_chunk_workspace_bytes(n, c["heads"], c["hd"], c["rank"], c["maxb"]),), 0xff, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((n, c["heads"], c["hd"]), 5.0, dtype=torch.float16, device="cuda")
    position = torch.tensor([before if position is None else position], dtype=torch.int32, device="cuda")
    ql.ql_mla_attn_chunk(dev(c["q"]), dev(c["w"]), dev(c["pool"]), dev(c["table"] if table is None else table), position, n, c["heads"], c["hd"],
                         c["rank"], 64, 16, c["maxb"], c["blocks"], c["scale"], out, ws)
    torch.cuda.synchronize()
    return out.cpu().numpy().astype(np.float64)


def chunk_bound(c, n, before):
    """The oracle's answer and its bound for the form that the call takes: up to 32 tokens go through the absorbed one where
    that costs less."""
    rows = rows_of(c, 0, before + n)
    if n > 32 or (n * 128 > c["heads"] * c["hd"] and (c["maxb"] > 64 or n * c["heads"] > 512)):
        return mla.attention(c["q"], rows, c["w"], c["scale"], before=before)
    both = [mla.absorbed(c["q"][i], rows[:before + i + 1], c["w"], c["scale"]) for i in range(n)]
    return np.stack([x for x, _ in both]), np.stack([x for _, x in both])


CHUNK = [(256, 5000, 2, 64, 256), (300, 2500, 7, 64, 256), (700, 900, 13, 64, 256), (40, 9000, 1, 128, 256), (1030, 0, 11, 64, 256), (600, 600, 50, 64, 256),
         (17, 0, 4, 64, 256), (32, 900, 16, 64, 512), (17, 1100, 4, 64, 256), (30, 900, 18, 64, 512), (5, 300, 5, 128, 256), (6, 300, 5, 128, 256), (32, 1000, 64, 64, 512), (33, 1000, 64, 64, 512), (20, 0, 33, 128, 512),
         (32, 500, 96, 128, 256), (33, 500, 96, 128, 256), (1, 0, 1, 64, 256), (1, 0, 32, 128, 512), (17, 0, 4, 64, 256), (16, 1, 2, 128, 512), (128, 0, 3, 128, 256), (129, 0, 2, 64, 512),
         (1, 700, 5, 128, 512), (7, 121, 3, 64, 256), (100, 1000, 2, 128, 512), (300, 333, 7, 64, 256), (513, 0, 2, 128, 512),
         (64, 2500, 1, 64, 512), (200, 57, 33, 64, 256), (40, 3, 70, 64, 512)]


@pytest.mark.parametrize("n,before,heads,hd,rank", CHUNK)
def test_chunk(n, before, heads, hd, rank):
    c = latent_case([before + n], heads, hd, rank, rows=n, seed=n + heads, stale=np.nan)
    got = chunk(c, n, before)
    want, bound = chunk_bound(c, n, before)
    assert np.all(np.abs(got - want) <= bound), float(np.max(np.abs(got - want) / bound))
    lib().ql_check_device_error()


def test_chunk_in_a_longer_table():
    """The table is far longer than the context: its other entries are never looked at."""
    c = latent_case([150], 4, 64, 512, rows=60, stale=np.inf)
    c["table"] = np.concatenate([c["table"], np.full((1, 300), 1 << 29, np.int32)], 1)
    c["maxb"] += 300
    got = chunk(c, 60, 90)
    want, bound = mla.attention(c["q"], rows_of(c, 0, 150), c["w"], c["scale"], before=90)
    assert np.all(np.abs(got - want) <= bound)
    lib().ql_check_device_error()


@pytest.mark.parametrize("order", ["rising", "falling", "large"])
def test_chunk_scores(order):
    n, before = 200, 400
    c = latent_case([n + before], 3, 128, 256, rows=n, seed=3)
    if order == "large":
        c["q"] *= np.float16(20)
    else:
        c["q"][..., 128:] = 0
        c["q"][..., 128] = 4.0
        for t in range(n + before):
            c["pool"][c["table"][0, t // 16], t % 16, 256] = (t if order == "rising" else n + before - t) * 0.5
    got = chunk(c, n, before)
    want, bound = mla.attention(c["q"], rows_of(c, 0, before + n), c["w"], c["scale"], before=before)
    assert np.all(np.abs(got - want) <= bound)


@pytest.mark.parametrize("heads", [3, 90])
def test_chunk_bad_blocks_and_positions(heads):
    """(The second in the absorbed form: 24 tokens are few for 90 heads of 128.)"""
    ql = lib()
    n, before = 40 if heads == 3 else 24, 100
    c = latent_case([n + before], heads, 64 if heads == 3 else 128, 256, rows=n, seed=5)
    table = c["table"].copy()
    table[0, 1], table[0, 7] = c["blocks"], -3
    got = chunk(c, n, before, table=table)
    with pytest.raises(ql.QLError):
        ql.ql_check_device_error()
    rows = rows_of(c, 0, n + before).astype(np.float64)
    keep = np.concatenate([np.arange(16), np.arange(32, 112), np.arange(128, 140)])
    for i in range(n):
        some = keep[keep <= before + i]
        want, bound = mla.attention(c["q"][i:i + 1], rows[some], c["w"], c["scale"]) if heads == 3 else mla.absorbed(
            c["q"][i], rows[some], c["w"], c["scale"])
        assert np.all(np.abs(got[i] - want.reshape(got[i].shape)) <= bound.reshape(got[i].shape))
    # the first queries see only keys of a bad block
    table = c["table"].copy()
    table[0, 0] = -1
    got = chunk(c, n, before, table=table, position=0)
    with pytest.raises(ql.QLError):
        ql.ql_check_device_error()
    assert np.all(got[:16] == 0) and np.all(np.abs(got[16:]).sum(-1) > 0)
    for bad in (-1, c["maxb"] * 16 - n + 1):
        assert np.all(chunk(c, n, before, position=bad) == 5.0)
        with pytest.raises(ql.QLError):
            ql.ql_check_device_error()


@pytest.mark.parametrize("n,before,heads,hd,rank", [(300, 50, 3, 64, 256), (300, 50, 3, 128, 512), (600, 0, 5, 64, 512), (129, 700, 2, 128, 256),
                                                    (20, 100, 32, 128, 512)])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", ["latent", "rotated"])
def test_chunk_broken_rows_stay_behind_the_mask(n, before, heads, hd, rank, value, at):
    """A token whose cache row holds NaN or an infinity is seen by the queries from it on, and by none before it."""
    c = latent_case([before + n], heads, hd, rank, rows=n, seed=n + heads)
    broken = n - n // 3
    row = before + broken
    c["pool"][c["table"][0, row // 16], row % 16, rank - 7 if at == "latent" else rank + 5] = value
    got = chunk(c, n, before)
    if at == "latent" or math.isnan(value):
        assert not np.any(np.isfinite(got[broken:]))
    sound = dict(c, q=c["q"][:broken])
    lens = before + broken
    rows = rows_of(c, 0, lens)
    if n > 32:
        want, bound = mla.attention(sound["q"], rows, c["w"], c["scale"], before=before)
    else:
        both = [mla.absorbed(c["q"][i], rows[:before + i + 1], c["w"], c["scale"]) for i in range(broken)]
        want, bound = np.stack([x for x, _ in both]), np.stack([x for _, x in both])
    assert np.all(np.abs(got[:broken] - want) <= bound)
    lib()


@pytest.mark.parametrize("hd,rank", [(64, 256), (128, 512)])
def test_chunk_keys_beyond_f16_are_recorded(hd, rank):
    ql = lib()
    c = latent_case([90], 3, hd, rank, rows=90, seed=4)
    c["w"][1, 3] = 300.0       # a key row of the second head
    c["pool"][:, :, :rank] = 1.0
    chunk(c, 90, 0)
    with pytest.raises(ql.QLError):
        ql.ql_check_device_error()
    c["w"][1, 3] = 0.0
    chunk(c, 90, 0)
    ql.ql_check_device_error()


def test_chunk_offsets_past_32_bits():
    """Keys and values of the last heads start beyond 2^32 bytes of the workspace, blocks of the cache beyond 2^32 bytes of the pool."""
    ql = lib()
    n, before, heads, hd, rank, maxb = 70, 30, 20, 128, 512, 1 << 16
    blocks = (1 << 32) // (16 * 576) + 5
    c = latent_case([before + n], heads, hd, rank, rows=n, seed=6)
    pool = torch.empty((blocks, 16, 576), dtype=torch.float16, device="cuda")
    ids = [blocks - 1, 3, blocks - 2, (1 << 31) // (16 * 576) + 1, 0, 7, blocks - 3]
    for i, b in enumerate(ids):
        pool[b] = dev(c["pool"][c["table"][0, i]])
    table = torch.full((maxb,), -1, dtype=torch.int32, device="cuda")
    table[:len(ids)] = torch.tensor(ids, dtype=torch.int32)
    out = torch.full((n, heads, hd), 5.0, dtype=torch.float16, device="cuda")
    ws = torch.empty(ql.ql_mla_chunk_workspace_bytes(n, heads, hd, rank, maxb), dtype=torch.uint8, device="cuda")
    assert heads * maxb * 16 * hd * 2 > 1 << 32
    ql.ql_mla_attn_chunk(dev(c["q"]), dev(c["w"]), pool, table, torch.tensor([before], dtype=torch.int32, device="cuda"), n, heads, hd, rank, 64, 16,
                         maxb, blocks, c["scale"], out, ws)
    torch.cuda.synchronize()
    want, bound = mla.attention(c["q"], rows_of(c, 0, before + n), c["w"], c["scale"], before=before)
    assert np.all(np.abs(out.cpu().numpy().astype(np.float64) - want) <= bound)
    ql.ql_check_device_error()


@pytest.mark.parametrize("n,before", [(3, 37), (40, 0), (260, 20)])
def test_chunk_1024_heads(n, before):
    c = latent_case([before + n], 1024, 64, 256, rows=n, seed=n)
    got = chunk(c, n, before)
    for heads in (slice(0, 3), slice(510, 514), slice(1020, 1024)):
        part = dict(c, q=c["q"][:, heads], w=c["w"][heads])
        rows = rows_of(c, 0, before + n)
        if n > 32:
            want, bound = mla.attention(part["q"], rows, part["w"], c["scale"], before=before)
        else:
            both = [mla.absorbed(part["q"][i], rows[:before + i + 1], part["w"], c["scale"]) for i in range(n)]
            want, bound = np.stack([x for x, _ in both]), np.stack([x for _, x in both])
        assert np.all(np.abs(got[:, heads] - want) <= bound)
    lib().ql_check_device_error()


@pytest.mark.parametrize("what,sizes", [("decode", ([3000, 1, 700, 64], 32, 128, 512)), ("decode", ([900, 5000], 70, 64, 256)),
                                        ("chunk", (200, 3000, 4, 128, 512)), ("chunk", (30, 2000, 32, 128, 256)), ("chunk", (600, 100, 6, 64, 512))])
def test_repeats_are_bit_identical(what, sizes):
    if what == "decode":
        c = latent_case(*sizes, seed=3)
        runs = [decode(c) for _ in range(4)]
    else:
        n, before, heads, hd, rank = sizes
        c = latent_case([before + n], heads, hd, rank, rows=n, seed=3)
        runs = [chunk(c, n, before) for _ in range(4)]
    assert all(np.array_equal(runs[0], r) for r in runs[1:])


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("graph", [False, True])
def test_steps_without_a_pause(graph):
    """60 steps of three sequences issued one after the other: each step's rows, slots, lengths and table entries are written on the
    stream right before the kernels that read them, while the kernels of the step before may still run."""
    ql = lib()
    heads, hd, rank, B, steps, start = 9, 64, 256, 3, 60, (1, 250, 63)
    g = np.random.default_rng(11)
    cos, sin = (dev(x) for x in tables(512))
    w = (g.standard_normal((heads, 2 * hd, rank)) / math.sqrt(rank)).astype(np.float16)
    maxb, blocks = 20, 70
    ids = g.permutation(blocks)[:B * maxb].reshape(B, maxb).astype(np.int32)
    pool = torch.full((blocks, 16, rank + 64), math.nan, dtype=torch.float16, device="cuda")
    first = [g.standard_normal((n, rank + 64)).astype(np.float16) for n in start]
    for b in range(B):
        for t in range(start[b]):
            pool[int(ids[b, t // 16]), t % 16] = dev(first[b][t])
    whole = dev(ids)
    table = torch.full((B, maxb), -1, dtype=torch.int32, device="cuda")
    lens = dev(np.array(start, np.int32))
    q = dev(g.standard_normal((steps, B, heads, hd + 64)).astype(np.float32))
    kv = dev(g.standard_normal((steps, B, rank + 64)).astype(np.float32))
    at = torch.zeros(1, dtype=torch.int64, device="cuda")
    norm, wd = torch.ones(rank, device="cuda"), dev(w)
    q_out = torch.zeros((B, heads, hd + 64), dtype=torch.float16, device="cuda")
    out = torch.zeros((B, heads, hd), dtype=torch.float16, device="cuda")
    ws = torch.empty(ql.ql_mla_decode_workspace_bytes(B, heads, hd, rank, maxb), dtype=torch.uint8, device="cuda")
    outs, qs = torch.zeros((steps, *out.shape), dtype=torch.float16, device="cuda"), torch.zeros((steps, *q_out.shape), dtype=torch.float16, device="cuda")
    blk = torch.arange(maxb, device="cuda")

    def step():
        pos = lens.clone()
        slots = whole.gather(1, (pos // 16).long()[:, None])[:, 0].long() * 16 + pos % 16
        table.copy_(torch.where(blk[None] <= (pos // 16)[:, None], whole, torch.full_like(whole, -1)))
        ql.ql_mla_append(q.index_select(0, at)[0], kv.index_select(0, at)[0], norm, cos, sin, pos, slots, EPS, heads, hd, rank, 64, q_out, pool,
                         blocks, 512)
        lens.add_(1)
        ql.ql_mla_attn_decode(q_out, wd, pool, table, lens, B, heads, hd, rank, 64, 16, maxb, blocks, 0.1, out, ws)
        outs.index_copy_(0, at, out[None])
        qs.index_copy_(0, at, q_out[None])
        at.add_(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        if graph:
            keep = (lens.clone(), at.clone(), pool.clone())
            step()
            for t, k in zip((lens, at, pool), keep):
                t.copy_(k)
            torch.cuda.synchronize()
            recorded = torch.cuda.CUDAGraph()
            with torch.cuda.graph(recorded, stream=s):
                step()
            for _ in range(steps):
                recorded.replay()
        else:
            for _ in range(steps):
                step()
    torch.cuda.synchronize()
    ql.ql_check_device_error()
    rows = pool.cpu().numpy()
    got, qn = outs.cpu().numpy().astype(np.float64), qs.cpu().numpy()
    for b in range(B):
        seq = rows[ids[b]].reshape(-1, rank + 64)
        assert np.array_equal(seq[:start[b]], first[b])
        for i in range(0, steps, 7):
            want, bound = mla.absorbed(qn[i, b], seq[:start[b] + i + 1], w, 0.1)
            assert np.all(np.abs(got[i, b] - want) <= bound), (b, i)


@pytest.mark.parametrize("heads,hd,rank", [(6, 64, 256), (34, 128, 512)])
def test_prompt_then_tokens(heads, hd, rank):
    """Two sequences: a prompt in two chunks each, then single tokens of both, each step's rows appended by the operator
    before they are attended to; the last steps replayed from one captured graph."""
    ql = lib()
    g = np.random.default_rng(heads)
    cos, sin = tables(512)
    cosd, sind = dev(cos), dev(sin)
    w = (g.standard_normal((heads, 2 * hd, rank)) / math.sqrt(rank)).astype(np.float16)
    norm = (1 + 0.1 * g.standard_normal(rank)).astype(np.float32)
    wd, nd = dev(w), dev(norm)
    maxb, blocks, scale = 16, 40, 1 / math.sqrt(hd + 64)
    ids = g.permutation(blocks)[:2 * maxb].reshape(2, maxb).astype(np.int32)
    table = dev(ids)
    pool = torch.full((blocks, 16, rank + 64), math.nan, dtype=torch.float16, device="cuda")
    held = [np.zeros((0, rank + 64), np.float16) for _ in range(2)]

    def slots(b, pos):
        return ids[b, pos // 16].astype(np.int64) * 16 + pos % 16

    def appended(q, kv, pos, want_rows):
        wq = mla.queries(q, cos[pos], sin[pos], hd)
        assert np.all(np.abs(want_rows.astype(np.float64) - mla.append(kv, norm, cos[pos], sin[pos], EPS, rank)) <= 4e-3 * (1 + np.abs(want_rows)))
        return wq
    for b, parts in enumerate([(70, 33), (128, 5)]):
        at = 0
        for n in parts:
            q = g.standard_normal((n, heads, hd + 64)).astype(np.float32)
            kv = g.standard_normal((n, rank + 64)).astype(np.float32)
            pos = np.arange(at, at + n).astype(np.int32)
            q_out = torch.zeros((n, heads, hd + 64), dtype=torch.float16, device="cuda")
            sl = slots(b, pos)
            ql.ql_mla_append(dev(q), dev(kv), nd, cosd, sind, dev(pos), dev(sl), EPS, heads, hd, rank, 64, q_out, pool, blocks, 512)
            out = torch.zeros((n, heads, hd), dtype=torch.float16, device="cuda")
            ws = torch.empty(ql.ql_mla_chunk_workspace_bytes(n, heads, hd, rank, maxb), dtype=torch.uint8, device="cuda")
            ql.ql_mla_attn_chunk(q_out, wd, pool, table[b:b + 1], dev(np.array([at], np.int32)), n, heads, hd, rank, 64, 16, maxb, blocks, scale,
                                 out, ws)
            torch.cuda.synchronize()
            new = pool.reshape(-1, rank + 64)[dev(sl)].cpu().numpy()
            appended(q, kv, pos, new)
            held[b] = np.concatenate([held[b], new])
            c = dict(q=q_out.cpu().numpy(), w=w, scale=scale, heads=heads, hd=hd, rank=rank, maxb=maxb, pool=pool.cpu().numpy(), table=ids[b:b + 1])
            want, bound = chunk_bound(c, n, at)
            assert np.all(np.abs(out.cpu().numpy() - want) <= bound)
            at += n
    ws = torch.empty(ql.ql_mla_decode_workspace_bytes(2, heads, hd, rank, maxb), dtype=torch.uint8, device="cuda")
    q, kv = torch.zeros((2, heads, hd + 64), device="cuda"), torch.zeros((2, rank + 64), device="cuda")
    pos, sl = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    q_out = torch.zeros((2, heads, hd + 64), dtype=torch.float16, device="cuda")
    out = torch.zeros((2, heads, hd), dtype=torch.float16, device="cuda")

    def step():
        ql.ql_mla_append(q, kv, nd, cosd, sind, pos, sl, EPS, heads, hd, rank, 64, q_out, pool, blocks, 512)
        ql.ql_mla_attn_decode(q_out, wd, pool, table, lens, 2, heads, hd, rank, 64, 16, maxb, blocks, scale, out, ws)
    graph = None
    for i in range(6):
        at = np.array([len(h) for h in held])
        q.copy_(torch.from_numpy(g.standard_normal((2, heads, hd + 64)).astype(np.float32)))
        kv.copy_(torch.from_numpy(g.standard_normal((2, rank + 64)).astype(np.float32)))
        pos.copy_(torch.from_numpy(at.astype(np.int32)))
        where = np.array([slots(b, at[b]) for b in range(2)])
        sl.copy_(torch.from_numpy(where))
        lens.copy_(torch.from_numpy((at + 1).astype(np.int32)))
        if i == 3:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                step()
        graph.replay() if graph is not None else step()
        torch.cuda.synchronize()
        new = pool.reshape(-1, rank + 64)[sl].cpu().numpy()
        for b in range(2):
            held[b] = np.concatenate([held[b], new[b:b + 1]])
            want, bound = mla.absorbed(q_out[b].cpu().numpy(), held[b], w, scale)
            assert np.all(np.abs(out[b].cpu().numpy() - want) <= bound)
    ql.ql_check_device_error()
