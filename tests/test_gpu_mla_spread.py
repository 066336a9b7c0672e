"""Latent attention at lengths where the elementwise bounds grow past the answer: the root mean square of the error against the spread that
the roundings leave (``oracle/mla.py``; ``test_oracle_mla_spread.py`` pins that a key, a tile or the low half of a pair that is left out lies
outside). 64 and more keys a query: with fewer the roundings are few, and the bounds of ``test_gpu_mla.py`` are sharp."""
import math

import numpy as np
import pytest
import torch

from gpu_util import dev, lib
from oracle import mla
from test_gpu_mla import EPS, chunk, decode, latent_case, rows_of, tables
from test_oracle_mla_spread import HEAD, WHOLE

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def record():
    """Each test starts with an empty device error record and leaves none."""
    ql = lib()
    try:
        ql.ql_check_device_error()
    except ql.QLError:
        pass
    yield
    ql.ql_check_device_error()


def check(got, want, var):
    whole, head = mla.off(got, want, var)
    assert whole <= WHOLE and head <= HEAD, (whole, head)


def check_decode(c, got, skip=()):
    """All sequences of 64 keys and more together, and each head of each."""
    pair = c["heads"] <= 32
    some = [b for b, n in enumerate(c["lens"]) if n >= 64 and b not in skip]
    to = [mla.absorbed_spread(c["q"][b], rows_of(c, b, c["lens"][b]), c["w"], c["scale"], pair) for b in some]
    check(got[some], np.stack([x for x, _ in to]), np.stack([x for _, x in to]))


def chunk_spread(c, n, before):
    """Of the form that the call takes."""
    rows = rows_of(c, 0, before + n)
    if n > 32 or (n * 128 > c["heads"] * c["hd"] and (c["maxb"] > 64 or n * c["heads"] > 512)):
        return mla.attention_spread(c["q"], rows, c["w"], c["scale"], before)
    both = [mla.absorbed_spread(c["q"][i], rows[:before + i + 1], c["w"], c["scale"], c["heads"] <= 32) for i in range(n)]
    return np.stack([x for x, _ in both]), np.stack([x for _, x in both])


@pytest.mark.parametrize("lens,heads,hd,rank", [
    ([2048], 32, 128, 512), ([12000], 8, 128, 512), ([0, 700, 0, 64], 20, 64, 256), ([1000, 3, 129, 640], 33, 64, 512), ([200, 90], 64, 128, 512),
    ([333, 1, 77], 65, 64, 256), ([70, 4000], 100, 64, 512), ([500] * 40, 8, 64, 256), ([2000, 100, 3000], 16, 128, 512), ([700, 70], 128, 128, 512),
    ([3000, 2999, 3001, 64, 65], 5, 128, 256), ([9000] + [64] * 70, 7, 64, 256)])
def test_decode(lens, heads, hd, rank):
    c = latent_case(lens, heads, hd, rank, seed=len(lens) + heads, stale=np.nan)
    check_decode(c, decode(c))


def test_decode_many_sequences():
    lens = list(np.random.default_rng(5).integers(0, 400, 300))
    c = latent_case(lens, 8, 64, 256, stale=np.inf)
    check_decode(c, decode(c))


def test_decode_small_scores():
    c = latent_case([900, 333], 8, 128, 512, seed=3)
    c["q"] *= np.float16(2.0 ** -6)
    check_decode(c, decode(c))


def test_decode_bad_blocks():
    """The keys of blocks outside the pool, and no others, are left out of a long context."""
    ql = lib()
    c = latent_case([3000, 2000], 8, 128, 512, seed=9)
    table = c["table"].copy()
    bad = [3, 60, 61, 62, 63, 187]
    table[0, bad] = [-1, c["blocks"], 1 << 30, -5, c["blocks"] + 7, -1 << 31]
    got = decode(c, table=table)
    with pytest.raises(ql.QLError):
        ql.ql_check_device_error()
    keep = ~np.isin(np.arange(3000) // 16, bad)
    check(got[:1], *(x[None] for x in mla.absorbed_spread(c["q"][0], rows_of(c, 0, 3000)[keep], c["w"], c["scale"], True)))
    check_decode(c, got, skip=(0,))


def test_decode_graph_and_streams():
    """One captured call at other lengths and queries at each replay, beside calls on another stream with a workspace of their own."""
    ql = lib()
    c, other = latent_case([2500, 100, 1800], 33, 128, 512, seed=1), latent_case([1500, 3000], 16, 64, 512, seed=2)
    a = {k: dev(c[k]) for k in ("q", "w", "pool", "table", "lens")}
    held = [dev(other[k]) for k in ("q", "w", "pool", "table", "lens")]
    ws = torch.full((ql.ql_mla_decode_workspace_bytes(3, 33, 128, 512, c["maxb"]),), 0xff, dtype=torch.uint8, device="cuda")
    ws2 = torch.full((ql.ql_mla_decode_workspace_bytes(2, 16, 64, 512, other["maxb"]),), 0xff, dtype=torch.uint8, device="cuda")
    out, out2 = torch.zeros((3, 33, 128), dtype=torch.float16, device="cuda"), torch.zeros((2, 16, 64), dtype=torch.float16, device="cuda")

    def call():
        ql.ql_mla_attn_decode(a["q"], a["w"], a["pool"], a["table"], a["lens"], 3, 33, 128, 512, 64, 16, c["maxb"], c["blocks"], c["scale"], out, ws)
    s, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
    torch.cuda.synchronize()
    for lens, turn in (([2500, 100, 1800], 0), ([777, 2000, 64], 1), ([65, 1600, 1799], 2)):
        now = {**c, "lens": np.minimum(lens, c["lens"]).astype(np.int32), "q": np.roll(c["q"], turn, 0)}
        a["lens"].copy_(torch.from_numpy(now["lens"]))
        a["q"].copy_(torch.from_numpy(now["q"]))
        torch.cuda.synchronize()
        for _ in range(3):
            with torch.cuda.stream(s):
                graph.replay()
            ql.ql_mla_attn_decode(*held, 2, 16, 64, 512, 64, 16, other["maxb"], other["blocks"], other["scale"], out2, ws2, stream=s2)
        torch.cuda.synchronize()
        check_decode(now, out.cpu().numpy())
        check_decode(other, out2.cpu().numpy())


@pytest.mark.parametrize("n,before,heads,hd,rank", [
    (256, 5000, 2, 64, 256), (300, 2500, 7, 64, 256), (40, 9000, 1, 128, 256), (1030, 100, 11, 64, 256), (100, 1000, 2, 128, 512), (300, 333, 7, 64, 256),
    (513, 64, 2, 128, 512), (64, 2500, 1, 64, 512), (200, 70, 33, 64, 256), (33, 500, 96, 128, 256), (600, 600, 50, 64, 256), (17, 1100, 4, 64, 256),
    (32, 500, 96, 128, 256), (1, 700, 8, 128, 512), (8, 4000, 32, 128, 512), (30, 900, 18, 64, 512), (32, 900, 16, 64, 512), (20, 100, 33, 128, 512)])
def test_chunk(n, before, heads, hd, rank):
    c = latent_case([before + n], heads, hd, rank, rows=n, seed=n + heads, stale=np.nan)
    check(chunk(c, n, before), *chunk_spread(c, n, before))


@pytest.mark.parametrize("heads,hd,rank", [(8, 64, 256), (34, 128, 512)])
def test_prompt_then_tokens(heads, hd, rank):
    """Two sequences: a prompt in two chunks each, then tokens of both one after the other without a pause, from one captured graph; each
    step's rows appended by the operator right before they are attended to."""
    ql = lib()
    g = np.random.default_rng(heads)
    cosd, sind = (dev(x) for x in tables(2048))
    w = (g.standard_normal((heads, 2 * hd, rank)) / math.sqrt(rank)).astype(np.float16)
    wd, norm = dev(w), torch.ones(rank, device="cuda")
    maxb, blocks, scale, steps = 96, 230, 1 / math.sqrt(hd + 64), 48
    ids = g.permutation(blocks)[:2 * maxb].reshape(2, maxb).astype(np.int32)
    table = dev(ids)
    pool = torch.full((blocks, 16, rank + 64), math.nan, dtype=torch.float16, device="cuda")
    flat = pool.reshape(-1, rank + 64)

    def rows(b, n):
        t = np.arange(n)
        return flat[dev(ids[b, t // 16].astype(np.int64) * 16 + t % 16)].cpu().numpy()
    parts, at = [(900, 133), (70, 630)], [0, 0]
    for b in range(2):
        for n in parts[b]:
            pos = np.arange(at[b], at[b] + n)
            q_out = torch.zeros((n, heads, hd + 64), dtype=torch.float16, device="cuda")
            q, kv = torch.randn((n, heads, hd + 64), device="cuda"), torch.randn((n, rank + 64), device="cuda")
            ql.ql_mla_append(q, kv, norm, cosd, sind, dev(pos.astype(np.int32)), dev(ids[b, pos // 16].astype(np.int64) * 16 + pos % 16), EPS, heads, hd,
                             rank, 64, q_out, pool, blocks, 2048)
            out = torch.zeros((n, heads, hd), dtype=torch.float16, device="cuda")
            ws = torch.empty(ql.ql_mla_chunk_workspace_bytes(n, heads, hd, rank, maxb), dtype=torch.uint8, device="cuda")
            ql.ql_mla_attn_chunk(q_out, wd, pool, table[b:b + 1], dev(np.array([at[b]], np.int32)), n, heads, hd, rank, 64, 16, maxb, blocks, scale, out, ws)
            torch.cuda.synchronize()
            late = slice(max(0, 64 - at[b]), None)
            if at[b] + n > 64:
                check(out.cpu().numpy()[late], *(x[late] for x in mla.attention_spread(q_out.cpu().numpy(), rows(b, at[b] + n), w, scale, at[b])))
            at[b] += n
    lens = dev(np.array(at, np.int32))
    q, kv = torch.randn((steps, 2, heads, hd + 64), device="cuda"), torch.randn((steps, 2, rank + 64), device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    q_out = torch.zeros((2, heads, hd + 64), dtype=torch.float16, device="cuda")
    out = torch.zeros((2, heads, hd), dtype=torch.float16, device="cuda")
    outs, qs = torch.zeros((steps, *out.shape), dtype=torch.float16, device="cuda"), torch.zeros((steps, *q_out.shape), dtype=torch.float16, device="cuda")
    ws = torch.empty(ql.ql_mla_decode_workspace_bytes(2, heads, hd, rank, maxb), dtype=torch.uint8, device="cuda")

    def token():
        pos = lens.clone()
        slots = table.gather(1, (pos // 16).long()[:, None])[:, 0].long() * 16 + pos % 16
        ql.ql_mla_append(q.index_select(0, step)[0], kv.index_select(0, step)[0], norm, cosd, sind, pos, slots, EPS, heads, hd, rank, 64, q_out, pool,
                         blocks, 2048)
        lens.add_(1)
        ql.ql_mla_attn_decode(q_out, wd, pool, table, lens, 2, heads, hd, rank, 64, 16, maxb, blocks, scale, out, ws)
        outs.index_copy_(0, step, out[None])
        qs.index_copy_(0, step, q_out[None])
        step.add_(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        token()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            token()
        for _ in range(steps - 1):
            graph.replay()
    torch.cuda.synchronize()
    got, qn = outs.cpu().numpy(), qs.cpu().numpy()
    for b in range(2):
        seq = rows(b, at[b] + steps)
        for i in range(0, steps, 5):
            check(got[i, b][None], *(x[None] for x in mla.absorbed_spread(qn[i, b], seq[:at[b] + i + 1], w, scale, heads <= 32)))
