"""Latent attention at the ends of its documented ranges: most sequences, most heads, longest chunks and tables. Samples of the outputs against
64 bits on the GPU, by the root mean square of a head's error, of which 0.002 is allowed: four half steps of f16, as for a few keys the roundings of
query, keys, weights and output may all go one way. Another sequence's or token's rows give another answer altogether."""
import math

import pytest
import torch

from gpu_util import lib

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def record():
    ql = lib()
    try:
        ql.ql_check_device_error()
    except ql.QLError:
        pass
    yield
    ql.ql_check_device_error()
    torch.cuda.empty_cache()


def rand(g, *shape):
    return torch.randn(shape, device="cuda", generator=g).half()


def exact(q, rows, w, scale):
    """One query's head [hd + 64] over rows [L, rank + 64], w [2 hd, rank]."""
    hd, c = q.numel() - 64, rows[:, :-64].double()
    kv = c @ w.double().T
    s = (kv[:, :hd] @ q[:hd].double() + rows[:, -64:].double() @ q[hd:].double()) * scale
    return torch.softmax(s, 0) @ kv[:, hd:]


def near(got, want):
    e = float((got.double() - want).norm() / want.norm())
    assert e < 2e-3, e


@pytest.mark.parametrize("batch,heads,hd,rank,longest", [(65535, 1, 64, 256, 40), (65535, 3, 64, 512, 3), (4096, 1000, 64, 256, 33), (4095, 1024, 128, 512, 2)])
def test_most_sequences_and_heads(batch, heads, hd, rank, longest):
    ql = lib()
    g = torch.Generator(device="cuda").manual_seed(batch)
    maxb, blocks, scale = (longest + 15) // 16, 5000, 1 / math.sqrt(hd + 64)
    pool, w, q = rand(g, blocks, 16, rank + 64), rand(g, heads, 2 * hd, rank) / math.sqrt(rank), rand(g, batch, heads, hd + 64)
    table = torch.randint(0, blocks, (batch, maxb), device="cuda", generator=g, dtype=torch.int32)
    lens = torch.randint(0, longest + 1, (batch,), device="cuda", generator=g, dtype=torch.int32)
    lens[-1] = longest
    out = torch.full((batch, heads, hd), 5.0, dtype=torch.float16, device="cuda")
    ws = torch.empty(ql.ql_mla_decode_workspace_bytes(batch, heads, hd, rank, maxb), dtype=torch.uint8, device="cuda")
    ql.ql_mla_attn_decode(q, w, pool, table, lens, batch, heads, hd, rank, 64, 16, maxb, blocks, scale, out, ws)
    idle = lens == 0
    assert bool((out[idle] == 5).all()) and not bool((out[~idle] == 5).all(-1).any())
    for b in (0, 1, 63, 64, batch // 2, batch - 2, batch - 1):
        n = int(lens[b])
        if n:
            rows = pool[table[b].long()].reshape(-1, rank + 64)[:n]
            for h in {0, heads // 2, heads - 1}:
                near(out[b, h], exact(q[b, h], rows, w[h], scale))


@pytest.mark.parametrize("n,before,heads,hd,rank,maxb", [(65535, 1, 2, 64, 256, 4096), (65535, 100, 1, 128, 512, 1 << 16), (4095, 0, 1024, 64, 256, 256), (40, (1 << 20) - 40, 1, 64, 256, 1 << 16),
                                                         (1, (1 << 20) - 1, 64, 128, 512, 1 << 16), (300, (1 << 20) - 300, 2, 128, 256, 1 << 16)])
def test_longest_chunks_and_tables(n, before, heads, hd, rank, maxb):
    """(Blocks of the longest contexts are repeated by the table.)"""
    ql = lib()
    g = torch.Generator(device="cuda").manual_seed(n)
    need, scale = (n + before + 15) // 16, 1 / math.sqrt(hd + 64)
    blocks = min(need, 5000)
    pool, w, q = rand(g, blocks, 16, rank + 64), rand(g, heads, 2 * hd, rank) / math.sqrt(rank), rand(g, n, heads, hd + 64)
    table = torch.full((maxb,), -1, dtype=torch.int32, device="cuda")
    table[:need] = torch.randint(0, blocks, (need,), device="cuda", generator=g, dtype=torch.int32)
    out = torch.full((n, heads, hd), 5.0, dtype=torch.float16, device="cuda")
    ws = torch.empty(ql.ql_mla_chunk_workspace_bytes(n, heads, hd, rank, maxb), dtype=torch.uint8, device="cuda")
    ql.ql_mla_attn_chunk(q, w, pool, table, torch.tensor([before], dtype=torch.int32, device="cuda"), n, heads, hd, rank, 64, 16, maxb, blocks, scale, out, ws)
    assert not bool((out == 5).all(-1).any())
    for i in sorted({0, 1, n // 3, n // 2, n - 1} & set(range(n))):
        rows = pool[table[:need].long()].reshape(-1, rank + 64)[:before + i + 1]
        for h in {0, heads - 1}:
            near(out[i, h], exact(q[i, h], rows, w[h], scale))


@pytest.mark.parametrize("lens,heads,hd,rank", [([(1 << 24) - 5, 3], 1, 64, 256), ([3, 1 << 20, 0, 1 << 20], 40, 128, 512)])
def test_longest_sequences(lens, heads, hd, rank):
    """A table of 2^20 blocks, and sequences cut over all windows."""
    ql = lib()
    g = torch.Generator(device="cuda").manual_seed(1)
    blocks, scale, batch = 5000, 1 / math.sqrt(hd + 64), len(lens)
    maxb = (max(lens) + 15) // 16
    pool, w, q = rand(g, blocks, 16, rank + 64), rand(g, heads, 2 * hd, rank) / math.sqrt(rank), rand(g, batch, heads, hd + 64)
    table = torch.randint(0, blocks, (batch, maxb), device="cuda", generator=g, dtype=torch.int32)
    out = torch.full((batch, heads, hd), 5.0, dtype=torch.float16, device="cuda")
    ws = torch.empty(ql.ql_mla_decode_workspace_bytes(batch, heads, hd, rank, maxb), dtype=torch.uint8, device="cuda")
    ql.ql_mla_attn_decode(q, w, pool, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), batch, heads, hd, rank, 64, 16, maxb, blocks, scale, out, ws)
    for b, n in enumerate(lens):
        if n == 0:
            assert bool((out[b] == 5).all())
            continue
        # rows of a block weigh alike wherever the table has it: each block's rows once, weighed by how often they are seen
        whole, left = n // 16, n % 16
        times = torch.bincount(table[b, :whole].long(), minlength=blocks).double()[:, None].repeat(1, 16)
        if left:
            times[int(table[b, whole]), :left] += 1
        rows, times = pool.reshape(-1, rank + 64), times.reshape(-1)
        for h in {0, heads - 1}:
            c = rows[:, :rank].double()
            kv = c @ w[h].double().T
            s = (kv[:, :hd] @ q[b, h, :hd].double() + rows[:, rank:].double() @ q[b, h, hd:].double()) * scale
            p = times * torch.exp(s - s[times > 0].max())
            near(out[b, h], (p @ kv[:, hd:]) / p.sum())
