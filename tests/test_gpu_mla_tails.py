"""Latent attention over one key that outweighs each of very many others, which together weigh something: weights far below the largest
must not vanish in f16. The cache is two blocks, repeated by the table, and the answer is worked out from the two rows."""
import math

import numpy as np
import pytest
import torch

from gpu_util import dev, lib
from oracle import mla

pytestmark = pytest.mark.gpu

BELOW = 25.2      # log2 of how far the others' weights lie below the largest


def case(heads, hd, rank, rows, seed, quiet, below=BELOW):
    g = np.random.default_rng(seed)
    scale = 0.125
    pool = np.zeros((2, 16, rank + 64), np.float16)
    latents = g.standard_normal((2, rank)).astype(np.float16)        # of the one key, of the others
    if quiet:      # the one key's value is 0: the sums hold nothing that the others' could be lost beside
        latents[0] = 0
    pool[..., :rank] = latents[1]
    pool[0, 0, :rank] = latents[0]
    pool[0, 0, rank] = 1.0
    q = np.zeros((rows, heads, hd + 64), np.float16)
    q[..., hd] = below * math.log(2) / scale
    w = (g.standard_normal((heads, 2 * hd, rank)) / math.sqrt(rank)).astype(np.float16)
    return pool, q, w, scale, float(q[0, 0, hd]) * scale, latents.astype(np.float64)


def answer(w, latents, score, n, hd, lift, sums):
    """The output of a query that sees n keys, and its bound. The others' weights are off by half a step of f16's subnormals each, all of
    them alike, where the largest weight is 2^lift: by n TINY 2^-lift of the whole. Then a half step of f16 for values and output, a step of
    f32 for each sum over the rank and the score's exponent (8 at most: product, difference, power). A sum over the keys takes 16 of them at
    a time (the depth of a product's instruction) into one f32 number, `sums` such numbers in turn: n / 16 / sums additions, each of which
    may drop what lies below a step of the number so far, up to E of the sum of the magnitudes."""
    v = latents @ w[:, hd:].astype(np.float64).transpose(0, 2, 1)    # [heads, 2, hd]
    size = np.abs(latents) @ np.abs(w[:, hd:].astype(np.float64)).transpose(0, 2, 1)
    other = math.exp(-score)
    total = 1 + (n - 1) * other
    p = np.array([1 / total, (n - 1) * other / total])
    out = np.einsum("t,htd->hd", p, v)
    off = n * mla.TINY * 2.0 ** -lift / total
    rank = latents.shape[-1]
    bound = ((off + 2 * p[0] * p[1] * (8 + score) * mla.E) * (np.abs(v[:, 0]) + np.abs(v[:, 1])) + (mla.U + (rank + n / 16 / sums) * mla.E) * np.einsum("t,htd->hd", p, size)
             + (2 * mla.U + 400 * mla.E) * np.abs(out) + mla.TINY)
    return out, bound


@pytest.mark.parametrize("quiet", [False, True])
@pytest.mark.parametrize("heads,hd,rank", [(2, 64, 256), (40, 64, 256)])
def test_decode(heads, hd, rank, quiet):
    """As many sequences as windows, so that few of them are cut."""
    ql = lib()
    n, batch = 1 << 19, 160
    maxb = n // 16
    pool, q, w, scale, score, latents = case(heads, hd, rank, batch, heads, quiet)
    table = torch.ones((batch, maxb), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    out = torch.zeros((batch, heads, hd), dtype=torch.float16, device="cuda")
    ws = torch.empty(ql.ql_mla_decode_workspace_bytes(batch, heads, hd, rank, maxb), dtype=torch.uint8, device="cuda")
    ql.ql_mla_attn_decode(dev(q), dev(w), dev(pool), table, torch.full((batch,), n, dtype=torch.int32, device="cuda"), batch, heads, hd, rank, 64, 16,
                          maxb, 2, scale, out, ws)
    torch.cuda.synchronize()
    ql.ql_check_device_error()
    want, bound = answer(w, latents, score, n, hd, 6, 1)
    worst = np.max(np.abs(out.cpu().numpy().astype(np.float64) - want) / bound)
    assert worst <= 1, worst


@pytest.mark.parametrize("quiet", [False, True])
@pytest.mark.parametrize("top", [0.0, 3.0, 30.0, -40.0])
def test_chunk(top, quiet):
    """As many units as are not cut. The reference is chosen by the first scores, so these lie at, above and below 0."""
    ql = lib()
    heads, hd, rank, n, rows = 160, 64, 256, 1 << 18, 40
    maxb = n // 16
    pool, q, w, scale, score, latents = case(heads, hd, rank, rows, 3, quiet)
    q[..., hd + 1] = top * math.log(2) / scale     # the same for every key
    pool[..., rank + 1] = 1.0
    table = torch.ones((1, maxb), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    out = torch.zeros((rows, heads, hd), dtype=torch.float16, device="cuda")
    ws = torch.empty(ql.ql_mla_chunk_workspace_bytes(rows, heads, hd, rank, maxb), dtype=torch.uint8, device="cuda")
    ql.ql_mla_attn_chunk(dev(q), dev(w), dev(pool), table, torch.tensor([n - rows], dtype=torch.int32, device="cuda"), rows, heads, hd, rank, 64, 16, maxb, 2,
                         scale, out, ws)
    torch.cuda.synchronize()
    ql.ql_check_device_error()
    got = out.cpu().numpy().astype(np.float64)
    for i in (0, rows // 2, rows - 1):
        want, bound = answer(w, latents, score, n - rows + i + 1, hd, 5, 2)
        worst = np.max(np.abs(got[i] - want) / bound)
        assert worst <= 1, (i, worst)
