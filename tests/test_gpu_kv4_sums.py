"""Sums of the 4-bit attention over contexts so long that a warp adds hundreds of tiles: codes are not
negative, so a sum of scaled codes and one of minima grow while the values that they stand for cancel."""
import numpy as np
import pytest
import torch

from gpu_util import lib, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,hd", [(16, 128), (32, 128), (32, 64)])
def test_long_means_of_values_that_cancel(heads, hd):
    """q = 0: every output is the mean of the values. 128 sequences share 4096 blocks (65536 tokens each), about 860 tiles a
    warp. Bound per element: the output's rounding, 2^-11 |out| + 2^-25, and two sums (scaled codes and minima; two matrix
    products a tile) whose additions truncate by 2^-23 of the sum at most. Settled every 8 tiles, the sum is k tiles' when the
    k-th is added: 2 * 2^-23 * (1 + ... + 8) / 8 = 9 * 2^-23 of the mean of d c, and as much of the mean of |m|. 2^-21 of the
    same covers the joins in f32."""
    ql = lib()
    B, n_kv, maxb = 128, 4, 4096
    g = torch.Generator(device="cuda").manual_seed(heads + hd)
    k, v = (torch.randn((maxb * 16, n_kv, hd), device="cuda", generator=g) for _ in range(2))
    slots = torch.randperm(maxb * 16, device="cuda", generator=g)
    pool = torch.zeros((maxb, n_kv, 20 * hd), dtype=torch.uint8, device="cuda")
    ql.ql_kv4_write(k, v, slots, n_kv, hd, pool, maxb)
    ql.ql_kv4_read(pool, slots, n_kv, hd, maxb, k, v)
    want = v.double().mean(0)
    low = v.double().view(-1, n_kv, hd // 32, 32).min(-1).values.abs().mean(0).amax()    # the least value is m + 0 d or near it
    q = torch.zeros((B, heads, hd), dtype=torch.float16, device="cuda")
    table = torch.arange(maxb, dtype=torch.int32, device="cuda").repeat(B, 1)
    lens = torch.full((B,), maxb * 16, dtype=torch.int32, device="cuda")
    out = torch.zeros((B, heads, hd), dtype=torch.float16, device="cuda")
    ws = torch.zeros(ql.ql_paged_attn_kv4_workspace_bytes(B, heads, n_kv, hd, maxb), dtype=torch.uint8, device="cuda")
    ql.ql_paged_attn_decode_kv4(q, pool, table, lens, B, heads, n_kv, hd, 16, maxb, maxb, 1.0, out, ws)
    ql.ql_check_device_error()
    want = want.repeat_interleave(heads // n_kv, 0)
    bound = 2.0 ** -11 * want.abs() + 2.0 ** -25 + float(low) * (2 * 9 * 2.0 ** -23 + 2 * 2.0 ** -21)
    err = (out.double() - want).abs()
    assert bool((err <= bound).all()), float((err / bound).max())
