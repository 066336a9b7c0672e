"""What lies behind a prompt chunk's last position, and blocks that a table does not have.

A block that a sequence takes over holds whatever its last owner left there: rows behind the chunk must not
reach the output, not even as 0 x NaN. The same for the buffer that a 4-bit model reads a context back into,
which all sequences share. Keys of an id outside the pool are left out of the softmax, by every path.
"""
import numpy as np
import pytest
import torch

import ql_inputs
from oracle import decode

from gpu_util import lib, dev
from test_gpu_kv4_model import Following, model

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("p0,T", [(0, 1), (0, 5), (21, 20), (40, 30)])
@pytest.mark.parametrize("stale", [float("nan"), float("inf")])
def test_chunk_attention_over_blocks_with_stale_rows(hd, p0, T, stale):
    """The output is bit for bit that over zeros in the same places."""
    ql = lib()
    rng = np.random.default_rng(p0 + T + hd)
    n_heads, n_kv = 8, 2
    L = p0 + T
    nb = (L + 15) // 16
    assert L % 16
    k, v = (rng.standard_normal((nb, n_kv, 16, hd)).astype(np.float16) for _ in range(2))
    table = rng.permutation(nb).astype(np.int32)
    q = rng.standard_normal((T, n_heads, hd)).astype(np.float16)
    ws = torch.empty(ql.ql_paged_attn_chunk_workspace_bytes(T, n_heads, n_kv, hd), dtype=torch.uint8, device="cuda")
    outs = []
    for behind in (0.0, stale):
        k[table[-1], :, L % 16:], v[table[-1], :, L % 16:] = behind, behind
        out = torch.full((T, n_heads * hd), 7.0, dtype=torch.float16, device="cuda")
        ql.ql_paged_attn_chunk(dev(q), dev(k), dev(v), dev(table), dev(np.array([p0], np.int32)), T, n_heads, n_kv, hd, 16, nb,
                               nb, 0.1, out, ws)
        ql.ql_check_device_error()
        outs.append(out.cpu().numpy())
    assert np.all(np.isfinite(outs[0])) and np.array_equal(*outs)


@pytest.mark.parametrize("hd", [64, 128])
def test_tokens_without_a_key_are_zero(hd):
    """The first block's id is outside the pool: tokens 0 - 15 see nothing, the others the second block."""
    ql = lib()
    rng = np.random.default_rng(hd)
    T, n_heads, n_kv = 24, 8, 2
    k, v = (rng.standard_normal((2, n_kv, 16, hd)).astype(np.float16) for _ in range(2))
    q = rng.standard_normal((T, n_heads, hd)).astype(np.float16)
    ws = torch.empty(ql.ql_paged_attn_chunk_workspace_bytes(T, n_heads, n_kv, hd), dtype=torch.uint8, device="cuda")
    out = torch.full((T, n_heads * hd), 7.0, dtype=torch.float16, device="cuda")
    ql.ql_paged_attn_chunk(dev(q), dev(k), dev(v), dev(np.array([-1, 1], np.int32)), dev(np.zeros(1, np.int32)), T, n_heads, n_kv, hd,
                           16, 2, 2, 0.1, out, ws)
    with pytest.raises(ql.QLError):
        ql.ql_check_device_error()
    got = out.cpu().numpy().reshape(T, n_heads, hd).astype(np.float64)
    assert np.all(got[:16] == 0)
    for t in range(16, T):
        for h in range(n_heads):
            x = k[1, h // 4, :t - 15].astype(np.float64) @ q[t, h].astype(np.float64) * 0.1
            p = np.exp(x - x.max())
            want = p @ v[1, h // 4, :t - 15].astype(np.float64) / p.sum()
            assert np.all(np.abs(got[t, h] - want) <= 2e-3 + 1e-2 * np.abs(want))


def prompt(gm, cfg, tokens, position, table):
    logits = torch.zeros(cfg.vocab, dtype=torch.float32, device="cuda")
    gm.ql_prefill_chunk(dev(tokens.astype(np.int32)), dev(np.array([position], np.int32)), dev(table), logits=logits)
    torch.cuda.synchronize()
    return logits.cpu().numpy()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), 2e5])
def test_a_sequence_does_not_reach_the_next_one_s_prompt(value):
    """A first sequence's context holds a value that is not finite (or not as f16) at position 30; a second one's
    prompt of 20 tokens gives the same logits as on a fresh handle."""
    ql = lib()
    cfg = ql_inputs.TINY
    one, two = np.array([0, 1, 2, 3], np.int32), np.array([7, 5, 4, 6], np.int32)
    tokens = ql_inputs.prompt_tokens(60, cfg.vocab, seed=3)
    got = []
    for spoiled in (False, True):
        gm, _ = model(cfg, 8, 40, 4)
        try:
            if spoiled:
                rows = torch.ones((32, cfg.n_kv_heads, cfg.head_dim), device="cuda")
                rows[30, :, ::3] = value
                for li in range(cfg.n_layers):
                    ql.ql_kv4_write(torch.ones_like(rows), rows, torch.arange(32, device="cuda"), cfg.n_kv_heads, cfg.head_dim,
                                    gm.kvq_pool[li], 8)
                prompt(gm, cfg, tokens[20:28], 32, one)
                with pytest.raises(ql.QLError):          # recorded, and cleared
                    gm.ql_check_device_error()
            got.append(prompt(gm, cfg, tokens[:20], 0, two))
            gm.ql_check_device_error()
        finally:
            gm.close()
    assert np.all(np.isfinite(got[0])) and np.array_equal(*got)


@pytest.mark.parametrize("bad", [-1, 8, 2 ** 31 - 1, -2 ** 31])
def test_a_chunk_leaves_out_the_keys_of_a_block_that_the_pool_does_not_have(bad, monkeypatch):
    """After another sequence's prompt, a chunk at position 48 whose table's second id is outside the pool: the oracle's
    logits over positions 0 - 15 and 32 on."""
    ql = lib()
    cfg = ql_inputs.TINY
    gm, om = model(cfg, 8, 64, 4)
    try:
        good = np.array([7, 5, 4, 6], np.int32)
        prompt(gm, cfg, ql_inputs.prompt_tokens(64, cfg.vocab, seed=5), 0, np.array([0, 1, 2, 3], np.int32))
        gm.ql_check_device_error()
        k, v = ql_inputs.kv_context(cfg.n_layers, cfg.n_kv_heads, cfg.head_dim, 48, seed=6)
        gm.write_context(good, k, v)
        broken = good.copy()
        broken[1] = bad
        tokens = ql_inputs.prompt_tokens(10, cfg.vocab, seed=7)
        got = prompt(gm, cfg, tokens, 48, broken).astype(np.float64)
        with pytest.raises(ql.QLError) as e:
            gm.ql_check_device_error()
        assert e.value.status == ql.QL_EDEVICE
        cache = Following(cfg, 1, 64, gm, good.reshape(1, -1))
        for li in range(cfg.n_layers):
            rows = cache.rows(li, 0, np.arange(48))
            cache.k[0, li, :, :48], cache.v[0, li, :, :48] = rows[0], rows[1]
        plain = decode.ops.gqa_attention
        monkeypatch.setattr(decode.ops, "gqa_attention",
                            lambda q, k, v, s: plain(q, np.delete(k, np.s_[16:32], 1), np.delete(v, np.s_[16:32], 1), s))
        for t in range(10):
            cache.begin([48 + t])
            want = decode.decode_step(om, cache, [int(tokens[t])], [48 + t])[0]
        assert decode.logits_close(got, want).all(), float(np.abs(got - want).max())
    finally:
        gm.close()


def test_a_context_s_value_above_f16_is_recorded():
    """The format holds it (m + 15 d up to 1e6), the chunk's attention reads it as f16."""
    ql = lib()
    cfg = ql_inputs.TINY
    gm, _ = model(cfg, 8, 40, 4)
    try:
        table, tokens = np.array([3, 0, 1, 2], np.int32), ql_inputs.prompt_tokens(8, cfg.vocab, seed=3)
        for value, fits in ((65000.0, True), (65504.0 * 1.2, False)):
            rows = torch.ones((16, cfg.n_kv_heads, cfg.head_dim), device="cuda")
            rows[9, 1, 40] = value
            ql.ql_kv4_write(torch.ones_like(rows), rows, 48 + torch.arange(16, device="cuda"), cfg.n_kv_heads, cfg.head_dim,
                            gm.kvq_pool[1], 8)
            gm.ql_check_device_error()                     # the row itself fits the format
            prompt(gm, cfg, tokens, 16, table)
            if fits:
                gm.ql_check_device_error()
            else:
                with pytest.raises(ql.QLError) as e:
                    gm.ql_check_device_error()
                assert e.value.status == ql.QL_EDEVICE
    finally:
        gm.close()
