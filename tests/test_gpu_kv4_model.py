"""The model with a 4-bit KV cache (``kv_format = QL_KV_Q4_1``) and with sampled tokens
(``ql_model_set_sampling``).

A code that lies next to a border may differ between the GPU's row and the oracle's (their rows
differ by the rounding of the GEMVs), and a step of the format is a quarter of the rows' spread. So
the oracle here keeps what the GPU stored: after each GPU step its new records are decoded (in f64)
into the oracle's cache, checked to be within half a step of the oracle's own rows plus the
difference that the f16-cache tests allow between rows (2e-3 + 1e-2 |ref| of layer 0, twice the
absolute part behind it) and the f16 rounding of scale and minimum (2^-10 of the block's largest
value). Logits then have to meet the step tolerance of every other test.
"""
import numpy as np
import pytest
import torch

import ql_inputs
from oracle import decode, kv4, sample as osample

from gpu_util import lib, dev

pytestmark = pytest.mark.gpu


def host(t):
    return t.cpu().numpy()


class Following(decode.KVCache):
    """A cache that stores the GPU's decoded rows for the tokens that a step appends."""

    def __init__(self, cfg, batch, capacity, gm, tables):
        super().__init__(cfg, batch, capacity)
        self.gm, self.tables, self.calls, self.positions = gm, tables, 0, None

    def begin(self, positions):
        self.calls, self.positions = 0, [int(p) for p in positions]

    def rows(self, li, b, pos):
        """Decoded K and V [n_kv, n, hd] of slot b's positions, and the scales d [n_kv, n, hd] of K's and V's blocks."""
        hd = self.cfg.head_dim
        pos = np.asarray(pos)
        blk = np.asarray(self.tables)[b][pos // 16]
        used, at = np.unique(blk, return_inverse=True)
        rec = host(self.gm.kvq_pool[li, torch.from_numpy(used.astype(np.int64)).cuda()])
        k, v = kv4.rows_of(rec, at, pos % 16, hd)
        ends = []
        for code in (0x00, 0x11):                        # every code 0, every code 1: m and d + m
            rec[..., :16 * hd] = code
            ends.append(kv4.rows_of(rec, at, pos % 16, hd))
        d = [one - zero for zero, one in zip(*ends)]
        return [x.transpose(1, 0, 2) for x in (k, v, *d)]

    def stored(self, k_rows, v_rows):
        B = len(self.positions)
        li, b = divmod(self.calls, B)
        self.calls += 1
        k, v, dk, dv = (x[:, 0] for x in self.rows(li, b, [self.positions[b]]))
        for got, want, d in ((k, k_rows, dk), (v, v_rows, dv)):
            block = np.repeat(np.abs(want).reshape(want.shape[0], -1, 32).max(-1), 32, axis=-1)
            bound = d / 2 + 2.0 ** -10 * block + (2e-3 if li == 0 else 4e-3) + 1e-2 * np.abs(want)
            assert np.all(np.abs(got - want) <= bound), (li, b, float((np.abs(got - want) / bound).max()))
        return k, v


def model(cfg, num_blocks, max_batch, maxb, w=None):
    ql = lib()
    from quantized_transformer_decode_ql_gb300.model import DeviceModel
    w = ql_inputs.weights(cfg, seed=0) if w is None else w
    return DeviceModel(cfg, w, num_blocks=num_blocks, max_batch=max_batch, max_blocks_per_seq=maxb,
                       kv_format=ql.QL_KV_Q4_1), decode.Q4Model(cfg, w)


@pytest.mark.parametrize("batch,moe", [(1, False), (3, False), (1, True)])
def test_decode_steps(batch, moe):
    cfg = ql_inputs.TINY_MOE if moe else ql_inputs.TINY
    gm, om = model(cfg, 32, 4, 4)
    try:
        bt = ql_inputs.fragmented_block_ids(32, seed=5)[: batch * 4].reshape(batch, 4).copy()
        cache = Following(cfg, batch, 64, gm, bt)
        tokens, positions, nxt = (torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(3))
        logits = torch.zeros((batch, cfg.vocab), dtype=torch.float32, device="cuda")
        table = dev(bt)                                  # the steps read it
        args = gm.step_args(tokens, positions, table, nxt, logits=logits)
        toks = ql_inputs.prompt_tokens(batch, cfg.vocab, seed=1).astype(np.int64)
        for step in range(20):
            tokens.copy_(torch.from_numpy(toks.astype(np.int32)))
            gm.ql_decode_step(args)
            torch.cuda.synchronize()
            cache.begin([step] * batch)
            want = decode.decode_step(om, cache, toks, [step] * batch)
            got = host(logits).astype(np.float64)
            for b in range(batch):
                assert decode.logits_close(got[b], want[b]).all(), (step, b, np.abs(got[b] - want[b]).max())
                if decode.greedy_must_agree(want[b]):
                    assert int(nxt[b]) == int(decode.greedy(want[b:b + 1])[0])
            toks = decode.greedy(want).astype(np.int64)
        assert host(positions).tolist() == [20] * batch
        gm.ql_check_device_error()
    finally:
        gm.close()


def test_an_inactive_slot_is_frozen_and_a_bad_table_is_recorded():
    ql = lib()
    cfg = ql_inputs.TINY
    gm, _ = model(cfg, 16, 3, 4)
    try:
        bt = np.arange(12, dtype=np.int32).reshape(3, 4)
        tokens = torch.ones(3, dtype=torch.int32, device="cuda")
        positions = dev(np.array([0, 5, 3], np.int32))
        nxt = torch.full((3,), -9, dtype=torch.int32, device="cuda")
        gm.kvq_pool.fill_(0x11)
        before = gm.kvq_pool.clone()
        table, active = dev(bt), dev(np.array([1, 0, 1], np.int32))
        gm.ql_decode_step(gm.step_args(tokens, positions, table, nxt, active=active))
        torch.cuda.synchronize()
        gm.ql_check_device_error()
        assert host(positions).tolist() == [1, 5, 4] and int(nxt[1]) == -9
        assert torch.equal(gm.kvq_pool[:, 4:8], before[:, 4:8]) and not torch.equal(gm.kvq_pool[:, 0], before[:, 0])
        table[0, 0] = 99
        gm.ql_decode_step(gm.step_args(tokens, positions, table, nxt))
        with pytest.raises(ql.QLError) as e:
            gm.ql_check_device_error()
        assert e.value.status == ql.QL_EDEVICE
        with pytest.raises(ql.QLError):
            gm.ql_model_set_option(ql.QL_OPT_STEP_KERNEL, ql.QL_STEP_PERSISTENT)
    finally:
        gm.close()


def test_prefill_chunks_then_decode():
    cfg = ql_inputs.TINY
    gm, om = model(cfg, 16, 64, 8)
    try:
        bt = ql_inputs.fragmented_block_ids(16, seed=6)[:8].copy()
        cache = Following(cfg, 1, 128, gm, bt.reshape(1, -1))
        prompt = ql_inputs.prompt_tokens(107, cfg.vocab, seed=2)
        position, nxt = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
        logits = torch.zeros(cfg.vocab, dtype=torch.float32, device="cuda")
        p = 0
        for T in (16, 1, 50, 2, 38):
            toks = prompt[p:p + T]
            chunk, table = dev(toks.astype(np.int32)), dev(bt)
            gm.ql_prefill_chunk(chunk, position, table, logits=logits, next_token=nxt)
            torch.cuda.synchronize()
            for t in range(T):
                cache.begin([p + t])
                want = decode.decode_step(om, cache, [int(toks[t])], [p + t])[0]
            p += T
            got = host(logits).astype(np.float64)
            assert decode.logits_close(got, want).all(), (p, np.abs(got - want).max())
            assert int(position) == p
        tok = int(decode.greedy(want))
        tokens, positions = dev(np.array([tok], np.int32)), dev(np.array([p], np.int32))
        lg = torch.zeros((1, cfg.vocab), dtype=torch.float32, device="cuda")
        table = dev(bt.reshape(1, -1))
        args = gm.step_args(tokens, positions, table, nxt, logits=lg)
        for step in range(5):
            tokens.fill_(tok)
            gm.ql_decode_step(args)
            torch.cuda.synchronize()
            cache.begin([p + step])
            want = decode.decode_step(om, cache, [tok], [p + step])[0]
            assert decode.logits_close(host(lg)[0].astype(np.float64), want).all(), step
            tok = int(decode.greedy(want))
        gm.ql_check_device_error()
    finally:
        gm.close()


def test_full_width_step_over_a_written_context():
    """The 8B width (two layers): contexts quantised by ``write_context``, then two steps of a batch of two."""
    ql = lib()
    from quantized_transformer_decode_ql_gb300.model import DeviceModel
    from test_gpu_decode_full import oracle_model
    cfg = ql_inputs.qwen3_8b_layers(2)
    lens, maxb = [900, 33], 60
    gm = DeviceModel.from_layer_fn(cfg, ql_inputs.device_tensor_fn(cfg, seed=0), num_blocks=2 * maxb, max_batch=2,
                                   max_blocks_per_seq=maxb, kv_format=ql.QL_KV_Q4_1)
    try:
        om = oracle_model(gm)
        bt = ql_inputs.fragmented_block_ids(2 * maxb, seed=5).reshape(2, maxb).copy()
        cache = Following(cfg, 2, maxb * 16, gm, bt)
        for b, n in enumerate(lens):
            k, v = ql_inputs.kv_context(cfg.n_layers, cfg.n_kv_heads, cfg.head_dim, n, seed=4, slot=b)
            gm.write_context(bt[b], k, v)
            torch.cuda.synchronize()
            for li in range(cfg.n_layers):
                rows = cache.rows(li, b, np.arange(n))
                want = kv4.dequantize(*kv4.quantize(k[li].reshape(-1, cfg.head_dim).astype(np.float32)))
                assert np.array_equal(rows[0].reshape(-1, cfg.head_dim), want)      # the codec's own values
                cache.k[b, li, :, :n], cache.v[b, li, :, :n] = rows[0], rows[1]
        toks = ql_inputs.prompt_tokens(2, cfg.vocab, seed=1).astype(np.int64)
        tokens, positions = dev(toks.astype(np.int32)), dev(np.array(lens, np.int32))
        nxt = torch.zeros(2, dtype=torch.int32, device="cuda")
        logits = torch.zeros((2, cfg.vocab), dtype=torch.float32, device="cuda")
        table = dev(bt)                                  # the steps read it
        args = gm.step_args(tokens, positions, table, nxt, logits=logits)
        pos = np.array(lens)
        for step in range(2):
            x0 = host(gm.embed[torch.from_numpy(toks).cuda()]).astype(np.float64)
            tokens.copy_(torch.from_numpy(toks.astype(np.int32)))
            gm.ql_decode_step(args)
            torch.cuda.synchronize()
            cache.begin(pos)
            want = decode.logits_by_rows(om.lm_head, decode.decode_hidden(om, cache, x0, pos))
            got = host(logits).astype(np.float64)
            for b in range(2):
                assert decode.logits_close(got[b], want[b]).all(), (step, b, np.abs(got[b] - want[b]).max())
            toks = decode.greedy(want).astype(np.int64)
            pos = pos + 1
        gm.ql_check_device_error()
    finally:
        gm.close()


def filters(batch, vocab, seed, steps=8):
    rng = np.random.default_rng(seed)
    return dict(uniform=rng.random((batch, steps)).astype(np.float32),
                temperature=rng.choice([0.0, 0.7, 1.3], batch).astype(np.float32),
                top_k=rng.choice([0, 5, 300], batch).astype(np.int32),
                top_p=rng.choice([0.6, 0.95, 1.0], batch).astype(np.float32),
                min_p=rng.choice([0.0, 0.05], batch).astype(np.float32))


@pytest.mark.parametrize("fmt", ["f16", "q4_1"])
@pytest.mark.parametrize("batch", [1, 3])
def test_sampled_steps_eager_and_captured(fmt, batch):
    """A prompt chunk, then steps whose tokens are drawn: every token is the one that the sampler's
    definition gives for the step's own logits and the position's number; a captured graph draws the same."""
    ql = lib()
    from quantized_transformer_decode_ql_gb300.model import DeviceModel
    cfg = ql_inputs.TINY
    gm = DeviceModel(cfg, ql_inputs.weights(cfg, seed=0), num_blocks=64, max_batch=16, max_blocks_per_seq=4,
                     kv_format=ql.QL_KV_Q4_1 if fmt == "q4_1" else ql.QL_KV_F16)
    try:
        bt = ql_inputs.fragmented_block_ids(64, seed=5)[: batch * 4].reshape(batch, 4).copy()
        f = filters(batch, cfg.vocab, batch)
        d = {k: dev(v) for k, v in f.items()}
        table = dev(bt)
        runs = []
        for captured in (False, True):
            start = []
            for b in range(batch):
                position, first = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
                gm.ql_prefill_chunk(dev(ql_inputs.prompt_tokens(9, cfg.vocab, seed=b).astype(np.int32)), position, table[b],
                                    next_token=first)
                start.append(first)
            tokens = torch.cat(start).clone()
            positions = torch.full((batch,), 9, dtype=torch.int32, device="cuda")
            logits = torch.zeros((batch, cfg.vocab), dtype=torch.float32, device="cuda")
            out = torch.full((batch, 40), -5, dtype=torch.int32, device="cuda")
            args = gm.step_args(tokens, positions, table, tokens, logits=logits, out_tokens=out)   # feeds itself
            gm.ql_model_set_sampling(**d)
            if captured:
                s = torch.cuda.Stream()
                torch.cuda.synchronize()
                with torch.cuda.stream(s):
                    gm.ql_decode_graph_capture(args, s)
                    gm.ql_decode_graph_replay(batch, 12, s)
                s.synchronize()
            else:
                sure = 0
                for step in range(12):
                    gm.ql_decode_step(args)
                    torch.cuda.synchronize()
                    x, got = host(logits), host(tokens)
                    for b in range(batch):
                        tok, _, gap = osample.sample(x[b], float(f["uniform"][b, (9 + step) % 8]), float(f["temperature"][b]),
                                                     int(f["top_k"][b]), float(f["top_p"][b]), float(f["min_p"][b]))
                        if gap > 1e-8:
                            sure += 1
                            assert got[b] == tok, (step, b)
                assert sure >= 11 * batch
            gm.ql_check_device_error()
            assert host(positions).tolist() == [21] * batch
            runs.append(host(out))
            gm.ql_model_set_sampling()
        assert np.array_equal(runs[0], runs[1])
        # without sampling: the arg max again, one step further
        positions.fill_(20)
        gm.ql_decode_step(args)
        torch.cuda.synchronize()
        assert host(tokens).tolist() == host(logits).argmax(1).tolist()
    finally:
        gm.close()


def test_sampling_refusals_and_inactive_slots():
    ql = lib()
    from quantized_transformer_decode_ql_gb300.model import DeviceModel
    cfg = ql_inputs.TINY
    gm = DeviceModel(cfg, ql_inputs.weights(cfg, seed=0), num_blocks=16, max_batch=2, max_blocks_per_seq=4)
    try:
        L = ql.lib()
        import ctypes
        for s in (ql.Sampling(None, None, None, None, None, 1), ql.Sampling(None, None, None, None, 64, 0),
                  ql.Sampling(66, None, None, None, 64, 1)):
            assert L.ql_model_set_sampling(gm.handle, ctypes.byref(s)) == ql.QL_EINVAL
        assert L.ql_model_set_sampling(None, None) == ql.QL_EINVAL
        u = torch.full((2,), 0.5, device="cuda")
        gm.ql_model_set_sampling(uniform=u, temperature=torch.tensor([1.0, -1.0], device="cuda"))
        tokens = torch.ones(2, dtype=torch.int32, device="cuda")
        positions = torch.zeros(2, dtype=torch.int32, device="cuda")
        nxt = torch.full((2,), -9, dtype=torch.int32, device="cuda")
        bt, active = dev(np.arange(8, dtype=np.int32).reshape(2, 4)), dev(np.array([1, 0], np.int32))
        gm.ql_decode_step(gm.step_args(tokens, positions, bt, nxt, active=active))
        gm.ql_check_device_error()
        assert int(nxt[0]) >= 0 and int(nxt[1]) == -9
        gm.ql_decode_step(gm.step_args(tokens, positions, bt, nxt))      # slot 1's temperature is out of range
        with pytest.raises(ql.QLError):
            gm.ql_check_device_error()
        assert int(nxt[1]) == -1
        if gm.ql_model_persistent_max_batch() > 0:
            gm.ql_model_set_option(ql.QL_OPT_STEP_KERNEL, ql.QL_STEP_PERSISTENT)
            with pytest.raises(ql.QLError) as e:
                gm.ql_decode_step(gm.step_args(tokens, positions, bt, nxt))
            assert e.value.status == ql.QL_EINVAL
    finally:
        gm.close()
