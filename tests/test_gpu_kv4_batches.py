"""Steps over the 4-bit cache at the batch sizes where the step's projections change their form (2, 3 - 32, above 32), some
slots inactive, tokens drawn: logits against the oracle that keeps the GPU's rows, tokens against the sampler's definition."""
import numpy as np
import pytest
import torch

import ql_inputs
from oracle import decode, sample as osample

from gpu_util import dev
from test_gpu_kv4_model import Following, host, model
from test_gpu_sample import eps

pytestmark = pytest.mark.gpu


class Partly(Following):
    """Slots that are not live keep the rows that the oracle computes."""
    live = ()

    def stored(self, k_rows, v_rows):
        if self.calls % len(self.positions) in self.live:
            return super().stored(k_rows, v_rows)
        self.calls += 1
        return k_rows, v_rows


@pytest.mark.parametrize("batch", [2, 17, 33, 40])
def test_drawn_steps(batch):
    cfg = ql_inputs.TINY
    gm, om = model(cfg, 2 * batch, batch, 2)
    try:
        bt = ql_inputs.fragmented_block_ids(2 * batch, seed=5).reshape(batch, 2).copy()
        cache = Partly(cfg, batch, 32, gm, bt)
        rng = np.random.default_rng(batch)
        on = (rng.random(batch) < 0.8).astype(np.int32)
        on[0] = 1
        u = rng.random((batch, 5)).astype(np.float32)
        t = rng.choice([0.0, 0.7, 1.5], batch).astype(np.float32)
        p = rng.choice([0.5, 0.95, 1.0], batch).astype(np.float32)
        keep = [dev(a) for a in (u, t, p, on, bt)]
        gm.ql_model_set_sampling(uniform=keep[0], temperature=keep[1], top_p=keep[2])
        tokens, positions = (torch.zeros(batch, dtype=torch.int32, device="cuda") for _ in range(2))
        nxt = torch.full((batch,), -9, dtype=torch.int32, device="cuda")
        logits = torch.zeros((batch, cfg.vocab), dtype=torch.float32, device="cuda")
        args = gm.step_args(tokens, positions, keep[4], nxt, logits=logits, active=keep[3])
        toks = ql_inputs.prompt_tokens(batch, cfg.vocab, seed=1).astype(np.int64)
        cache.live = set(np.nonzero(on)[0].tolist())
        for step in range(18):
            tokens.copy_(torch.from_numpy(toks.astype(np.int32)))
            gm.ql_decode_step(args)
            torch.cuda.synchronize()
            gm.ql_check_device_error()
            cache.begin([step] * batch)
            want = decode.decode_step(om, cache, toks, [step] * batch)
            got, drawn = host(logits).astype(np.float64), host(nxt)
            for b in range(batch):
                if not on[b]:
                    assert drawn[b] == -9
                    continue
                assert decode.logits_close(got[b], want[b]).all(), (step, b, np.abs(got[b] - want[b]).max())
                tok, _, gap = osample.sample(host(logits)[b], float(u[b, step % 5]), float(t[b]), 0, float(p[b]))
                assert drawn[b] == tok or gap <= 2 * eps(cfg.vocab), (step, b)
            toks = np.where(on, drawn, toks).astype(np.int64)
        assert host(positions).tolist() == (18 * on).tolist()
    finally:
        gm.close()
