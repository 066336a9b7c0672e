"""The 4-bit attention at the ends of its ranges (rows of q that are 4-byte aligned, one sequence over the whole GPU,
empty sequences before the only full one, ids that no block has) and sampling arrays that only a graph still needs."""
import gc
import math

import numpy as np
import pytest
import torch

import ql_inputs
from oracle import kv4

from gpu_util import lib, dev
from test_gpu_kv4 import attend, check, random_records, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads,n_kv,hd", [(8, 2, 128), (8, 1, 64), (12, 1, 128)])
def test_rows_of_q_and_out_that_are_4_byte_aligned(heads, n_kv, hd):
    ql = lib()
    rng = np.random.default_rng(heads + hd)
    lens = np.array([3, 50], np.int32)
    bt, blocks = tables(rng, lens, 4)
    rec = random_records(rng, blocks, n_kv, hd)
    q = rng.standard_normal((2, heads, hd)).astype(np.float16)
    wide = torch.zeros(2 + q.size, dtype=torch.float16, device="cuda")
    qd = wide[2:].view(q.shape)
    qd.copy_(dev(q))
    out = torch.full((2 + q.size,), 7.0, dtype=torch.float16, device="cuda")
    attend(ql, qd, dev(rec), dev(bt), dev(lens), 0.1, out=out[2:].view(q.shape))
    ql.ql_check_device_error()
    check(out[2:].view(q.shape).cpu().numpy(), q, rec, bt, lens, 0.1)
    assert out[:2].tolist() == [7.0, 7.0]


@pytest.mark.parametrize("heads", [2, 7, 16])
def test_one_sequence_over_the_whole_gpu(heads):
    ql = lib()
    rng = np.random.default_rng(heads)
    lens = np.array([120007], np.int32)
    bt, blocks = tables(rng, lens, 7600)
    rec = random_records(rng, blocks, 1, 64)
    q = rng.standard_normal((1, heads, 64)).astype(np.float16)
    ws = torch.zeros(ql.ql_paged_attn_kv4_workspace_bytes(1, heads, 1, 64, 7600), dtype=torch.uint8, device="cuda")
    for _ in range(2):   # the second call finds the workspace as the first left it
        got = attend(ql, dev(q), dev(rec), dev(bt), dev(lens), 0.125, ws=ws)
        ql.ql_check_device_error()
        check(got.cpu().numpy(), q, rec, bt, lens, 0.125)


def test_empty_sequences_before_the_only_full_one():
    ql = lib()
    rng = np.random.default_rng(3)
    for at in (0, 31, 32, 4999):
        lens = np.zeros(5000, np.int32)
        lens[at] = 333
        bt, blocks = tables(rng, lens, 21)
        rec = random_records(rng, blocks, 2, 64)
        q = rng.standard_normal((5000, 4, 64)).astype(np.float16)
        got = attend(ql, dev(q), dev(rec), dev(bt), dev(lens), 0.125).cpu().numpy()
        ql.ql_check_device_error()
        assert np.all(np.delete(got, at, 0) == 7.0)
        check(got[at:at + 1], q[at:at + 1], rec, bt[at:at + 1], lens[at:at + 1], 0.125)


@pytest.mark.parametrize("bad", [-2 ** 31, -1, 2 ** 31 - 1])
def test_ids_that_no_block_has(bad):
    """Their keys are left out: the output is that of the other blocks."""
    ql = lib()
    rng = np.random.default_rng(4)
    lens = np.array([640, 48], np.int32)
    bt, blocks = tables(rng, lens, 40)
    rec = random_records(rng, blocks, 2, 128)
    q = rng.standard_normal((2, 8, 128)).astype(np.float16)
    broken = bt.copy()
    broken[0, 17] = broken[1, 0] = bad
    got = attend(ql, dev(q), dev(rec), dev(broken), dev(lens), 0.1)
    with pytest.raises(ql.QLError) as e:
        ql.ql_check_device_error()
    assert e.value.status == ql.QL_EDEVICE
    left = bt.copy()
    left[0, 17:39], left[1, 0:2] = bt[0, 18:40], bt[1, 1:3]
    check(got.cpu().numpy(), q, rec, left, lens - 16, 0.1)


def test_a_graph_keeps_its_sampling_arrays():
    ql = lib()
    from quantized_transformer_decode_ql_gb300.model import DeviceModel
    cfg = ql_inputs.TINY
    gm = DeviceModel(cfg, ql_inputs.weights(cfg, seed=0), num_blocks=8, max_batch=1, max_blocks_per_seq=4,
                     kv_format=ql.QL_KV_Q4_1)
    try:
        table = dev(np.arange(4, dtype=np.int32).reshape(1, 4))
        runs = []
        for renewed in (False, True):
            tokens = torch.ones(1, dtype=torch.int32, device="cuda")
            positions = torch.zeros(1, dtype=torch.int32, device="cuda")
            out = torch.full((1, 40), -5, dtype=torch.int32, device="cuda")
            args = gm.step_args(tokens, positions, table, tokens, out_tokens=out)
            u = torch.rand((1, 32), generator=torch.Generator().manual_seed(1)).cuda()
            gm.ql_model_set_sampling(uniform=u, temperature=torch.full((1,), 1.5, device="cuda"))
            del u
            s = torch.cuda.Stream()
            torch.cuda.synchronize()
            gm.ql_decode_graph_capture(args, s)
            if renewed:
                gm.ql_model_set_sampling()
                gc.collect()
                junk = [torch.zeros((1, 32), device="cuda") for _ in range(64)]   # noqa: F841 (would take a freed array's place)
            torch.cuda.synchronize()
            gm.ql_decode_graph_replay(1, 30, s)
            s.synchronize()
            runs.append(out.cpu().numpy())
        gm.ql_check_device_error()
        assert np.array_equal(runs[0], runs[1])
    finally:
        gm.close()
