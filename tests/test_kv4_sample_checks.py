"""Refusals of the 4-bit pool's and the sampler's Python entry points that need no GPU: arrays of another type, too short,
or not contiguous never reach the library."""
import pytest
import torch

import quantized_transformer_decode_ql_gb300 as ql
from quantized_transformer_decode_ql_gb300.model import DeviceModel


def refused(f, *a, **k):
    with pytest.raises(ql.QLError) as e:
        f(*a, **k)
    assert e.value.status == ql.QL_EINVAL


def test_sample_arrays():
    lg, u, tok = torch.zeros((4, 10)), torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    f4, i4 = torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    for bad in (dict(uniform=torch.zeros(3)), dict(uniform=u.double()), dict(uniform=torch.zeros(8)[::2]), dict(tokens=tok.long()),
                dict(tokens=tok[:3]), dict(temperature=f4[:3]), dict(temperature=i4), dict(top_k=i4.long()), dict(top_k=f4),
                dict(top_p=f4.half()), dict(min_p=torch.zeros(8)[::2]), dict(probs=f4[:1]), dict(active=torch.ones(4)),
                dict(active=i4[:2])):
        refused(ql.ql_sample, lg, **{**dict(uniform=u, tokens=tok), **bad})


def test_slots():
    k = torch.zeros((3, 2, 64))
    pool = torch.zeros((2, 2, 1280), dtype=torch.uint8)
    for slots in (torch.zeros(3, dtype=torch.int32), torch.zeros(6, dtype=torch.int64)[::2]):
        refused(ql.ql_kv4_write, k, k, slots, 2, 64, pool, 2)
        refused(ql.ql_kv4_read, pool, slots, 2, 64, 2, k, k)


def test_model_sampling_arrays():
    m = DeviceModel.__new__(DeviceModel)
    m.handle, m._sampling, m._graph_sampling = None, None, {}
    u = torch.zeros((2, 5))
    for bad in (dict(uniform=torch.zeros(())), dict(uniform=torch.zeros((2, 2, 2))), dict(uniform=u.double()), dict(uniform=u.t()),
                dict(temperature=torch.zeros(1)), dict(top_k=torch.zeros(2)), dict(top_p=torch.zeros(2, dtype=torch.int32)),
                dict(min_p=torch.zeros(4)[::2])):
        refused(m.ql_model_set_sampling, **{**dict(uniform=u), **bad})
    assert m._sampling is None
    m._sampling = (u, None, None, None, None)
    args = ql.StepArgs()
    args.batch = 3
    refused(m.ql_decode_step, args)
    refused(m.ql_decode_graph_capture, args, None)


def test_library_refusals():
    import ctypes
    L = ql.lib()
    s = ql.Sampling(None, None, None, None, 64, 1)
    assert L.ql_model_set_sampling(None, ctypes.byref(s)) == ql.QL_EINVAL
    assert L.ql_model_set_sampling(None, None) == ql.QL_EINVAL
    for batch, heads, maxb in ((1, 8, 1 << 27), (1, 8, 1 << 25), (60000, 32, 1 << 26), (65536, 8, 4), (65535, 512, 4), (1, (1 << 20) + 8, 4)):
        assert L.ql_paged_attn_decode_kv4(64, 1024, 64, 64, batch, heads, 8, 128, 16, maxb, 9, 0.1, 64, 64, 1 << 40, None) == ql.QL_EINVAL
