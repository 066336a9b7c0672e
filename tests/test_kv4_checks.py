"""Refusals of the 4-bit pool's and the sampler's Python entry points that need no GPU: tensors of another type, too small for
the sizes given with them, not contiguous, or not on the GPU never reach the library."""
import pytest
import torch

import quantized_transformer_decode_ql_gb300 as ql
from quantized_transformer_decode_ql_gb300.model import DeviceModel


def refused(word, f, *a, **k):
    with pytest.raises(ql.QLError) as e:
        f(*a, **k)
    assert e.value.status == ql.QL_EINVAL and word in str(e.value), str(e.value)


class Gpu(torch.Tensor):
    """A host tensor that says it is on the current GPU."""

    def get_device(self):
        return 0


@pytest.fixture
def gpu(monkeypatch):
    from quantized_transformer_decode_ql_gb300 import _lib
    monkeypatch.setattr(_lib, "_current_device", lambda: 0)
    return lambda t: t.as_subclass(Gpu)


@pytest.fixture
def no_library(monkeypatch):
    """Nothing may get past the checks."""
    import quantized_transformer_decode_ql_gb300 as m
    from quantized_transformer_decode_ql_gb300 import model

    def called():
        raise AssertionError("the library was called")
    monkeypatch.setattr(m, "lib", called)
    monkeypatch.setattr(model, "lib", called)


@pytest.mark.parametrize("hd", [64, 128])
def test_pools_smaller_than_num_blocks(gpu, no_library, hd):
    k = gpu(torch.zeros((3, 2, hd)))
    slots = gpu(torch.zeros(3, dtype=torch.int64))
    pool = gpu(torch.zeros((2, 2, 20 * hd), dtype=torch.uint8))
    wide = gpu(torch.zeros((2, 4, 20 * hd), dtype=torch.uint8)[:, ::2])
    for p, blocks in ((pool, 3), (pool[:, :1], 2), (pool.flatten()[1:], 2), (None, 1), (wide, 2)):
        refused("pool", ql.ql_kv4_write, k, k, slots, 2, hd, p, blocks)
        refused("pool", ql.ql_kv4_read, p, slots, 2, hd, blocks, k, k)


def attention(**over):
    B, H, G, hd, maxb, blocks = 2, 8, 2, 64, 3, 5
    a = dict(q=torch.zeros((B, H, hd), dtype=torch.float16), pool=torch.zeros((blocks, G, 20 * hd), dtype=torch.uint8),
             block_tables=torch.zeros((B, maxb), dtype=torch.int32), context_lens=torch.zeros(B, dtype=torch.int32), batch=B,
             n_heads=H, n_kv_heads=G, head_dim=hd, block_size=16, max_blocks_per_seq=maxb, num_blocks=blocks, scale=0.1,
             out=torch.zeros((B, H, hd), dtype=torch.float16), workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    return {**a, **over}


def test_attention_arrays(gpu, no_library):
    good = attention()
    for name in ("q", "out"):
        t = good[name]
        for bad in (t.float(), t.bfloat16(), t[:1], t[:, :, ::2], torch.zeros((2, 64, 8), dtype=torch.float16).transpose(1, 2)):
            refused(name, ql.ql_paged_attn_decode_kv4, **{k: gpu(v) if torch.is_tensor(v) else v
                                                          for k, v in attention(**{name: bad}).items()})
    table, lens = good["block_tables"], good["context_lens"]
    for name, bad in (("block_tables", table.long()), ("block_tables", table[:1]), ("block_tables", torch.zeros((3, 2), dtype=torch.int32).t()),
                      ("context_lens", lens.long()), ("context_lens", lens[:1]), ("context_lens", torch.zeros(4, dtype=torch.int32)[::2]),
                      ("pool", good["pool"][:4]), ("pool", good["pool"][:, :1]), ("workspace", torch.zeros(1 << 21, dtype=torch.uint8)[::2])):
        refused(name, ql.ql_paged_attn_decode_kv4, **{k: gpu(v) if torch.is_tensor(v) else v
                                                      for k, v in attention(**{name: bad}).items()})


def test_host_tensors(gpu, no_library):
    k, slots = torch.zeros((3, 2, 64)), torch.zeros(3, dtype=torch.int64)
    pool = torch.zeros((2, 2, 1280), dtype=torch.uint8)
    for host in range(4):
        t = [x if i == host else gpu(x) for i, x in enumerate((k, k, slots, pool))]
        refused("GPU", ql.ql_kv4_write, t[0], t[1], t[2], 2, 64, t[3], 2)
        refused("GPU", ql.ql_kv4_read, t[3], t[2], 2, 64, 2, t[0], t[1])
    for host in ("q", "pool", "block_tables", "context_lens", "out", "workspace"):
        refused("GPU", ql.ql_paged_attn_decode_kv4, **{n: gpu(v) if torch.is_tensor(v) and n != host else v
                                                       for n, v in attention().items()})
    f, i = torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    args = dict(logits=torch.zeros((4, 9)), uniform=f, tokens=i, temperature=f, top_k=i, top_p=f, min_p=f, probs=f.clone(), active=i.clone())
    for host in args:
        refused("GPU", ql.ql_sample, **{n: v if n == host else gpu(v) for n, v in args.items()})


def test_a_tensor_on_another_gpu(no_library, monkeypatch, gpu):
    from quantized_transformer_decode_ql_gb300 import _lib
    monkeypatch.setattr(_lib, "_current_device", lambda: 1)
    refused("GPU", ql.ql_paged_attn_decode_kv4, **{n: gpu(v) if torch.is_tensor(v) else v for n, v in attention().items()})


def test_model_sampling_arrays_on_the_host(gpu, no_library):
    m = DeviceModel.__new__(DeviceModel)
    m.handle, m._sampling, m._graph_sampling = None, None, {}
    u, f = torch.zeros((2, 5)), torch.zeros(2)
    for over in (dict(uniform=u), dict(uniform=gpu(u), temperature=f), dict(uniform=gpu(u), min_p=f)):
        refused("GPU", m.ql_model_set_sampling, **over)
    assert m._sampling is None


def test_addresses_pass_the_checks(gpu, monkeypatch):
    """As everywhere else in the binding a plain address stands for an array; the sizes are then the caller's."""
    import quantized_transformer_decode_ql_gb300 as m

    class Library:
        called = 0

        def ql_paged_attn_decode_kv4(self, *a):
            Library.called += 1
            return 0
        ql_kv4_write = ql_kv4_read = ql_paged_attn_decode_kv4
    monkeypatch.setattr(m, "lib", Library)
    ql.ql_paged_attn_decode_kv4(**attention(q=64, pool=64, block_tables=64, context_lens=64, out=64, workspace=gpu(torch.zeros(64))), stream=5)
    k, slots = gpu(torch.zeros((3, 2, 64))), gpu(torch.zeros(3, dtype=torch.int64))
    ql.ql_kv4_write(k, k, slots, 2, 64, 4096, 1 << 20, stream=5)
    ql.ql_kv4_read(4096, slots, 2, 64, 1 << 20, k, k, stream=5)
    ql.ql_kv4_write(k, k, slots, 2, 64, gpu(torch.zeros((2, 2, 1280), dtype=torch.uint8)), 2, stream=5)
    assert Library.called == 4


def test_misaligned_tables_and_lengths():
    for table, lens in ((66, 64), (64, 65), (67, 66)):
        assert ql.lib().ql_paged_attn_decode_kv4(64, 1024, table, lens, 1, 8, 8, 128, 16, 4, 9, 0.1, 64, 64, 1 << 40, None) == ql.QL_EINVAL
        assert "misaligned" in ql.lib().ql_last_error().decode()


def test_sampled_outputs_that_overlap():
    """(Pointers only: nothing is launched.)"""
    L, B, V = ql.lib(), 8, 100

    def status(**over):
        a = dict(logits=1 << 20, temperature=0x1000, top_k=0x2000, top_p=0x3000, min_p=0x4000, uniform=0x5000, active=0x6000,
                 tokens=0x7000, probs=0x8000)
        a.update(over)
        return L.ql_sample(a["logits"], ql.QL_DTYPE_F32, V + 3, B, V, a["temperature"], a["top_k"], a["top_p"], a["min_p"], a["uniform"],
                           a["active"], a["tokens"], a["probs"], None)
    end = (1 << 20) + ((B - 1) * (V + 3) + V) * 4
    for out in ("tokens", "probs"):
        for at in [0x1000 * i + d for i in range(1, 7) for d in (-28, 0, 28)] + [(1 << 20) - 28, end - 4]:
            assert status(**{out: at}) == ql.QL_EINVAL and "overlap" in L.ql_last_error().decode(), (out, hex(at))
    assert status(tokens=0x8000) == ql.QL_EINVAL and status(probs=0x7000 + 28) == ql.QL_EINVAL


def test_rows_of_another_type(gpu, no_library):
    slots, pool = gpu(torch.zeros(3, dtype=torch.int64)), gpu(torch.zeros((2, 2, 1280), dtype=torch.uint8))
    k = torch.zeros((3, 2, 64))
    for a, b in ((k.long(), k.long()), (k, k.half()), (k.bfloat16(), k.bfloat16()), (k.double(), k.double())):
        for _ in range(2):
            refused("float32", ql.ql_kv4_write, gpu(a), gpu(b), slots, 2, 64, pool, 2)
            refused("float32", ql.ql_kv4_read, pool, slots, 2, 64, 2, gpu(a), gpu(b))
