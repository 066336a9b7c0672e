"""Refusals of the latent attention's entry points that need no GPU: tensors of another type, too small, not contiguous or on the
host never reach the library; sizes, alignments and overlaps that the library refuses before it touches a device."""
import math

import pytest
import torch

import quantized_transformer_decode_ql_gb300 as ql


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
    return lambda a: {k: v.as_subclass(Gpu) if torch.is_tensor(v) else v for k, v in a.items()}


@pytest.fixture
def no_library(monkeypatch):
    """Nothing may get past the checks."""
    import quantized_transformer_decode_ql_gb300 as m

    def called():
        raise AssertionError("the library was called")
    monkeypatch.setattr(m, "lib", called)


N, HEADS, HD, RANK, BLOCKS, MAXB = 3, 5, 64, 256, 4, 2
HALF, WHOLE = torch.float16, torch.int32


def append(**over):
    return {**dict(q=torch.zeros((N, HEADS, HD + 64)), kv=torch.zeros((N, RANK + 64)), norm_w=torch.zeros(RANK), cos_t=torch.zeros((9, 32)),
                   sin_t=torch.zeros((9, 32)), positions=torch.zeros(N, dtype=WHOLE), slots=torch.zeros(N, dtype=torch.int64), eps=1e-6,
                   n_heads=HEADS, head_dim=HD, rank=RANK, rope_dim=64, q_out=torch.zeros((N, HEADS, HD + 64), dtype=HALF),
                   pool=torch.zeros((BLOCKS, 16, RANK + 64), dtype=HALF), num_blocks=BLOCKS, max_position=9), **over}


def decode(**over):
    return {**dict(q=torch.zeros((N, HEADS, HD + 64), dtype=HALF), w_kv=torch.zeros((HEADS, 2 * HD, RANK), dtype=HALF),
                   pool=torch.zeros((BLOCKS, 16, RANK + 64), dtype=HALF), block_tables=torch.zeros((N, MAXB), dtype=WHOLE),
                   context_lens=torch.zeros(N, dtype=WHOLE), batch=N, n_heads=HEADS, head_dim=HD, rank=RANK, rope_dim=64, block_size=16,
                   max_blocks_per_seq=MAXB, num_blocks=BLOCKS, scale=0.1, out=torch.zeros((N, HEADS, HD), dtype=HALF),
                   workspace=torch.zeros(1 << 10, dtype=torch.uint8)), **over}


def chunk(**over):
    a = decode()
    a.pop("batch")
    a["block_table"], a["position"], a["n_tokens"] = a.pop("block_tables")[:1], a.pop("context_lens")[:1], N
    return {**a, **over}


APPEND = [("norm_w", append()["norm_w"].half()), ("norm_w", torch.zeros(RANK - 1)), ("cos_t", torch.zeros((8, 32))), ("sin_t", torch.zeros((9, 64))[:, ::2]),
          ("positions", torch.zeros(N, dtype=torch.int64)), ("positions", torch.zeros(N - 1, dtype=WHOLE)), ("slots", torch.zeros(N, dtype=WHOLE)),
          ("slots", torch.zeros(2 * N, dtype=torch.int64)[::2]), ("pool", torch.zeros((BLOCKS, 16, RANK + 64))),
          ("pool", torch.zeros((BLOCKS - 1, 16, RANK + 64), dtype=HALF)), ("q_out", torch.zeros((N, HEADS, HD + 64))),
          ("q_out", torch.zeros((N, HEADS, HD), dtype=HALF))]


@pytest.mark.parametrize("name,bad", APPEND, ids=range(len(APPEND)))
def test_append_arrays(gpu, no_library, name, bad):
    refused(name, ql.ql_mla_append, **gpu(append(**{name: bad})))


def test_append_rows(gpu, no_library):
    refused("float32", ql.ql_mla_append, **gpu(append(q=torch.zeros((N, HEADS, HD + 64), dtype=HALF))))
    refused("float32", ql.ql_mla_append, **gpu(append(kv=torch.zeros((N, RANK + 64), dtype=torch.bfloat16), q=None, q_out=None)))
    refused("together", ql.ql_mla_append, **gpu(append(q=None)))
    refused("together", ql.ql_mla_append, **gpu(append(q_out=None)))
    for bad in (torch.zeros((N, HEADS, HD)), torch.zeros((N + 1, HEADS, HD + 64)), torch.zeros((N, HEADS, 2 * HD + 128))[:, :, ::2]):
        refused("rows", ql.ql_mla_append, **gpu(append(q=bad)))
    for bad in (torch.zeros((N, RANK)), torch.zeros((N, 2 * RANK + 128))[:, ::2]):
        refused("rows", ql.ql_mla_append, **gpu(append(kv=bad)))


@pytest.mark.parametrize("make,call", [(decode, "ql_mla_attn_decode"), (chunk, "ql_mla_attn_chunk")])
def test_attention_arrays(gpu, no_library, make, call):
    good = make()
    table, lens = ("block_tables", "context_lens") if make is decode else ("block_table", "position")
    for name, word in (("q", "q"), ("w_kv", "w_kv"), ("pool", "pool"), ("out", "out"), (table, "table"), (lens, "lengths")):
        t = good[name]
        wide = torch.zeros((*t.shape[:-1], 2 * t.shape[-1]), dtype=t.dtype)[..., ::2]
        for bad in (t.float(), t.flatten()[1:], *([wide] if t.numel() > 1 else [])):
            refused(word, getattr(ql, call), **gpu(make(**{name: bad})))
    refused("contiguous", getattr(ql, call), **gpu(make(workspace=torch.zeros(1 << 11, dtype=torch.uint8)[::2])))


@pytest.mark.parametrize("make,call", [(append, "ql_mla_append"), (decode, "ql_mla_attn_decode"), (chunk, "ql_mla_attn_chunk")])
def test_host_tensors_and_another_gpu(gpu, no_library, monkeypatch, make, call):
    names = [k for k, v in make().items() if torch.is_tensor(v)]
    for host in names:
        refused("GPU", getattr(ql, call), **{**gpu(make()), host: make()[host]})
    from quantized_transformer_decode_ql_gb300 import _lib
    monkeypatch.setattr(_lib, "_current_device", lambda: 1)
    refused("GPU", getattr(ql, call), **gpu(make()))


# ---------------------------------------------------------------- the library (addresses only: nothing is launched)
def address(k):
    return (k + 1) << 30


def attention(call, **over):
    a = dict(q=address(0), w=address(1), pool=address(2), table=address(3), lens=address(4), rows=2, heads=8, hd=128, rank=512, rope=64, block=16,
             maxb=4, blocks=9, scale=0.1, out=address(5), ws=address(6), size=1 << 40, stream=None)
    assert set(over) <= set(a)
    return getattr(ql.lib(), call)(*{**a, **over}.values())


BAD = [dict(hd=96), dict(hd=256), dict(rank=128), dict(rank=384), dict(rope=32), dict(block=32), dict(rows=0), dict(rows=65536), dict(heads=0),
       dict(heads=1025), dict(rows=65535, heads=65), dict(maxb=0), dict(blocks=0), dict(blocks=1 << 27), dict(scale=0.0), dict(scale=-1.0),
       dict(scale=math.inf), dict(scale=math.nan), dict(size=1000), dict(q=None), dict(w=None), dict(pool=None), dict(table=None), dict(lens=None),
       dict(out=None), dict(ws=None), dict(q=address(0) + 8), dict(w=address(1) + 2), dict(pool=address(2) + 4), dict(table=address(3) + 2),
       dict(lens=address(4) + 1), dict(out=address(5) + 8), dict(ws=address(6) + 64), dict(out=address(0)), dict(out=address(1) + 16),
       dict(out=address(2)), dict(ws=address(2)), dict(ws=address(5)), dict(ws=address(4)), dict(out=address(3))]


@pytest.mark.parametrize("call", ["ql_mla_attn_decode", "ql_mla_attn_chunk"])
@pytest.mark.parametrize("bad", BAD, ids=[" ".join(f"{k}={v}" for k, v in b.items()) for b in BAD])
def test_attention_refusals(call, bad):
    assert attention(call, **bad) == ql.QL_EINVAL and call in ql.lib().ql_last_error().decode()


def test_tables_too_long():
    assert attention("ql_mla_attn_decode", maxb=(1 << 20) + 1) == ql.QL_EINVAL
    assert attention("ql_mla_attn_decode", rows=5000, maxb=1 << 20) == ql.QL_EINVAL
    assert attention("ql_mla_attn_chunk", maxb=(1 << 16) + 1) == ql.QL_EINVAL


def test_workspace_sizes():
    for size, most in ((ql.ql_mla_decode_workspace_bytes, 1 << 20), (ql.ql_mla_chunk_workspace_bytes, 1 << 16)):
        assert size(1, 8, 128, 512, most) > 0 and size(1, 8, 128, 512, most + 1) == 0
        assert size(0, 8, 128, 512, 4) == size(1, 0, 128, 512, 4) == size(1, 8, 96, 512, 4) == size(1, 8, 128, 100, 4) == size(1, 8, 128, 512, 0) == 0
        assert size(40, 8, 64, 256, 100) >= size(4, 8, 64, 256, 100)


def test_append_refusals():
    L = ql.lib()
    good = dict(q=address(0), kv=address(1), dtype=ql.QL_DTYPE_F32, qs=8 * 192, ks=576, norm=address(2), cos=address(3), sin=address(4), pos=address(5),
                slots=address(6), eps=1e-6, n=4, heads=8, hd=128, rank=512, rope=64, q_out=address(7), pool=address(8), blocks=9, most=100, stream=None)
    for bad in (dict(dtype=2), dict(hd=96), dict(rank=300), dict(rope=128), dict(n=-1), dict(n=1 << 31), dict(heads=0), dict(heads=1025), dict(blocks=0),
                dict(most=0), dict(kv=None), dict(norm=None), dict(cos=None), dict(pos=None), dict(slots=None), dict(pool=None), dict(q=None),
                dict(q_out=None), dict(qs=8 * 192 - 4), dict(qs=8 * 192 + 2), dict(ks=572), dict(ks=578), dict(q=address(0) + 8), dict(kv=address(1) + 4),
                dict(norm=address(2) + 4), dict(cos=address(3) + 4), dict(slots=address(6) + 4), dict(pos=address(5) + 2), dict(q_out=address(7) + 2),
                dict(pool=address(8) + 8), dict(q_out=address(0)), dict(q_out=address(1)), dict(pool=address(0)), dict(pool=address(1)),
                dict(q_out=address(8) + 16)):
        assert L.ql_mla_append(*{**good, **bad}.values()) == ql.QL_EINVAL, bad
        assert "ql_mla_append" in L.ql_last_error().decode()
    assert L.ql_mla_append(*{**good, "n": 0}.values()) == ql.QL_OK


@pytest.mark.parametrize("heads,hd,rank,maxb", [(1, 64, 256, 4096), (3, 128, 512, 2048), (32, 128, 512, 512), (90, 64, 256, 64), (1024, 128, 256, 8)])
def test_chunk_workspace_is_enough_for_fewer_tokens(heads, hd, rank, maxb):
    need = [ql.ql_mla_chunk_workspace_bytes(n, heads, hd, rank, maxb) for n in range(1, 2000)]
    assert need[0] > 0 and all(a <= b for a, b in zip(need, need[1:]))
