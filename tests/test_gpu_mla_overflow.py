"""Latent attention where a number is beyond f16: what is recorded, with which index, and who is spoilt by it."""
import math

import numpy as np
import pytest
import torch

from gpu_util import dev, lib
from oracle import mla
from test_gpu_mla import chunk, decode, latent_case, rows_of

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def record():
    """Each test starts with an empty device error record and leaves none that it has not read."""
    ql = lib()
    try:
        ql.ql_check_device_error()
    except ql.QLError:
        pass
    yield
    ql.ql_check_device_error()


def recorded():
    """The message of the record, which is empty then."""
    ql = lib()
    with pytest.raises(ql.QLError) as e:
        ql.ql_check_device_error()
    assert e.value.status == ql.QL_EDEVICE
    return str(e.value)


@pytest.mark.parametrize("n,before,heads,hd,rank,at", [(300, 50, 3, 64, 256, 150), (300, 50, 3, 128, 512, 0), (600, 0, 5, 64, 512, 599), (129, 700, 2, 128, 256, 70)])
def test_chunk_value_beyond_f16_stays_behind_the_mask(n, before, heads, hd, rank, at):
    """Queries before a token whose value f16 does not hold weigh it with 0."""
    c = latent_case([before + n], heads, hd, rank, rows=n, seed=n)
    row = before + at
    w = c["w"][1, hd + 3].astype(np.float64)
    big = np.sign(w) * math.ceil(80000 / np.abs(w).sum())
    c["pool"][c["table"][0, row // 16], row % 16, :rank] = big
    assert 70000 < big @ w and np.abs(c["w"][:, :hd].astype(np.float64) @ big).max() < 65000
    got = chunk(c, n, before)
    said = recorded()
    assert "key or value" in said and f"(index {row}, value 1)" in said, said
    if at:
        want, bound = mla.attention(c["q"][:at], rows_of(c, 0, row), c["w"], c["scale"], before=before)
        assert np.all(np.abs(got[:at] - want) <= bound)
    # heads whose values f16 holds answer for every query that does not see the row, and for the others as well
    assert np.all(np.isfinite(got[:, 0]))


@pytest.mark.parametrize("hd,heads", [(128, 7), (64, 130)])
@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("what", ["value", "rotated", "nan"])
def test_append_query_beyond_f16_is_recorded(hd, heads, f16, what):
    """One head of one row; written all the same, and no other row or head is spoilt."""
    ql = lib()
    n, row, head, rank = 5, 3, heads - 2, 256
    cos, sin = np.empty((9, 32), np.float32), np.empty((9, 32), np.float32)
    ql.ql_rope_tables(cos, sin, 1e4)
    q = torch.randn((n, heads, hd + 64), device="cuda")
    q[row, head, 11 if what != "rotated" else hd + 5] = math.nan if what == "nan" else 7e4 if what == "value" else 6e4
    if what == "rotated":       # each half is held, their turn by 45 degrees is not
        q[row, head, hd + 37] = 6e4
        cos[4, 5] = sin[4, 5] = math.sqrt(0.5)
    q = q.half() if f16 else q
    kv = torch.randn((n, rank + 64), device="cuda").to(q.dtype)
    pos, slots = torch.tensor([0, 1, 2, 4, 3], dtype=torch.int32, device="cuda"), torch.arange(n, device="cuda")
    pool = torch.zeros((1, 16, rank + 64), dtype=torch.float16, device="cuda")
    q_out = torch.full((n, heads, hd + 64), 9.0, dtype=torch.float16, device="cuda")
    args = (torch.ones(rank, device="cuda"), dev(cos), dev(sin), pos, slots, 1e-6, heads, hd, rank, 64, q_out, pool, 1, 9)
    ql.ql_mla_append(q, kv, *args)
    said = recorded()
    assert f"(index {row}, value {1 + head})" in said, said
    broken = ~torch.isfinite(q_out).all(-1)
    assert broken.sum() == 1 and bool(broken[row, head])
    q[row, head] = 1.0
    ql.ql_mla_append(q, kv, *args)
    ql.ql_check_device_error()


@pytest.mark.parametrize("hd,rank", [(64, 256), (128, 512)])
@pytest.mark.parametrize("at,head,heads", [(1, 1, 2), (13, 0, 3), (31, 30, 32), (70, 39, 40)])
def test_decode_absorbed_query_beyond_f16_names_its_sequence(hd, rank, at, head, heads):
    c = latent_case([5] * (at + 2), heads, hd, rank, seed=at)
    c["q"][at, head, :hd] = 6e4
    c["w"][head, :hd, 7] = np.where(np.arange(hd) < hd // 2, 6e4, 0)
    c["q"][np.arange(at + 2) != at, head, :hd] = 0
    decode(c)
    said = recorded()
    assert "absorbed query" in said and f"(index {at}, value {head})" in said, said


def test_chunk_absorbed_query_beyond_f16_names_its_token():
    c = latent_case([60 + 20], 32, 128, 512, rows=20, seed=1)
    c["q"][:, 9, :128] = 0
    c["q"][17, 9, :128] = 6e4
    c["w"][9, :128, 300] = 6e4
    chunk(c, 20, 60)
    said = recorded()
    assert "absorbed query" in said and "(index 17, value 9)" in said, said


@pytest.mark.parametrize("hd,rank", [(64, 256), (128, 512)])
def test_chunk_key_beyond_f16_names_its_position(hd, rank):
    c = latent_case([90], 3, hd, rank, rows=90, seed=4)
    c["w"][1, 3] = 300.0
    c["pool"][:, :, :rank] = 0.01
    c["pool"][c["table"][0, 4], 9, :rank] = 1.0
    chunk(c, 90, 0)
    said = recorded()
    assert "key or value" in said and "(index 73, value 1)" in said, said


@pytest.mark.parametrize("value,at,form,records", [(math.nan, "latent", "expanded", False), (math.inf, "latent", "expanded", True), (math.inf, "rotated", "expanded", False),
                                                   (math.nan, "latent", "absorbed", False), (math.inf, "latent", "absorbed", False)])
def test_what_a_broken_row_records(value, at, form, records):
    """An infinite latent makes infinite keys, which are recorded; NaN, or a rotated part, is not a number beyond f16."""
    heads, hd, rank, n, before = (3, 64, 256, 60, 50) if form == "expanded" else (32, 128, 512, 20, 50)
    c = latent_case([before + n], heads, hd, rank, rows=n, seed=n)
    row = before + 10
    c["pool"][c["table"][0, row // 16], row % 16, rank - 7 if at == "latent" else rank + 5] = value
    got = chunk(c, n, before)
    assert np.all(np.isfinite(got[:10]))
    if records:
        assert "key or value" in recorded()
