"""Latent attention where a number is beyond f16: what is recorded, with which index, and who is spoilt by it."""
import math

import numpy as np
import pytest
import torch

from gpu_util import dev, lib
from oracle import mla
from test_gpu_mla import chunk, latent_case, rows_of

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
    assert "f16" in recorded()
    if at:
        want, bound = mla.attention(c["q"][:at], rows_of(c, 0, row), c["w"], c["scale"], before=before)
        assert np.all(np.abs(got[:at] - want) <= bound)
    # heads whose values f16 holds answer for every query that does not see the row, and for the others as well
    assert np.all(np.isfinite(got[:, 0]))
