"""ql_mla_append refuses outputs that overlap any of its inputs (addresses only: nothing is launched, no GPU)."""
import pytest

import quantized_transformer_decode_ql_gb300 as ql

N, HEADS, HD, RANK, BLOCKS, MOST = 4, 8, 128, 512, 9, 100


def address(k):
    return (k + 1) << 30


GOOD = dict(q=address(0), kv=address(1), dtype=ql.QL_DTYPE_F32, qs=HEADS * (HD + 64), ks=RANK + 64, norm=address(2), cos=address(3), sin=address(4),
            pos=address(5), slots=address(6), eps=1e-6, n=N, heads=HEADS, hd=HD, rank=RANK, rope=64, q_out=address(7), pool=address(8), blocks=BLOCKS,
            most=MOST, stream=None)
BYTES = dict(q=N * HEADS * (HD + 64) * 4, kv=N * (RANK + 64) * 4, norm=RANK * 4, cos=MOST * 32 * 4, sin=MOST * 32 * 4, pos=N * 4, slots=N * 8)
OUT = dict(q_out=N * HEADS * (HD + 64) * 2, pool=BLOCKS * 16 * (RANK + 64) * 2)


@pytest.mark.parametrize("out", sorted(OUT))
@pytest.mark.parametrize("name", sorted(BYTES))
def test_append_outputs_over_an_input(out, name):
    L = ql.lib()
    # the same place, the input's last 16 bytes, the output's last 16 bytes
    for at in (GOOD[name], GOOD[name] + (BYTES[name] - 16) // 16 * 16, GOOD[name] - OUT[out] + 16):
        assert L.ql_mla_append(*{**GOOD, out: at}.values()) == ql.QL_EINVAL, (out, name, at - GOOD[name])
        assert "overlap" in L.ql_last_error().decode()


def test_append_output_over_the_last_reachable_table_row():
    """Sizes whose product passes 64 bits do not hide an overlap: positions reach 2^31 rows."""
    L = ql.lib()
    for most in (1 << 31, 1 << 62):
        assert L.ql_mla_append(*{**GOOD, "cos": 1 << 46, "most": most, "pool": (1 << 46) + (1 << 38) - (1 << 20)}.values()) == ql.QL_EINVAL
        assert "overlap" in L.ql_last_error().decode()
