"""The latent attention's workspaces are as large as the heads that there are need (sizes only, no GPU)."""
import pytest

import quantized_transformer_decode_ql_gb300 as ql


@pytest.mark.parametrize("rank", [256, 512])
@pytest.mark.parametrize("heads", [1, 5, 31, 32, 33, 64, 65, 200])
@pytest.mark.parametrize("batch", [1, 40, 4096])
def test_decode(batch, heads, rank):
    """Absorbed queries (two f16 numbers for each up to 32 heads), and a part of the answer in f32, with its reference and sum, for each
    sequence and each of up to 161 windows, over the heads, or over groups of 64."""
    per, groups = (heads, 1) if heads <= 64 else (64, -(-heads // 64))
    parts = groups * (batch + 160 // groups + 1) * per
    need = batch * heads * (rank + 64) * (4 if heads <= 32 else 2) + parts * (4 * rank + 8)
    got = ql.ql_mla_decode_workspace_bytes(batch, heads, 128, rank, 64)
    assert need <= got <= need + 1024
