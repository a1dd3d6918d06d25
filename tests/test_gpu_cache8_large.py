"""Calls of the 8-bit cache's attention near its limits: wide tables, many row tiles."""
import pytest
import torch

from tests.test_gpu_cache8 import DT, Setup, _check_attention, _i32
from tests.test_gpu_cache8_paths import _check_large

pytestmark = pytest.mark.gpu
tq = pytest.importorskip("kv_cache_vector_rope_b200")


@pytest.mark.parametrize("code,d,heads,nq,dtype", [("e4m3", 128, 8, 1, "bf16"), ("int8", 64, 16, 3, "f32"), ("e4m3", 128, 8, 70, "bf16"),
                                                   ("int8", 64, 8, 70, "f32")])
def test_short_sequences_under_a_table_of_2_to_the_29_tokens(code, d, heads, nq, dtype):
    # 2^22 units of 128 keys or more x 8 heads and more of a sequence that has room for them, 300 keys in it.
    lens = [300, 17]
    s = Setup(d + nq, lens, heads, d, 16, code)
    s.write(lens, [0, 0])
    table = torch.full((2, 1 << 25), -1, dtype=torch.int32, device="cuda")
    table[:, :s.table.shape[1]] = s.dtable
    q = torch.from_numpy(s.rg.standard_normal((2, 2 * heads, nq, d))).to(DT[dtype]).cuda()
    out, lse = torch.empty_like(q), torch.empty(2, 2 * heads, nq, device="cuda")
    ws = tq.cache8_attention_workspace(s.cache, 2, 2 * heads, nq)
    tq.tq_cache8_attention(s.cache, q, _i32(lens), out, ws, block_table=table, lse_out=lse, d_status=s.status)
    assert int(s.status.item()) == 0
    _check_attention(s, q, lens, out, lse, dtype)


def test_a_prompt_beyond_2_to_the_25_units():
    # 65536 rows of 2 x 4 heads over 65536 keys: 1024 row tiles x 517 units x 2 heads, and a table eight times as wide.
    n, d, heads, group = 65536, 64, 2, 4
    s = Setup(1, [n], heads, d, 128, "e4m3")
    s.write([n], [0])
    table = torch.full((1, 40000), -1, dtype=torch.int32, device="cuda")
    table[:, :s.table.shape[1]] = s.dtable
    q = torch.randn(1, heads * group, n, d, device="cuda").to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(1, heads * group, n, device="cuda")
    ws = tq.cache8_attention_workspace(s.cache, 1, heads * group, n)
    tq.tq_cache8_attention(s.cache, q, _i32([n]), out, ws, block_table=table, lse_out=lse, d_status=s.status)
    assert int(s.status.item()) == 0
    for r0, r1 in ((0, 40), (30000, 30060), (n - 40, n)):
        # The same rows as the newest of a shorter sequence.
        _check_large(s.cache, s.dtable, q[:, :, r0:r1].contiguous(), [r1], out[:, :, r0:r1], lse[:, :, r0:r1], "bf16")
    assert bool(torch.isfinite(out).all())
