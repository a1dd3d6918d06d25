"""The kernel for more than 64 query rows that are fp32, or of 256 coordinates: types, codes, ragged rows, ranges of several
streams, bad pages and lengths, spoiled queries, softmax scales, page offsets beyond 32 bits, more sequences than a launch.

Tolerances are those of the other attention tests.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_cache8 import Setup, _check_attention, _i32
from tests.test_gpu_cache8_paths import _attend, _check_large, _filled, _queries

pytestmark = pytest.mark.gpu
tq = pytest.importorskip("kv_cache_vector_rope_b200")

# code, d, query heads per KV head, rows (products: not multiples of 16 or 128, or just that), query and output types
ROWS = [("e4m3", 64, 1, 65, "f32", "f32"), ("int8", 64, 3, 43, "f32", "f32"), ("int8", 64, 2, 64, "bf16", "f32"),
        ("e4m3", 64, 5, 27, "f32", "bf16"), ("e4m3", 128, 2, 129, "f32", "f32"), ("int8", 128, 1, 77, "f32", "f32"),
        ("int8", 128, 4, 17, "bf16", "f32"), ("e4m3", 128, 7, 19, "f32", "bf16"), ("e4m3", 256, 1, 65, "f32", "f32"),
        ("int8", 256, 2, 41, "f32", "f32"), ("e4m3", 256, 3, 50, "bf16", "bf16"), ("int8", 256, 1, 257, "bf16", "bf16"),
        ("e4m3", 256, 2, 35, "bf16", "f32"), ("int8", 256, 5, 14, "f32", "bf16")]


@pytest.mark.parametrize("code,d,group,nq,qd,od", ROWS)
def test_types_codes_and_ragged_rows(code, d, group, nq, qd, od):
    lens = [321, 1, 0, 16, 47, 128, 2, 63, 65]
    s = _filled(lens, 2, d, 16, code, nq)
    q = _queries(s, len(lens), nq, 2 * group, d, qd)
    for causal, window in ((True, 0), (True, 37), (False, 0)):
        out, lse = _attend(s, q, lens, od, causal=causal, window=window)
        _check_attention(s, q, lens, out, lse, od, causal=causal, window=window)
        again, _ = _attend(s, q, lens, od, causal=causal, window=window)
        assert torch.equal(again, out)
    assert int(s.status.item()) == 0


@pytest.mark.parametrize("b,hkv,group,nq,n,d,block,code,window,dtype", [
    (9, 8, 2, 70, 2500, 64, 128, "int8", 0, "f32"), (40, 8, 1, 90, 700, 64, 16, "e4m3", 0, "f32"),
    (9, 8, 4, 65, 1500, 128, 32, "e4m3", 513, "f32"), (24, 8, 1, 129, 600, 128, 64, "int8", 0, "f32"),
    (9, 6, 2, 70, 1200, 256, 16, "int8", 0, "f32"), (24, 8, 1, 66, 600, 256, 64, "e4m3", 100, "bf16"),
    (2, 2, 4, 300, 5000, 256, 128, "e4m3", 0, "bf16")])
def test_ranges_of_several_streams_a_cta(b, hkv, group, nq, n, d, block, code, window, dtype):
    rg = np.random.default_rng(n)
    lens = [n] + [int(x) for x in rg.integers(1, n + 1, b - 1)]
    s = Setup(n + d, lens, hkv, d, block, code)
    s.write(lens, [0] * b, scale=2.0)
    q = _queries(s, b, nq, hkv * group, d, dtype)
    ws = tq.cache8_attention_workspace(s.cache, b, hkv * group, nq)
    out, lse = _attend(s, q, lens, dtype, ws=ws, window=window)
    assert int(s.status.item()) == 0
    _check_large(s.cache, s.dtable, q, lens, out, lse, dtype, window=window)
    for _ in range(3):
        again, _ = _attend(s, q, lens, dtype, ws=ws, window=window)
        assert torch.equal(again, out)


@pytest.mark.parametrize("d,dtype,code", [(64, "f32", "e4m3"), (128, "f32", "int8"), (256, "bf16", "e4m3"), (256, "f32", "int8")])
def test_bad_pages_and_lengths(d, dtype, code):
    s = _filled([200, 200], 2, d, 32, code)
    bad = s.table.copy()
    bad[0, 2], bad[1, 0] = -7, s.cache.k.shape[0]
    bad[1, 6] = 1 << 30
    q = _queries(s, 2, 70, 4, d, dtype)
    out, lse = _attend(s, q, [200, 200], dtype, table=bad)
    assert int(s.status.item()) == tq.TQ_DEV_BAD_BLOCK
    _check_attention(s, q, [200, 200], out, lse, dtype, table=bad)
    s.status.zero_()
    gone = s.table.copy()
    gone[:, :3] = -1                                                 # behind every row's window
    out, lse = _attend(s, q, [200, 200], dtype, table=gone, window=20)
    assert int(s.status.item()) == 0
    _check_attention(s, q, [200, 200], out, lse, dtype, table=gone, window=20)
    out, lse = _attend(s, q, [10 ** 6, -3], dtype)
    assert int(s.status.item()) & tq.TQ_DEV_BAD_LENGTH
    assert bool((out[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())


@pytest.mark.parametrize("code,d,dtype", [("int8", 64, "f32"), ("e4m3", 128, "f32"), ("e4m3", 256, "bf16"), ("int8", 256, "f32")])
def test_queries_that_are_not_numbers_spoil_their_own_rows_only(code, d, dtype):
    lens, nq = [300, 40], 66
    s = _filled(lens, 2, d, 16, code)
    q = _queries(s, 2, nq, 4, d, dtype).contiguous()
    good, _ = _attend(s, q, lens, dtype)
    _check_attention(s, q, lens, good, None, dtype)
    q[0, 1, nq - 1, 7] = float("nan")
    q[1, 2, 0, d - 1] = float("inf")                                 # row 0 of 66 sees none of 40 keys
    q[1, 3, 50, 5] = -float("inf")
    out, lse = _attend(s, q, lens, dtype)
    spoilt = torch.zeros(2, 4, nq, dtype=torch.bool, device="cuda")
    spoilt[0, 1, nq - 1] = spoilt[1, 3, 50] = True
    seen = torch.isfinite(lse) | torch.isneginf(lse)
    assert torch.equal(~seen, spoilt)
    assert bool(torch.isnan(out[spoilt]).all()) and torch.equal(out[~spoilt], good[~spoilt])
    assert bool((out[1, 2, 0] == 0).all())


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.5])
@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "f32"), (256, "f32"), (256, "bf16")])
def test_any_softmax_scale(d, dtype, scale):
    lens = [150, 33]
    s = _filled(lens, 1, d, 32, "e4m3")
    q = _queries(s, 2, 70, 2, d, dtype)
    out, lse = _attend(s, q, lens, dtype, scale=scale)
    _check_attention(s, q, lens, out, lse, dtype, scale=scale)


@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "f32"), (256, "bf16")])
def test_more_sequences_than_one_launch_takes(d, dtype):
    b, nq = 600, 66
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 40, b)]
    s = Setup(4, [max(n, 1) for n in lens], 1, d, 16, "int8")
    s.write(lens, [0] * b)
    q = _queries(s, b, nq, 1, d, dtype)
    out, lse = _attend(s, q, lens, dtype)
    assert int(s.status.item()) == 0
    _check_attention(s, q, lens, out, lse, dtype)


@pytest.mark.parametrize("d,dtype", [(64, "f32"), (128, "f32"), (256, "bf16")])
def test_pages_beyond_32_bits(d, dtype):
    heads, block = 4, 128
    last = (1 << 32) // (heads * block * d)
    n = last + 64
    cache = tq.Cache8(torch.empty(n, heads, block, d, dtype=torch.uint8, device="cuda"),
                      torch.empty(n, heads, block, d, dtype=torch.uint8, device="cuda"),
                      torch.zeros(n, heads, device="cuda"), torch.zeros(n, heads, device="cuda"), "e4m3")
    table = _i32([[n - 1, 0, n - 2, last]])
    rg = np.random.default_rng(2)
    x = [torch.from_numpy(rg.standard_normal((400, heads, d))).to(torch.bfloat16).cuda() for _ in range(2)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_cache8_write(cache, x[0], x[1], _i32([0, 400]), _i32([0]), block_table=table, d_status=st)
    small = tq.alloc_cache8(4, heads, block, d, "e4m3")
    tq.tq_cache8_write(small, x[0], x[1], _i32([0, 400]), _i32([0]), block_table=_i32([[0, 1, 2, 3]]))
    q = torch.from_numpy(rg.standard_normal((1, heads, 70, d))).to(torch.float32 if dtype == "f32" else torch.bfloat16).cuda()
    a, b = torch.empty_like(q), torch.empty_like(q)
    ws = tq.cache8_attention_workspace(cache, 1, heads, 70)
    tq.tq_cache8_attention(cache, q, _i32([400]), a, ws, block_table=table, d_status=st)
    tq.tq_cache8_attention(small, q, _i32([400]), b, ws, block_table=_i32([[0, 1, 2, 3]]), d_status=st)
    assert torch.equal(a, b) and int(st.item()) == 0
