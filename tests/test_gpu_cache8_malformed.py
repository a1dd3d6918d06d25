"""Lengths that the arrays do not allow: what is left out, and that nothing else is touched."""
import numpy as np
import pytest
import torch

from oracle import cache8 as o8
from tests.test_gpu_cache8 import Setup, _i32, _np, _same

pytestmark = pytest.mark.gpu
tq = pytest.importorskip("kv_cache_vector_rope_b200")

# cu_tokens, start of three sequences with a capacity of 64 tokens, over 128 rows
MALFORMED = [
    ([0, 64, 128, 128], [40, -1, 0]), ([0, 64, 60, 128], [0, 0, 0]), ([-5, 3, 100, 128], [0, 0, 9]),
    ([0, 0, 500, 520], [0, 50, 0]), ([0, 128, 128, 128], [64, 0, 0]), ([0, 128, 0, 128], [65, 3, 3]),
    ([120, 2 ** 31 - 1, -2 ** 31, 128], [2 ** 31 - 1, 0, -2 ** 31]), ([200, 300, 300, 128], [0, 0, 0]),
    ([0, 40, 80, 120], [30, -2 ** 31, 2 ** 31 - 1])]


def _allowed(cu, start, n, cap):
    """(first row, rows, position) of each sequence that is left of malformed lengths."""
    out = []
    for b, st in enumerate(start):
        lo, hi = cu[b], cu[b + 1]
        if lo < 0 or hi < lo or st < 0:
            out.append((0, 0, 0))
            continue
        lo, hi = min(lo, n), min(hi, n)
        out.append((lo, max(0, min(hi - lo, cap - st)), st))
    return out


@pytest.mark.parametrize("code,dtype", [("e4m3", torch.float32), ("int8", torch.bfloat16)])
@pytest.mark.parametrize("cu,start", MALFORMED)
def test_a_write_leaves_out_what_does_not_fit(cu, start, code, dtype):
    s = Setup(5, [64, 64, 64], 2, 64, 16, code)
    s.write([64, 64, 64], [0, 0, 0])
    ref = s.host()
    x = [torch.from_numpy(np.random.default_rng(i).standard_normal((128, 2, 64))).to(dtype) for i in (1, 2)]
    tq.tq_cache8_write(s.cache, x[0].cuda(), x[1].cuda(), _i32(cu), _i32(start), block_table=s.dtable, d_status=s.status)
    assert int(s.status.item()) == tq.TQ_DEV_BAD_LENGTH
    for b, (row, n, pos) in enumerate(_allowed(cu, start, 128, 64)):
        if n:
            o8.write(ref, _np(x[0])[row:row + n], _np(x[1])[row:row + n], [0, n], [pos], s.table[b:b + 1])
    _same(s.cache, ref)


@pytest.mark.parametrize("code,dtype", [("e4m3", torch.bfloat16), ("int8", torch.float32)])
@pytest.mark.parametrize("cu,start", MALFORMED)
def test_a_read_leaves_out_what_does_not_fit(cu, start, code, dtype):
    s = Setup(6, [64, 64, 64], 2, 64, 16, code)
    s.write([64, 64, 64], [0, 0, 0])
    ref = s.host()
    out = torch.full((130, 2, 64), 9.0, dtype=dtype, device="cuda")
    tq.tq_cache8_read(s.cache, out[1:129], None, _i32(cu), _i32(start), block_table=s.dtable, d_status=s.status)
    assert int(s.status.item()) == tq.TQ_DEV_BAD_LENGTH
    want = np.full((130, 2, 64), 9.0)
    free = np.zeros(130, bool)                                    # rows that two sequences claim may hold either's
    for b, (row, n, pos) in enumerate(_allowed(cu, start, 128, 64)):
        if n:
            free[1 + row:1 + row + n] |= want[1 + row:1 + row + n, 0, 0] != 9.0
            want[1 + row:1 + row + n] = o8.read(ref, [0, n], [pos], s.table[b:b + 1])[0]
    assert np.array_equal(_np(out)[~free], want[~free])


def test_overlapping_lengths_beyond_32_bits_of_blocks():
    # 512 sequences that all claim the same 2^26 rows (one row, repeated), each followed by one whose length falls: 2^31
    # blocks in all, none of which is in the cache.
    n, b = 1 << 26, 1024
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs a block table of 17 GB")
    table = torch.full((b, n // 16), -1, dtype=torch.int32, device="cuda")
    cache = tq.alloc_cache8(4, 1, 16, 16, "int8")
    for t in (cache.k, cache.v):
        t.fill_(77)
    cache.k_scale.fill_(3.0), cache.v_scale.fill_(3.0)
    x = torch.randn(1, 1, 16, device="cuda").to(torch.bfloat16).expand(n, 1, 16)
    cu, st = _i32([0, n] * (b // 2) + [0]), torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_cache8_write(cache, x, x, cu, _i32([0] * b), block_table=table, d_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == tq.TQ_DEV_BAD_LENGTH | tq.TQ_DEV_BAD_BLOCK
    assert bool((cache.k == 77).all()) and bool((cache.v == 77).all())
    assert bool((cache.k_scale == 3).all()) and bool((cache.v_scale == 3).all())
