"""Limits and overlaps that the 8-bit cache's entry points refuse, on each side of the border (CPU: nothing is launched)."""
import ctypes

import pytest

import kv_cache_vector_rope_b200 as tq
from tests.test_cache8_host import INVALID, UNSUPPORTED, WORKSPACE, _attend, _cache, _rows


def _overlap(status):
    return status == INVALID and b"overlap" in tq._lib.tq_last_error_string()


# A call that nothing else is wrong with is refused for its workspace, which comes behind the strides: nothing is launched.
@pytest.mark.parametrize("batch,hq,nq,obs,ohs,ors,overlaps", [
    (2, 32, 1, 128, 128, 4096, True),          # a batch stride of one row, 32 heads
    (2, 32, 1, 4096, 128, 128, False),         # [batch, heads, d]
    (2, 32, 1, 4088, 128, 128, True),
    (2, 32, 1, 128, 256, 128, False),          # [heads, batch, d]
    (3, 32, 1, 128, 256, 128, True),
    (2, 32, 3, 32 * 3 * 128, 128, 4096, False),     # [batch, rows, heads, d]
    (2, 32, 3, 32 * 3 * 128 - 8, 128, 4096, True),
    (2, 32, 3, 128, 256, 32 * 256, False),     # [rows, heads, batch, d]
    (2, 32, 3, 4096, 128, 8192, False),        # [rows, batch, heads, d]
    (2, 32, 3, 4096, 128, 8184, True),
    (1, 32, 1, 0, 128, 0, False),              # strides of dimensions of one index are not looked at
    (2, 32, 1, 0, 128, 128, True),
    (2, 32, 1, 136 * 32, 136, 136, False),     # a wider tensor's slice
    (2, 32, 3, 1 << 62, 1 << 61, 128, True)])  # beyond 64 bits
def test_rows_of_out_that_overlap(batch, hq, nq, obs, ohs, ors, overlaps):
    st = _attend(batch=batch, hq=hq, nq=nq, qrs=4096, obs=obs, ohs=ohs, ors=ors, ws=0)
    assert _overlap(st) if overlaps else st == WORKSPACE


@pytest.mark.parametrize("n,kts,khs,overlaps", [(4, 1024, 128, False), (4, 1016, 128, True), (4, 128, 512, False),
                                                (5, 128, 512, True), (1, 0, 128, False), (4, 0, 128, True)])
def test_rows_read_that_overlap(n, kts, khs, overlaps):
    # The launch itself is kept away by rows of v that are not aligned, which are looked at behind those of k.
    st = _rows(tq._lib.tq_cache8_read, _cache(), n=n, kts=kts, khs=khs, v=0x2008)
    assert st == INVALID and (b"overlap" in tq._lib.tq_last_error_string()) == overlaps


def test_bytes_of_sizes_that_no_call_takes():
    f = tq.tq_cache8_bytes
    assert f(128, 8, 64, 10) == 2 * 10 * 8 * (64 * 128 + 4) and f(16, 1, 16, 0) == 0
    most = 2 * 65000 * ((1 << 31) - 1) * (128 * 256 + 4)
    assert most < 1 << 63 < 2 * 65535 * ((1 << 31) - 1) * (128 * 256 + 4)
    assert f(256, 65000, 128, (1 << 31) - 1) == most and f(256, 65535, 128, (1 << 31) - 1) == -1
    for bad in ((128, 8, 48, 10), (128, 8, 0, 10), (128, 8, -16, 10), (128, 8, 256, 10), (128, 70000, 64, 10), (128, 65536, 64, 1),
                (128, 0, 64, 10), (128, -1, 64, 10), (128, 8, 64, 1 << 60), (128, 8, 64, 1 << 31), (128, 8, 64, -1),
                (100, 8, 64, 10), (272, 8, 64, 10), (0, 8, 64, 10)):
        assert f(*bad) == -1, bad
        assert b"tq_cache8_bytes" in tq._lib.tq_last_error_string()
