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


def _size(heads, group, nq, tokens, d=128, dtype=1, code=0):
    """The status of a call over a table of that many tokens that has no workspace: TQ_ERR_WORKSPACE where its sizes are fine."""
    hq = heads * group
    c = _cache(d=d, heads=heads, block=128, code=code, n=1 << 24)
    return _attend(c, hq=hq, nq=nq, qd=dtype, od=dtype, qbs=hq * nq * d, qhs=d, qrs=hq * d, obs=hq * nq * d, ohs=d, ors=hq * d,
                   stride=tokens // 128, ws=0)


@pytest.mark.parametrize("heads,group,nq,tokens,kw,fine", [
    (63, 1, 1, 1 << 30, {}, True), (64, 1, 1, 1 << 30, {}, False),
    (8, 4, 1, 1 << 30, {}, True), (32, 8, 1, 1 << 20, {}, True),
    (8, 4, 262144, 262144, {}, True),                             # a prompt of 262144 tokens in one call
    (8, 4, 1 << 20, 1 << 20, {}, False), (8, 4, 1 << 20, 1 << 16, {}, True),
    (1, 1, 1 << 29, 128, {}, True), (1, 1, 1 << 29, 1 << 20, {}, False),
    (8, 4, 65536, 262144, dict(d=256), True), (8, 4, 1 << 20, 262144, dict(d=256, dtype=0), False),
    (65535, 1, 1, 1 << 19, {}, True), (65535, 1, 1, 1 << 20, {}, False),
    (1, 1, 1, (1 << 30) + 128, {}, False)])
def test_sizes_on_each_side_of_the_limit(heads, group, nq, tokens, kw, fine):
    assert _size(heads, group, nq, tokens, **kw) == (WORKSPACE if fine else UNSUPPORTED)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("code", [0, 1])
def test_what_the_header_names_as_supported_is_taken(d, dtype, code):
    for heads, group, nq in ((1, 1, 1), (8, 4, 1), (3, 5, 7), (2, 8, 8), (4, 13, 5), (8, 4, 2048), (16, 1, 9999)):
        rows = group * nq
        t = -(-rows // (4 if rows <= 64 else 128))
        tokens = min(1 << 30, 64 * ((1 << 30) // (heads * t) - 18)) // 128 * 128
        assert _size(heads, group, nq, tokens, d=d, dtype=dtype, code=code) == WORKSPACE
