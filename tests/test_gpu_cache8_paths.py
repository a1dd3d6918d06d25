"""The 8-bit cache's attention where its kernels differ: rows per KV head, codes and types, segments and merges, masked
and spoiled inputs, waits that run out, streams and graphs, offsets beyond 32 bits.

Tolerances are those of the other attention tests. Keys whose block scale lies far below the largest of 128 keys lose
bits where many rows go together: their codes, times the ratio, are halves, off by up to half of 2^-24 of the largest
scale r, so a score is off by up to 2^-25 r |scale| sum |q_i| beside the rest, and the outputs by that times 2 spread.
"""
import numpy as np
import pytest
import torch

from oracle import cache8 as o8
from tests.test_gpu_cache8 import DT, HALF, Setup, _check_attention, _i32, _np, _values

pytestmark = pytest.mark.gpu
tq = pytest.importorskip("kv_cache_vector_rope_b200")


def _attend(s, q, lens, od="bf16", ws=None, table=None, **kw):
    b, hq, nq, d = q.shape
    out = torch.full((b, nq, hq, d), 5.0, dtype=DT[od], device="cuda").transpose(1, 2)
    lse = torch.full((b, hq, nq), 5.0, device="cuda")
    ws = tq.cache8_attention_workspace(s.cache, b, hq, nq) if ws is None else ws
    tq.tq_cache8_attention(s.cache, q, _i32(lens), out, ws, block_table=s.dtable if table is None else _i32(table.tolist()),
                           lse_out=lse, d_status=s.status, **kw)
    torch.cuda.synchronize()
    return out, lse


def _queries(s, b, nq, hq, d, dtype, by=1.5):
    return torch.from_numpy(_values(s.rg, b, nq, hq, d) * by).to(DT[dtype]).cuda().transpose(1, 2)


def _filled(lens, heads, d, block, code, seed=0):
    s = Setup(sum(lens) + d + seed, lens, heads, d, block, code)
    half = [n // 2 for n in lens]
    s.write(half, [0] * len(lens))
    s.write([n - h for n, h in zip(lens, half)], half, scale=3.0)
    return s


ROWS = [(code, d, group, nq, qd, od) for code, d, group, nq, qd, od in [
    # up to four rows
    ("int8", 64, 4, 1, "bf16", "bf16"), ("int8", 64, 1, 2, "bf16", "f32"), ("int8", 64, 3, 1, "f32", "bf16"),
    ("int8", 128, 4, 1, "bf16", "f32"), ("int8", 128, 4, 1, "f32", "bf16"), ("int8", 128, 1, 3, "f32", "f32"),
    ("int8", 256, 4, 1, "bf16", "bf16"), ("int8", 256, 2, 2, "bf16", "f32"), ("int8", 256, 1, 1, "f32", "f32"),
    ("int8", 256, 4, 1, "f32", "bf16"), ("e4m3", 64, 1, 1, "f32", "f32"), ("e4m3", 256, 4, 1, "f32", "bf16"),
    # five to eight
    ("int8", 64, 5, 1, "bf16", "bf16"), ("int8", 64, 2, 4, "f32", "f32"), ("int8", 128, 8, 1, "bf16", "bf16"),
    ("int8", 128, 1, 7, "f32", "f32"), ("int8", 256, 3, 2, "bf16", "bf16"), ("int8", 256, 8, 1, "f32", "f32"),
    ("e4m3", 64, 8, 1, "bf16", "f32"), ("e4m3", 128, 4, 2, "f32", "bf16"), ("e4m3", 256, 5, 1, "bf16", "f32"),
    # nine to sixty-four
    ("int8", 64, 3, 3, "bf16", "bf16"), ("int8", 64, 1, 16, "bf16", "bf16"), ("int8", 128, 4, 16, "bf16", "bf16"),
    ("int8", 128, 9, 1, "bf16", "bf16"), ("int8", 256, 4, 5, "bf16", "bf16"), ("e4m3", 64, 4, 16, "bf16", "bf16"),
    ("e4m3", 128, 3, 17, "f32", "f32"), ("e4m3", 64, 1, 33, "f32", "bf16"),
    # more
    ("int8", 128, 4, 33, "bf16", "bf16"), ("int8", 64, 5, 13, "bf16", "bf16"), ("e4m3", 64, 1, 65, "bf16", "bf16"),
    ("e4m3", 128, 3, 90, "bf16", "bf16"), ("e4m3", 128, 1, 70, "bf16", "f32"), ("int8", 256, 1, 70, "bf16", "bf16"),
]]


@pytest.mark.parametrize("code,d,group,nq,qd,od", ROWS)
def test_rows_and_types(code, d, group, nq, qd, od):
    # Lengths around groups of 16, pairs of them, units and tiles; none at all; fewer keys than rows.
    lens = [321, 1, 0, 16, 47, 128, 2]
    s = _filled(lens, 2, d, 16, code, nq)
    q = _queries(s, len(lens), nq, 2 * group, d, qd)
    # Once with a table that cannot hold longer sequences, once with room, where the streams are split between CTAs.
    room = np.full((len(lens), 80), -1, np.int32)
    room[:, :s.table.shape[1]] = s.table
    for table in (s.table, room):
        for window in (0, 37):
            out, lse = _attend(s, q, lens, od, table=table, window=window)
            _check_attention(s, q, lens, out, lse, od, window=window)
    assert int(s.status.item()) == 0


@pytest.mark.parametrize("code,d,nq", [("e4m3", 128, 1), ("int8", 64, 2), ("e4m3", 64, 100), ("int8", 128, 100)])
def test_long_sequences_cut_between_many_ctas(code, d, nq):
    lens = [9001, 63, 4500]
    s = _filled(lens, 1, d, 64, code)
    q = _queries(s, 3, nq, 2, d, "bf16")
    for window in (0, 4097):
        out, lse = _attend(s, q, lens, window=window)
        _check_attention(s, q, lens, out, lse, "bf16", window=window)
    assert int(s.status.item()) == 0


@pytest.mark.parametrize("code,d", [("e4m3", 64), ("int8", 128)])
def test_many_rows_with_scores_that_rise_and_scales_that_jump(code, d):
    n, nq = 1100, 80
    s = Setup(78, [n], 1, d, 16, code)
    k = s.rg.standard_normal((n, 1, d)) * (np.linspace(0.1, 40.0, n) * 2.0 ** (9 * np.sin(np.arange(n) / 40.0)))[:, None, None]
    v = s.rg.standard_normal((n, 1, d)) * 2.0 ** (30.0 * np.sin(np.arange(n) / 90.0))[:, None, None]
    tq.tq_cache8_write(s.cache, torch.from_numpy(k).float().cuda(), torch.from_numpy(v).float().cuda(), _i32([0, n]),
                       _i32([0]), block_table=s.dtable, d_status=s.status)
    q = torch.from_numpy(s.rg.standard_normal((1, 2, nq, d))).to(torch.bfloat16).cuda()
    q[0, 0, 3] *= 1e-30
    q[0, 1, 5] *= 1e3
    q[0, 1, 7] = 0.0
    out, lse = _attend(s, q, [n])
    assert int(s.status.item()) == 0
    ref, rl, A, B, top = o8.attention(s.host(), _np(q), [n], s.table)
    B = B[..., None] + 0.0
    r = float(s.cache.k_scale[s.dtable[0, :-(-n // 16)].long()].max())
    es = ((2 * d / 16 + 8) * 2.0 ** -23 + 2.0 ** -22) * B
    es = es + 2.0 ** -25 * r * np.abs(_np(q)).sum(-1, keepdims=True) / np.sqrt(d)
    ew = es + 2.0 ** -22 + 2 * (2 * B + 20) * 2.0 ** -24 + 2.0 ** -12 + (n / 16 + 40) * 2.0 ** -23
    tol = HALF["bf16"] * np.abs(ref) + 2 * ew * A + n * 2.0 ** -30 * top[..., None]
    assert np.all(np.abs(_np(out) - ref) <= tol)
    assert np.all(np.abs(_np(lse) - rl) <= ew[..., 0] + 2.0 ** -22 * (1 + np.abs(rl)))


def test_many_rows_with_bad_pages_and_lengths():
    s = _filled([200, 200], 2, 128, 32, "e4m3")
    bad = s.table.copy()
    bad[0, 2], bad[1, 0] = -7, s.cache.k.shape[0]
    bad[1, 6] = 1 << 30
    q = _queries(s, 2, 70, 4, 128, "bf16")
    out, lse = _attend(s, q, [200, 200], table=bad)
    assert int(s.status.item()) == tq.TQ_DEV_BAD_BLOCK
    _check_attention(s, q, [200, 200], out, lse, "bf16", table=bad)
    s.status.zero_()
    gone = s.table.copy()
    gone[:, :3] = -1                                                 # behind every row's window
    out, lse = _attend(s, q, [200, 200], table=gone, window=20)
    assert int(s.status.item()) == 0
    _check_attention(s, q, [200, 200], out, lse, "bf16", table=gone, window=20)
    out, lse = _attend(s, q, [10 ** 6, -3])
    assert int(s.status.item()) & tq.TQ_DEV_BAD_LENGTH
    assert bool((out[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())


@pytest.mark.parametrize("code,d,qd,nq", [("int8", 64, "f32", 2), ("int8", 128, "bf16", 2), ("e4m3", 128, "bf16", 4),
                                          ("e4m3", 256, "f32", 3), ("int8", 64, "bf16", 12), ("e4m3", 128, "bf16", 66)])
def test_queries_that_are_not_numbers_spoil_their_own_rows_only(code, d, qd, nq):
    lens = [300, 40]
    s = _filled(lens, 2, d, 16, code)
    q = _queries(s, 2, nq, 4, d, qd).contiguous()
    good, _ = _attend(s, q, lens, qd)
    _check_attention(s, q, lens, good, None, qd)
    q[0, 1, nq - 1, 7] = float("nan")
    q[1, 2, 0, d - 1] = float("inf")
    out, lse = _attend(s, q, lens, qd)
    spoilt = torch.zeros(2, 4, nq, dtype=torch.bool, device="cuda")
    spoilt[0, 1, nq - 1] = spoilt[1, 2, 0] = True
    seen = torch.isfinite(lse) | torch.isneginf(lse)
    if nq == 66:
        spoilt[1, 2, 0] = False                                      # 66 rows over 40 keys: row 0 sees none of them
        assert bool((out[1, 2, 0] == 0).all())
    assert torch.equal(~seen, spoilt)
    assert bool(torch.isnan(out[spoilt]).all()) and torch.equal(out[~spoilt], good[~spoilt])


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.5])
def test_any_softmax_scale(scale):
    lens = [150, 33]
    for code, nq, qd in (("int8", 1, "bf16"), ("e4m3", 3, "f32"), ("e4m3", 70, "bf16")):
        s = _filled(lens, 1, 128, 32, code)
        q = _queries(s, 2, nq, 2, 128, qd)
        out, lse = _attend(s, q, lens, qd, scale=scale)
        _check_attention(s, q, lens, out, lse, qd, scale=scale)


def test_many_sequences_of_many_rows():
    # More sequences than one launch takes.
    b, nq = 300, 66
    lens = [int(x) for x in np.random.default_rng(3).integers(0, 40, b)]
    s = Setup(4, [max(n, 1) for n in lens], 1, 64, 16, "int8")
    s.write(lens, [0] * b)
    q = _queries(s, b, nq, 1, 64, "bf16")
    out, lse = _attend(s, q, lens)
    assert int(s.status.item()) == 0
    _check_attention(s, q, lens, out, lse, "bf16")


@pytest.mark.parametrize("b", [700, 1300])
def test_many_sequences_of_one_row(b):
    # More than one launch takes, each a CTA's own and dealt out.
    lens = [int(x) for x in np.random.default_rng(b).integers(0, 40, b)]
    s = Setup(b, [max(n, 1) for n in lens], 1, 128, 16, "e4m3")
    s.write(lens, [0] * b)
    q = _queries(s, b, 1, 3, 128, "bf16")
    out, lse = _attend(s, q, lens)
    assert int(s.status.item()) == 0
    _check_attention(s, q, lens, out, lse, "bf16")


@pytest.mark.parametrize("nq,code,d", [(1, "e4m3", 128), (1, "int8", 256), (80, "e4m3", 128)])
def test_waits_that_run_out_are_reported_and_leave_nothing_behind(monkeypatch, nq, code, d):
    monkeypatch.delenv("TQ_TEST_WAIT_NS", raising=False)
    # Long enough that every warp's ring goes round many times, and bound by the copies: only then are they waited for.
    lens = [200000, 40, 700] if nq < 9 else [60000, 40, 700]
    s = Setup(7, lens, 8, d, 64, code)
    for x in (s.cache.k, s.cache.v):
        x.copy_(torch.randint(0, 256, x.shape, dtype=torch.uint8, device="cuda") & 0x77)
    s.cache.k_scale.fill_(2.0 ** -6)
    s.cache.v_scale.fill_(2.0 ** -6)
    q = _queries(s, 3, nq, 16, d, "bf16")
    ws = tq.cache8_attention_workspace(s.cache, 3, 16, nq)
    want, _ = _attend(s, q, lens, ws=ws)
    assert int(s.status.item()) == 0
    monkeypatch.setenv("TQ_TEST_WAIT_NS", "0")
    seen = False
    flush = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    for _ in range(20):
        flush.zero_()
        s.status.zero_()
        _attend(s, q, lens, ws=ws)
        seen |= bool(int(s.status.item()) & tq.TQ_DEV_TIMEOUT)
    assert seen
    monkeypatch.delenv("TQ_TEST_WAIT_NS")
    s.status.zero_()
    out, _ = _attend(s, q, lens, ws=ws)
    assert int(s.status.item()) == 0 and torch.equal(out, want)


def test_two_streams_and_two_graphs():
    lens = [700, 90]
    sets = []
    for i, (nq, code) in enumerate(((1, "e4m3"), (90, "int8"))):
        s = _filled(lens, 2, 128, 16, code, i)
        q = _queries(s, 2, nq, 4, 128, "bf16")
        want, _ = _attend(s, q, lens)
        sets.append((s, q, want))
    # Two calls at a time on two streams, each with its workspace, both behind a long kernel.
    streams = [torch.cuda.Stream() for _ in sets]
    own = [tq.cache8_attention_workspace(s.cache, *q.shape[:3]) for s, q, _ in sets]
    outs = [torch.zeros_like(w) for _, _, w in sets]
    seq = _i32(lens)
    torch.cuda.synchronize()
    for st, (s, q, _), ws, out in zip(streams, sets, own, outs):
        with torch.cuda.stream(st):
            torch.cuda._sleep(200000)
            for _ in range(20):
                tq.tq_cache8_attention(s.cache, q, seq, out, ws, block_table=s.dtable)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, (_, _, w) in zip(outs, sets))
    # Two graphs that share one workspace, replayed in turn on one stream.
    shared = max(own, key=lambda w: w.numel())
    graphs = []
    for (s, q, _), out in zip(sets, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tq.tq_cache8_attention(s.cache, q, seq, out, shared, block_table=s.dtable)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, (_, _, w) in zip(outs, sets))
    # Longer lengths, in place, after the capture.
    seq.copy_(_i32([300, 7]))
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for (s, q, _), o in zip(sets, outs):
        _check_attention(s, q, [300, 7], o, None, "bf16")


def test_pages_beyond_32_bits():
    # Codes of 4.4 GB for keys and as much for values; a sequence lives in the last and the first pages.
    heads, block, d = 4, 128, 128
    n = (1 << 32) // (heads * block * d) + 2048
    cache = tq.Cache8(torch.empty(n, heads, block, d, dtype=torch.uint8, device="cuda"),
                      torch.empty(n, heads, block, d, dtype=torch.uint8, device="cuda"),
                      torch.zeros(n, heads, device="cuda"), torch.zeros(n, heads, device="cuda"), "e4m3")
    rows = [n - 1, 0, n - 2, (1 << 32) // (heads * block * d)]
    table = _i32([rows])
    rg = np.random.default_rng(2)
    x = [torch.from_numpy(rg.standard_normal((400, heads, d))).to(torch.bfloat16).cuda() for _ in range(2)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_cache8_write(cache, x[0], x[1], _i32([0, 400]), _i32([0]), block_table=table, d_status=st)
    small = tq.alloc_cache8(4, heads, block, d, "e4m3")
    tq.tq_cache8_write(small, x[0], x[1], _i32([0, 400]), _i32([0]), block_table=_i32([[0, 1, 2, 3]]))
    got, want = (torch.zeros(400, heads, d, device="cuda") for _ in range(2))
    tq.tq_cache8_read(cache, got, None, _i32([0, 400]), _i32([0]), block_table=table, d_status=st)
    tq.tq_cache8_read(small, want, None, _i32([0, 400]), _i32([0]), block_table=_i32([[0, 1, 2, 3]]))
    assert torch.equal(got, want)
    for nq in (1, 70):
        q = torch.from_numpy(rg.standard_normal((1, heads, nq, d))).to(torch.bfloat16).cuda()
        a, b = torch.empty_like(q), torch.empty_like(q)
        ws = tq.cache8_attention_workspace(cache, 1, heads, nq)
        tq.tq_cache8_attention(cache, q, _i32([400]), a, ws, block_table=table, d_status=st)
        tq.tq_cache8_attention(small, q, _i32([400]), b, ws, block_table=_i32([[0, 1, 2, 3]]), d_status=st)
        assert torch.equal(a, b)
    assert int(st.item()) == 0


def _check_large(cache, table, q, lens, out, lse, od, causal=True, window=0):
    """Against 64 bits on the device, over the codes read back (exact, as tested by themselves); a sequence and a KV head
    at a time."""
    b, hq, nq, d = q.shape
    h = cache.k.shape[1]
    g = hq // h
    for i in range(b):
        n = lens[i]
        kv = [torch.empty(n, h, d, device="cuda") for _ in range(2)]
        tq.tq_cache8_read(cache, kv[0], kv[1], _i32([0, n]), _i32([0]), block_table=table[i:i + 1].contiguous())
        at = torch.arange(n, device="cuda")
        pos = n - nq + torch.arange(nq, device="cuda") if causal else torch.full((nq,), n - 1, device="cuda")
        see = at[None] <= pos[:, None]
        if window:
            see &= at[None] > pos[:, None] - window
        for j in range(h):
            k, v = kv[0][:, j].double(), kv[1][:, j].double()
            x = q[i, j * g:j * g + g].double()
            s = (x @ k.T / d ** 0.5).masked_fill(~see, -torch.inf)
            m = s.amax(-1, keepdim=True)
            p = (s - torch.where(torch.isinf(m), 0.0, m)).exp()
            tot = p.sum(-1, keepdim=True)
            some = tot > 0
            ref = torch.where(some, p @ v / tot, 0.0)
            A = torch.where(some, p @ v.abs() / tot, 0.0)
            B = (x.abs() @ k.abs().T / d ** 0.5).masked_fill(~see, 0.0).amax(-1, keepdim=True)
            es = ((2 * d / 16 + 8) * 2.0 ** -23 + 2.0 ** -22) * B
            ew = es + 2.0 ** -22 + 2 * (2 * B + 20) * 2.0 ** -24
            ew = ew + (2.0 ** -21 if od == "f32" else 2.0 ** -12) + (n / 16 + 40) * 2.0 ** -23
            most = {"e4m3": 448.0, "int8": 127.0}[cache.code] * cache.v_scale[table[i, :-(-n // cache.k.shape[2])].long(), j].max()
            tol = HALF[od] * ref.abs() + 2 * ew * A + n * 2.0 ** -30 * float(most)
            err = (out[i, j * g:j * g + g].double() - ref).abs()
            assert bool((err <= tol).all()), (i, j, float((err / tol).max()))
            want = torch.where(some, m + tot.log(), -torch.inf)[..., 0]
            got = lse[i, j * g:j * g + g].double()
            assert torch.equal(torch.isneginf(got), torch.isneginf(want))
            fine = ~torch.isneginf(want)
            assert bool(((got - want).abs() <= ew[..., 0] + 2.0 ** -22 * (1 + want.abs()))[fine].all())


@pytest.mark.parametrize("b,hkv,group,nq,n,d,block,code,window,dtype", [
    (2, 8, 4, 600, 4096, 128, 64, "e4m3", 0, "bf16"), (4, 4, 4, 1024, 1024, 128, 16, "int8", 0, "bf16"),
    (3, 6, 1, 700, 3001, 64, 32, "e4m3", 513, "bf16"), (9, 8, 2, 129, 2500, 64, 128, "int8", 0, "bf16"),
    (16, 8, 4, 1, 5000, 128, 64, "e4m3", 0, "bf16"), (16, 12, 1, 4, 3000, 64, 16, "int8", 1000, "f32"),
    (16, 8, 4, 3, 4000, 128, 32, "e4m3", 0, "bf16"), (9, 4, 4, 2, 3000, 256, 16, "int8", 0, "f32")])
def test_ranges_of_several_streams_a_cta(b, hkv, group, nq, n, d, block, code, window, dtype):
    # More streams than CTAs: a CTA ends one, starts the next, and their copies, products and merges overlap.
    rg = np.random.default_rng(n)
    lens = [n] + [int(x) for x in rg.integers(1, n + 1, b - 1)] if nq < 600 else [n] * b
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
