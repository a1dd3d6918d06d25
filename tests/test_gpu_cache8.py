"""The 8-bit cache on the GPU against its fp64 oracle: q/k norm with RoPE, write, read back, attention.

Tolerances, per element, from the arithmetic (u = 2^-24, one fp32 rounding):

norm_rope   the norm's factor errs by at most (d/8 + 5 + 1) u in the sum of squares (d/LPR fused products per lane,
            shuffles; halved by the root), 2 ulp in rsqrt and 3 roundings of products, an angle by pi u (rounded
            remainder) and sincospi by 2 ulp; with d <= 256: below 48 u (|a| + |b|) for a pair (a, b), plus half a step
            of the output type.
write/read  codes, scales and values are exact: equal bytes.
attention   with B the oracle's `size` (scale times the largest sum |q_i k_i|) and A its `spread` (softmax mean of |v|):
            a score errs by (2 d/16 + 8) 2^-23 B (the matrix unit cuts each of its sums; two limbs for fp32) + 2^-22 of
            q's limbs B; its weight then by that, by 2^-22 of ex2 and 2 |s| u, |s| <= 2 B + 20 octaves, and by the half
            limbs (2^-12 with bf16 outputs, 2^-22 with fp32 ones). The value sum adds n/16 + 40 roundings (cut: 2^-23).
            All of it times 2 A (numerator and sum), plus half a step of the output type. Halves end at 2^-24: a weight
            2^(s - m + 6), times a value scale over the largest so far, is off by up to 2^-25 beside that, which is
            2^-31 of a weight sum of at least 1 (the largest score's own weight) for each key and a code of at most M
            in units of the largest scale: n 2^-31 top, top = M times the largest value scale; doubled for fp32's sums.
"""
import numpy as np
import pytest
import torch

from oracle import cache8 as o8

pytestmark = pytest.mark.gpu
tq = pytest.importorskip("kv_cache_vector_rope_b200")

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def _np(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _values(rg, *shape):
    x = rg.standard_normal(shape)
    x[..., rg.integers(shape[-1])] *= 9.0
    return x


class Setup:
    """A cache of random pages: every byte 0xff and every scale NaN until something is written."""

    def __init__(self, seed, caps, heads, d, block, code):
        self.rg = np.random.default_rng(seed)
        per = [-(-c // block) for c in caps]
        n = sum(per) + 2
        order = self.rg.permutation(n)
        self.table = np.full((len(caps), max(max(per), 1)), -1, np.int32)
        at = 0
        for b, p in enumerate(per):
            self.table[b, :p] = order[at:at + p]
            at += p
        self.cache = tq.alloc_cache8(n, heads, block, d, code)
        self.cache.k.fill_(255)
        self.cache.v.fill_(255)
        self.cache.k_scale.fill_(float("nan"))
        self.cache.v_scale.fill_(float("nan"))
        self.dtable = _i32(self.table.tolist())
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def host(self):
        c = self.cache
        return {"k": c.k.cpu().numpy().copy(), "v": c.v.cpu().numpy().copy(), "k_scale": c.k_scale.cpu().numpy().copy(),
                "v_scale": c.v_scale.cpu().numpy().copy(), "code": c.code}

    def write(self, new, start, dtype="bf16", scale=1.0, ref=None):
        """Writes `new[b]` tokens behind start[b]; with `ref`, the oracle's cache follows."""
        c = self.cache
        cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        h, d = c.k.shape[1], c.k.shape[3]
        x = [torch.from_numpy(_values(self.rg, int(cu[-1]), h, d) * scale).to(DT[dtype]) for _ in range(2)]
        tq.tq_cache8_write(c, x[0].cuda(), x[1].cuda(), _i32(cu.tolist()), _i32(list(start)), block_table=self.dtable,
                           d_status=self.status)
        torch.cuda.synchronize()
        if ref is not None:
            o8.write(ref, _np(x[0]), _np(x[1]), cu, start, self.table)
        return x


def _same(cache, ref):
    got = {"k": cache.k, "v": cache.v, "k_scale": cache.k_scale, "v_scale": cache.v_scale}
    for name, t in got.items():
        assert np.array_equal(t.cpu().numpy(), ref[name], equal_nan=name.endswith("scale")), name


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("n,hq,hkv,d,rot,dtype,norm,pos", [
    (1, 32, 8, 128, 128, "bf16", True, True), (7, 20, 20, 64, 32, "f32", True, True), (1021, 4, 1, 256, 256, "bf16", True, True),
    (3, 5, 3, 80, 48, "f32", True, True), (130, 3, 2, 8, 8, "bf16", False, True), (33, 2, 0, 200, 200, "bf16", True, True),
    (5, 0, 3, 16, 0, "f32", True, False), (6000, 2, 1, 128, 64, "bf16", True, True), (9, 7, 2, 24, 16, "f32", False, False)])
def test_qk_norm_rope(n, hq, hkv, d, rot, dtype, norm, pos):
    rg = np.random.default_rng(n * 31 + d)
    qkv = torch.from_numpy(_values(rg, n, hq + 2 * hkv + 1, d)).to(DT[dtype]).cuda()
    q, k = qkv[:, :hq], qkv[:, hq:hq + hkv]                        # slices of a fused projection
    w = [torch.from_numpy(1 + 0.3 * rg.standard_normal(d)).float().cuda() if norm else None for _ in range(2)]
    p = _i32(rg.integers(0, 1 << 20, n).tolist()) if pos else None
    out = torch.full((n, hq + hkv, d + 8), 7.0, dtype=DT[dtype], device="cuda")
    qo, ko = out[:, :hq, :d], out[:, hq:, :d]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tq.tq_qk_norm_rope(q if hq else None, k if hkv else None, qo if hq else None, ko if hkv else None, w[0], w[1], 1e-5, p,
                       10000.0, rot, d_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and bool((out[..., d:] == 7).all())
    for x, o, wt in ((q, qo, w[0]), (k, ko, w[1])):
        if x.shape[1] == 0:
            continue
        P = None if p is None else p.cpu().numpy()
        ref = o8.norm_rope(_np(x), None if wt is None else _np(wt), 1e-5, P, 10000.0, rot)
        y = np.abs(o8.norm_rope(_np(x), None if wt is None else _np(wt), 1e-5, None, 10000.0, rot))
        mag = y.copy()
        mag[..., :rot // 2] += y[..., rot // 2:rot]
        mag[..., rot // 2:rot] += y[..., :rot // 2]
        assert np.all(np.abs(_np(o) - ref) <= HALF[dtype] * np.abs(ref) + 48 * 2.0 ** -24 * mag)


def test_qk_norm_rope_in_place_and_bad_position():
    x = torch.randn(11, 6, 64, device="cuda")
    w = torch.rand(64, device="cuda") + 0.5
    pos = torch.arange(11, dtype=torch.int32, device="cuda")
    ref = torch.empty_like(x)
    tq.tq_qk_norm_rope(x[:, :4], x[:, 4:], ref[:, :4], ref[:, 4:], w, w, positions=pos)
    y = x.clone()
    tq.tq_qk_norm_rope(y[:, :4], y[:, 4:], y[:, :4], y[:, 4:], w, w, positions=pos)
    assert torch.equal(y, ref)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos[3] = -1
    tq.tq_qk_norm_rope(x[:, :4], None, ref[:, :4], None, w, positions=pos, d_status=st)
    assert int(st.item()) == tq.TQ_DEV_BAD_POSITION


# ------------------------------------------------------------------ write and read
@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d,block,heads,dtype", [(128, 64, 8, "bf16"), (64, 16, 3, "f32"), (256, 128, 2, "bf16"),
                                                 (80, 32, 5, "f32"), (16, 16, 1, "bf16")])
def test_write_and_read_are_exact(code, d, block, heads, dtype):
    caps = [300, 17, 1, 128, 65]
    s = Setup(d + block, caps, heads, d, block, code)
    ref = s.host()
    start = [0] * len(caps)
    # Prompts, one token each, growing values, a ragged mix with empty sequences.
    for new, scale in (([100, 16, 0, 64, 63], 1.0), ([1, 1, 1, 1, 1], 30.0), ([1, 0, 0, 1, 1], 0.01),
                       ([131, 0, 0, 62, 0], 4.0), ([60, 0, 0, 0, 0], 1000.0)):
        s.write(new, start, dtype, scale, ref)
        start = [a + n for a, n in zip(start, new)]
        _same(s.cache, ref)
    assert int(s.status.item()) == 0
    a, n = [3, 0, 0, 64, 2], [250, 17, 1, 40, 0]
    cu = np.concatenate([[0], np.cumsum(n)])
    want = o8.read(ref, cu, a, s.table)
    for out in (torch.bfloat16, torch.float32):
        rows = torch.full((int(cu[-1]) + 2, heads, d + 8), 5.0, dtype=out, device="cuda")
        k, v = rows.clone(), rows.transpose(0, 1).contiguous().transpose(0, 1)
        tq.tq_cache8_read(s.cache, k[..., :d], v[..., :d], _i32(cu.tolist()), _i32(a), block_table=s.dtable, d_status=s.status)
        for got, w in ((k, want[0]), (v, want[1])):
            assert np.array_equal(_np(got[:-2, :, :d]), w)
            assert bool((got[-2:] == 5).all()) and bool((got[..., d:] == 5).all())
        only = rows.clone()
        tq.tq_cache8_read(s.cache, None, only[..., :d], _i32(cu.tolist()), _i32(a), block_table=s.dtable)
        assert np.array_equal(_np(only[:-2, :, :d]), want[1])
    assert int(s.status.item()) == 0


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_write_values_that_are_not_finite_zero_and_extreme(code):
    s = Setup(3, [64], 1, 32, 16, code)
    ref = s.host()
    x = torch.randn(48, 1, 32)
    x[0, 0, 3], x[1, 0, 4], x[2, 0, 5], x[3, 0, 6] = float("inf"), -float("inf"), float("nan"), 3e38
    x[16:32] = 0.0
    x[32:48] *= 1e-42
    y = torch.randn(48, 1, 32) * 1e37
    tq.tq_cache8_write(s.cache, x.cuda(), y.cuda(), _i32([0, 48]), _i32([0]), block_table=s.dtable, d_status=s.status)
    o8.write(ref, x.double().numpy(), y.double().numpy(), [0, 48], [0], s.table)
    _same(s.cache, ref)
    assert int(s.status.item()) == tq.TQ_DEV_NONFINITE
    k = torch.empty(48, 1, 32, device="cuda")
    tq.tq_cache8_read(s.cache, k, None, _i32([0, 48]), _i32([0]), block_table=s.dtable)
    assert bool(torch.isfinite(k).all()) and bool((k[16:32] == 0).all())


def test_write_without_a_table_and_many_sequences():
    # 1500 sequences (more than one launch handles) of a contiguous cache, two blocks each.
    b, h, d, blk = 1500, 1, 32, 16
    rg = np.random.default_rng(8)
    c = tq.alloc_cache8(2 * b, h, blk, d, "int8")
    c.k.zero_(), c.v.zero_(), c.k_scale.zero_(), c.v_scale.zero_()
    ref = {"k": c.k.cpu().numpy().copy(), "v": c.v.cpu().numpy().copy(), "k_scale": c.k_scale.cpu().numpy().copy(),
           "v_scale": c.v_scale.cpu().numpy().copy(), "code": "int8"}
    table = np.arange(2 * b).reshape(b, 2)
    start = np.zeros(b, np.int64)
    for top in (20, 13):
        new = rg.integers(0, top, b)
        cu = np.concatenate([[0], np.cumsum(new)])
        x, y = (torch.from_numpy(rg.standard_normal((int(cu[-1]), h, d))).to(torch.bfloat16) for _ in range(2))
        tq.tq_cache8_write(c, x.cuda(), y.cuda(), _i32(cu.tolist()), _i32(start.tolist()))
        o8.write(ref, _np(x), _np(y), cu, start, table)
        start = start + new
    _same(c, ref)
    cu = np.concatenate([[0], np.cumsum(start)])
    k = torch.empty(int(cu[-1]), h, d, device="cuda")
    tq.tq_cache8_read(c, k, None, _i32(cu.tolist()), _i32([0] * b))
    assert np.array_equal(_np(k), o8.read(ref, cu, np.zeros(b, np.int64), table)[0])


def test_bad_pages_and_lengths_are_reported_and_left_alone():
    s = Setup(5, [64, 64], 2, 64, 16, "e4m3")
    ref = s.host()
    bad = s.table.copy()
    bad[0, 1], bad[1, 0] = -1, s.cache.k.shape[0]
    x = torch.randn(128, 2, 64)
    tq.tq_cache8_write(s.cache, x.cuda(), x.cuda(), _i32([0, 64, 128]), _i32([0, 0]), block_table=_i32(bad.tolist()),
                       d_status=s.status)
    assert int(s.status.item()) == tq.TQ_DEV_BAD_BLOCK
    xs = x.double().numpy()
    for b, j in ((0, 0), (0, 2), (0, 3), (1, 1), (1, 2), (1, 3)):
        rows = xs[64 * b + 16 * j:64 * b + 16 * j + 16]
        o8.write(ref, rows, rows, [0, 16], [16 * j], s.table[b:b + 1])
    _same(s.cache, ref)
    s.status.zero_()
    k = torch.full((128, 2, 64), 9.0, device="cuda")
    tq.tq_cache8_read(s.cache, k, None, _i32([0, 64, 128]), _i32([0, 0]), block_table=_i32(bad.tolist()), d_status=s.status)
    assert int(s.status.item()) == tq.TQ_DEV_BAD_BLOCK and bool((k[16:32] == 0).all()) and bool((k[64:80] == 0).all())
    # Beyond the table, negative starts, lengths that fall: reported, nothing out of range touched.
    for cu, start in (([0, 64, 128], [40, -1]), ([0, 64, 60], [0, 0]), ([-5, 3, 128], [0, 0]), ([0, 0, 500], [0, 50])):
        s.status.zero_()
        tq.tq_cache8_write(s.cache, x.cuda(), x.cuda(), _i32(cu), _i32(start), block_table=s.dtable, d_status=s.status)
        assert int(s.status.item()) & tq.TQ_DEV_BAD_LENGTH


# ------------------------------------------------------------------ attention
def _check_attention(s, q, lens, out, lse, dtype, causal=True, window=0, scale=None, table=None):
    ref, rl, A, B, top = o8.attention(s.host(), _np(q), lens, s.table if table is None else table, causal, window, scale)
    d, n = q.shape[3], max(max(lens), 1)
    B = B[..., None]
    es = ((2 * d / 16 + 8) * 2.0 ** -23 + 2.0 ** -22) * B
    ew = es + 2.0 ** -22 + 2 * (2 * B + 20) * 2.0 ** -24
    ew = ew + (2.0 ** -21 if dtype == "f32" else 2.0 ** -12) + (n / 16 + 40) * 2.0 ** -23
    tol = HALF[dtype] * np.abs(ref) + 2 * ew * A + n * 2.0 ** -30 * top[..., None]
    err = np.abs(_np(out) - ref)
    worst = np.unravel_index(np.argmax(err / np.maximum(tol, 1e-300)), err.shape)
    if not (err <= tol).all():
        pytest.fail(f"{worst}: err {err[worst]}, bound {tol[worst]}, value {ref[worst]}, spread {A[worst]}")
    if lse is not None:
        got = _np(lse)
        empty = np.isinf(rl)
        assert np.array_equal(np.isneginf(got), empty)
        tl = (ew[..., 0] + 2.0 ** -22 * (1 + np.abs(np.where(empty, 0, rl))))[~empty]
        assert np.all(np.abs(got[~empty] - rl[~empty]) <= tl)
    return err, tol


CASES = [
    # lens, heads, group, nq, d, block, code, q dtype, out dtype, causal, window
    ([777], 2, 4, 1, 128, 64, "e4m3", "bf16", "bf16", True, 0),
    ([1], 1, 1, 1, 64, 16, "int8", "f32", "f32", True, 0),
    ([5, 0, 16, 17, 700, 64, 63, 65], 2, 4, 1, 128, 16, "int8", "bf16", "bf16", True, 0),
    ([300, 2, 33, 0, 130], 3, 1, 4, 64, 16, "int8", "f32", "f32", True, 0),
    ([300, 2, 33, 0, 130], 1, 7, 3, 128, 32, "e4m3", "bf16", "f32", True, 0),
    ([90, 1, 257], 2, 8, 2, 256, 128, "e4m3", "bf16", "bf16", True, 0),
    ([90, 1, 257], 1, 3, 5, 256, 64, "int8", "f32", "f32", True, 0),
    ([513, 60], 2, 2, 40, 64, 64, "e4m3", "bf16", "bf16", True, 0),
    ([200, 31], 1, 5, 33, 128, 32, "int8", "f32", "bf16", True, 0),
    ([400, 129, 7], 2, 4, 1, 128, 64, "e4m3", "bf16", "bf16", True, 100),
    ([400, 129, 7], 2, 2, 6, 64, 16, "int8", "f32", "f32", True, 1),
    ([1000, 129, 7], 1, 4, 9, 128, 128, "e4m3", "bf16", "bf16", True, 33),
    ([300, 77, 0], 2, 2, 7, 128, 16, "e4m3", "bf16", "bf16", False, 0),
    ([4097], 1, 16, 1, 128, 64, "int8", "bf16", "f32", True, 0),
    ([640, 100], 2, 4, 130, 128, 64, "e4m3", "bf16", "bf16", True, 0),
    ([640, 100], 1, 1, 257, 64, 32, "int8", "bf16", "bf16", True, 200),
    ([300, 512], 1, 2, 129, 256, 64, "e4m3", "bf16", "bf16", True, 0),
    ([300, 70], 2, 2, 150, 128, 16, "e4m3", "bf16", "bf16", False, 0),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{i}-d{c[4]}-{c[6]}-nq{c[3]}-g{c[2]}-{c[7]}-{c[8]}" for i, c in enumerate(CASES)])
def test_attention(case):
    lens, heads, group, nq, d, block, code, qd, od, causal, window = case
    s = Setup(sum(lens) + d + nq, lens, heads, d, block, code)
    half = [n // 2 for n in lens]
    s.write(half, [0] * len(lens))
    s.write([n - h for n, h in zip(lens, half)], half, scale=3.0)
    q = torch.from_numpy(_values(s.rg, len(lens), nq, heads * group, d) * 1.5).to(DT[qd]).cuda().transpose(1, 2)
    out = torch.full((len(lens), nq, heads * group, d + 8), 5.0, dtype=DT[od], device="cuda")
    o = out[..., :d].transpose(1, 2)
    lse = torch.full((len(lens), heads * group, nq), 5.0, device="cuda")
    ws = tq.cache8_attention_workspace(s.cache, len(lens), heads * group, nq)
    ws.fill_(0xff)
    tq.tq_cache8_attention(s.cache, q, _i32(lens), o, ws, block_table=s.dtable, causal=causal, window=window, lse_out=lse,
                           d_status=s.status)
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0 and bool((out[..., d:] == 5).all())
    _check_attention(s, q, lens, o, lse, od, causal, window)
    # The same call again, without the lse, gives the same bits.
    again = torch.empty_like(o)
    tq.tq_cache8_attention(s.cache, q, _i32(lens), again, ws, block_table=s.dtable, causal=causal, window=window)
    assert torch.equal(again, o)


def test_attention_scores_that_rise_and_scales_that_jump():
    # Keys whose scores climb by hundreds of octaves from block to block, values whose scale jumps by 2^40 both ways.
    for code in ("e4m3", "int8"):
        n, d = 1500, 64
        s = Setup(77, [n], 1, d, 16, code)
        k = s.rg.standard_normal((n, 1, d)) * np.linspace(0.1, 40.0, n)[:, None, None]
        v = s.rg.standard_normal((n, 1, d)) * 2.0 ** (40.0 * np.sin(np.arange(n) / 90.0))[:, None, None]
        tq.tq_cache8_write(s.cache, torch.from_numpy(k).float().cuda(), torch.from_numpy(v).float().cuda(), _i32([0, n]),
                           _i32([0]), block_table=s.dtable, d_status=s.status)
        for qd in ("bf16", "f32"):
            q = torch.from_numpy(s.rg.standard_normal((1, 4, 3, d)) * 3).to(DT[qd]).cuda()
            q[0, 1] *= 1e-30
            q[0, 2] *= 1e3
            q[0, 3, 0] = 0.0
            out = torch.empty(1, 4, 3, d, device="cuda")
            lse = torch.empty(1, 4, 3, device="cuda")
            c = tq.Cache8(s.cache.k, s.cache.v, s.cache.k_scale, s.cache.v_scale, code)
            # Four query heads share the one KV head.
            ws = tq.cache8_attention_workspace(c, 1, 4, 3)
            tq.tq_cache8_attention(c, q, _i32([n]), out, ws, block_table=s.dtable, lse_out=lse, d_status=s.status)
            _check_attention(s, q, [n], out, lse, "f32")
    assert int(s.status.item()) == 0


def test_attention_bad_pages_and_lengths():
    s = Setup(9, [200, 200], 2, 128, 32, "e4m3")
    s.write([200, 200], [0, 0])
    bad = s.table.copy()
    bad[0, 2], bad[1, 0] = -7, s.cache.k.shape[0]
    bad[1, 6] = 1 << 30
    q = torch.randn(2, 4, 2, 128, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    lse = torch.empty(2, 4, 2, device="cuda")
    ws = tq.cache8_attention_workspace(s.cache, 2, 4, 2)
    tq.tq_cache8_attention(s.cache, q, _i32([200, 200]), out, ws, block_table=_i32(bad.tolist()), lse_out=lse,
                           d_status=s.status)
    assert int(s.status.item()) == tq.TQ_DEV_BAD_BLOCK
    _check_attention(s, q, [200, 200], out, lse, "bf16", table=bad)
    # A window leaves early pages untouched, and they may be gone.
    s.status.zero_()
    gone = s.table.copy()
    gone[:, :5] = -1
    tq.tq_cache8_attention(s.cache, q, _i32([200, 200]), out, ws, block_table=_i32(gone.tolist()), lse_out=lse, window=39,
                           d_status=s.status)
    assert int(s.status.item()) == 0
    _check_attention(s, q, [200, 200], out, lse, "bf16", window=39, table=gone)
    cap = s.table.shape[1] * 32
    s.write([cap - 200, cap - 200], [200, 200]) if cap > 200 else None
    tq.tq_cache8_attention(s.cache, q, _i32([cap + 5, -3]), out, ws, block_table=s.dtable, lse_out=lse, d_status=s.status)
    assert int(s.status.item()) & tq.TQ_DEV_BAD_LENGTH
    _check_attention(s, q, [cap, 0], out, lse, "bf16")


def test_attention_of_many_sequences_without_a_table():
    b, h, d, blk = 1100, 1, 64, 16
    rg = np.random.default_rng(4)
    lens = rg.integers(0, 33, b)
    c = tq.alloc_cache8(2 * b, h, blk, d, "e4m3")
    c.k.fill_(255), c.v.fill_(255)
    cu = np.concatenate([[0], np.cumsum(lens)])
    x, y = (torch.from_numpy(rg.standard_normal((int(cu[-1]), h, d))).to(torch.bfloat16).cuda() for _ in range(2))
    tq.tq_cache8_write(c, x, y, _i32(cu.tolist()), _i32([0] * b))
    q = torch.from_numpy(rg.standard_normal((b, 2, 1, d))).to(torch.bfloat16).cuda()
    out, lse = torch.empty_like(q), torch.empty(b, 2, 1, device="cuda")
    tq.tq_cache8_attention(c, q, _i32(lens.tolist()), out, tq.cache8_attention_workspace(c, b, 2, 1), lse_out=lse)

    class S:
        table = np.arange(2 * b).reshape(b, 2)

        @staticmethod
        def host():
            return {"k": c.k.cpu().numpy(), "v": c.v.cpu().numpy(), "k_scale": c.k_scale.cpu().numpy(),
                    "v_scale": c.v_scale.cpu().numpy(), "code": "e4m3"}
    _check_attention(S, q, lens.tolist(), out, lse, "bf16")


def test_binding_refusals_on_the_device():
    s = Setup(2, [32], 2, 64, 16, "e4m3")
    x = torch.zeros(4, 2, 64, device="cuda")
    for cu, start, table in ((_i32([0, 4]).long(), _i32([0]), s.dtable), (_i32([0, 4, 4]), _i32([0]), s.dtable),
                             (_i32([0, 4]), _i32([0]), s.dtable.t()), (_i32([0, 4]), _i32([0]), s.dtable.cpu()),
                             (_i32([0, 4]).cpu(), _i32([0]), s.dtable)):
        with pytest.raises(ValueError):
            tq.tq_cache8_write(s.cache, x, x, cu, start, block_table=table)
    with pytest.raises(ValueError):
        tq.tq_cache8_write(s.cache, x, x, _i32([0, 4]), _i32([0]), block_table=s.dtable, d_status=torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError):
        tq.tq_cache8_write(s.cache, x.half(), x.half(), _i32([0, 4]), _i32([0]), block_table=s.dtable)
    with pytest.raises(tq.TQError):
        tq.tq_cache8_read(s.cache, x[:, :, :64].expand(4, 2, 64)[:1].expand(4, 2, 64), None, _i32([0, 4]), _i32([0]),
                          block_table=s.dtable)                      # rows of an output that overlap
    q = torch.zeros(1, 2, 1, 64, device="cuda")
    with pytest.raises(tq.TQError) as e:
        tq.tq_cache8_attention(s.cache, q, _i32([1]), q, torch.zeros(256, dtype=torch.uint8, device="cuda"), block_table=s.dtable)
    assert e.value.status == tq.TQ_ERR_WORKSPACE


# ------------------------------------------------------------------ together
def test_prompt_then_steps_together_eager_and_in_a_graph():
    """norm + rotation, write, attention over a prompt and three steps; the steps also replayed from one graph on a side
    stream, whose lengths live in device memory."""
    b, hq, hkv, d, blk, nq = 3, 8, 2, 128, 16, 20
    lens = [nq, nq, nq]
    s = Setup(12, [64, 64, 64], hkv, d, blk, "e4m3")
    ref = s.host()
    rg = s.rg
    w = [torch.from_numpy(1 + 0.1 * rg.standard_normal(d)).float().cuda() for _ in range(2)]

    def layer(qkv, pos, cu, start, seq, n, q, k, out, ws, stream=None):
        tq.tq_qk_norm_rope(qkv[:, :hq], qkv[:, hq:hq + hkv], q, k, w[0], w[1], 1e-6, pos, 10000.0, stream=stream)
        tq.tq_cache8_write(s.cache, k, qkv[:, hq + hkv:], cu, start, block_table=s.dtable, d_status=s.status, stream=stream)
        qv = q.view(b, n, hq, d).transpose(1, 2)
        tq.tq_cache8_attention(s.cache, qv, seq, out, ws, block_table=s.dtable, d_status=s.status, stream=stream)
        return qv

    def check(qkv, pos, q, k, n, start, out):
        kx = _np(qkv[:, hq:hq + hkv])
        kr = o8.norm_rope(kx, _np(w[1]), 1e-6, pos.cpu().numpy(), 10000.0, d)
        assert np.all(np.abs(_np(k) - kr) <= 2.0 ** -7 * np.abs(kr).max(-1, keepdims=True))
        cu = np.arange(b + 1) * n
        o8.write(ref, _np(k), _np(qkv[:, hq + hkv:]), cu, start, s.table)
        _same(s.cache, ref)
        _check_attention(s, q.view(b, n, hq, d).transpose(1, 2), [a + n for a in start], out, None, "bf16")

    ws = tq.cache8_attention_workspace(s.cache, b, hq, nq)
    qkv = torch.from_numpy(_values(rg, b * nq, hq + 2 * hkv, d)).to(torch.bfloat16).cuda()
    q, k = torch.empty_like(qkv[:, :hq]).contiguous(), torch.empty(b * nq, hkv, d, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(b, hq, nq, d, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(nq, dtype=torch.int32, device="cuda").repeat(b)
    layer(qkv, pos, _i32([0, nq, 2 * nq, 3 * nq]), _i32([0] * b), _i32(lens), nq, q, k, out, ws)
    check(qkv, pos, q, k, nq, [0] * b, out)

    q1, k1 = q[:b].clone(), k[:b].clone()
    out1 = torch.empty(b, hq, 1, d, dtype=torch.bfloat16, device="cuda")
    step = torch.empty(b, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")
    pos1, start, seq, cu = _i32([nq] * b), _i32([nq] * b), _i32([nq + 1] * b), _i32(list(range(b + 1)))
    side = torch.cuda.Stream()
    graph = None
    for t in range(3):
        step.copy_(torch.from_numpy(_values(rg, b, hq + 2 * hkv, d) * (t + 1)).to(torch.bfloat16))
        if t == 0:
            torch.cuda.synchronize()
            layer(step, pos1, cu, start, seq, 1, q1, k1, out1, ws, stream=side)
            side.synchronize()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    layer(step, pos1, cu, start, seq, 1, q1, k1, out1, ws)
            graph.replay()
        torch.cuda.synchronize()
        check(step, pos1, q1, k1, 1, [nq + t] * b, out1)
        pos1 += 1
        start += 1
        seq += 1
    assert int(s.status.item()) == 0
    # The same arithmetic on the default stream gives the same bits.
    ref_out = out1.clone()
    seq -= 1
    qv = q1.view(b, 1, hq, d).transpose(1, 2)
    tq.tq_cache8_attention(s.cache, qv, seq, out1, ws, block_table=s.dtable)
    assert torch.equal(out1, ref_out)
