"""Attention over the 8-bit cache where block scales lie far apart: what a row returns goes by the keys that it sees and
by their weights, whatever the scales of others.

Tolerances, per element, from the arithmetic of tests/test_gpu_cache8.py taken key by key, so that a key of small weight
or one that the row does not see grants nothing. With p the softmax weights, B_k = scale * sum |q_i k_i| of key k and u =
2^-24: a weight errs by ew_k = (2 d/16 + 8) 2^-23 B_k + 2^-22 B_k (score) + 2^-22 (ex2) + 2 u (2 B_k + 20 + D) (roundings
of the exponent, |s - m| plus D octaves between the smallest and the largest value scale, 60 at most) + 2^-11 (one half:
10 fraction bits, so steps of 2^-10 and roundings of 2^-11 of a value; 2^-21 for the two of an fp32 output) + (n/16 + 40) 2^-23 (sums, of a matrix unit that cuts). The output errs by the sum of
p_k ew_k (|v_k| + |out|), plus half a step of its type, plus what lies below a half: 2^-25 (2^-36 with a second half kept
times 2^11) of a weight in units where the largest addend of a code that is not zero, T = max p_k scale_k, is at least
2^5.5, for each key, with codes of at most M: n M T 2^-30 (n M T 2^-41).
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_cache8 import DT, HALF, Setup, _i32

pytestmark = pytest.mark.gpu
tq = pytest.importorskip("kv_cache_vector_rope_b200")

HEADS, BLOCK = 2, 16


def _make(rg, lens, d, code, shape, key=None):
    """A cache whose value scales are set by `shape(position, length)` (octaves), suppressed keys (negative score) by the
    first coordinate, which every query holds as 8; `key(position, length)` sets the keys' octaves. Returns the setup."""
    s = Setup(int(rg.integers(1 << 30)), lens, HEADS, d, BLOCK, code)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        octaves, score = shape(np.arange(n), n)
        k, v = rg.standard_normal((n, HEADS, d)), rg.standard_normal((n, HEADS, d))
        k[..., 0] = (score * np.sqrt(d) / 8)[:, None]
        v *= 2.0 ** octaves[:, None, None]
        if key is not None:
            k *= 2.0 ** key(np.arange(n), n)[:, None, None]
        row = s.dtable[b:b + 1].contiguous()
        tq.tq_cache8_write(s.cache, torch.from_numpy(k).float().cuda(), torch.from_numpy(v).float().cuda(), _i32([0, n]),
                           _i32([0]), block_table=row, d_status=s.status)
    return s


def _queries(rg, b, hq, nq, d, dtype):
    q = rg.standard_normal((b, hq, nq, d))
    q[..., 0] = 8.0
    return torch.from_numpy(q).to(DT[dtype]).cuda()


def _check(s, q, lens, out, lse, od, causal=True, window=0):
    b, hq, nq, d = q.shape
    g = hq // HEADS
    M = {"e4m3": 448.0, "int8": 127.0}[s.cache.code]
    for i in range(b):
        n = lens[i]
        if n == 0:
            assert bool((out[i] == 0).all()) and bool(torch.isneginf(lse[i]).all())
            continue
        pages = s.dtable[i, :-(-n // BLOCK)].long()
        at = torch.arange(n, device="cuda")
        pos = n - nq + torch.arange(nq, device="cuda") if causal else torch.full((nq,), n - 1, device="cuda")
        see = at[None] <= pos[:, None]
        if window:
            see &= at[None] > pos[:, None] - window
        for j in range(HEADS):
            kv = []
            for name in ("k", "v"):
                codes = getattr(s.cache, name)[pages, j].view(torch.float8_e4m3fn if s.cache.code == "e4m3" else torch.int8)
                x = codes.double() if s.cache.code == "int8" else codes.float().double()
                kv.append((x * getattr(s.cache, name + "_scale")[pages, j].double()[:, None, None]).reshape(-1, d)[:n])
            k, v = kv
            sv = s.cache.v_scale[pages, j].double().repeat_interleave(BLOCK)[:n]
            some = (v != 0).any(-1)
            D = min(60.0, float((sv.max() / sv.min()).log2()))
            x = q[i, j * g:j * g + g].double()
            score = (x @ k.T / d ** 0.5).masked_fill(~see, -torch.inf)
            m = score.amax(-1, keepdim=True)
            p = (score - torch.where(torch.isinf(m), 0.0, m)).exp()
            tot = p.sum(-1, keepdim=True)
            any_key = tot > 0
            p = torch.where(any_key, p / tot, 0.0)
            ref = p @ v
            B = x.abs() @ k.abs().T / d ** 0.5
            ew = ((2 * d / 16 + 8) * 2.0 ** -23 + 2.0 ** -22) * B + 2.0 ** -22 + 2 * 2.0 ** -24 * (2 * B + 20 + D)
            ew = ew + (2.0 ** -21 if od == "f32" else 2.0 ** -11) + (n / 16 + 40) * 2.0 ** -23
            pe = p * ew
            T = (p * sv * some).amax(-1, keepdim=True)
            tol = HALF[od] * ref.abs() + pe @ v.abs() + ref.abs() * pe.sum(-1, keepdim=True)
            tol = tol + n * M * T * (2.0 ** -41 if od == "f32" else 2.0 ** -30)
            got = out[i, j * g:j * g + g].double()
            err = (got - ref).abs()
            assert bool((err <= tol).all()), (i, j, float((err / tol).max()), float((err / ref.abs().clamp(min=1e-300)).max()))
            want = torch.where(any_key, m + tot.log(), -torch.inf)[..., 0]
            have = lse[i, j * g:j * g + g].double()
            assert torch.equal(torch.isneginf(have), torch.isneginf(want))
            fine = ~torch.isneginf(want)
            assert bool(((have - want).abs() <= pe.sum(-1) + 2.0 ** -22 * (1 + want.abs()))[fine].all())


def _attend(s, q, lens, od, **kw):
    b, hq, nq, d = q.shape
    out = torch.full((b, hq, nq, d), 5.0, dtype=DT[od], device="cuda")
    lse = torch.full((b, hq, nq), 5.0, device="cuda")
    tq.tq_cache8_attention(s.cache, q, _i32(lens), out, tq.cache8_attention_workspace(s.cache, b, hq, nq),
                           block_table=s.dtable, lse_out=lse, d_status=s.status, **kw)
    torch.cuda.synchronize()
    assert int(s.status.item()) == 0
    return out, lse


# code, d, query heads per KV head, rows, query and output types: each way of forming weights.
FEW = [("int8", 64, 4, 1, "bf16", "bf16"), ("int8", 64, 1, 4, "f32", "f32"), ("int8", 128, 2, 2, "f32", "f32"),
       ("int8", 256, 1, 3, "bf16", "bf16"), ("e4m3", 64, 2, 4, "bf16", "bf16"), ("e4m3", 64, 1, 4, "f32", "f32"),
       ("e4m3", 128, 4, 1, "bf16", "bf16"), ("e4m3", 128, 1, 7, "f32", "f32"), ("e4m3", 128, 3, 4, "bf16", "bf16"),
       ("int8", 64, 4, 4, "bf16", "bf16"), ("e4m3", 256, 2, 3, "f32", "f32"), ("e4m3", 128, 2, 4, "bf16", "f32")]
CHUNK = [("int8", 64, 2, 40, "bf16", "bf16"), ("e4m3", 64, 1, 140, "bf16", "bf16"), ("e4m3", 128, 2, 35, "bf16", "bf16"),
         ("int8", 128, 4, 70, "bf16", "bf16")]
MANY = CHUNK + [("int8", 64, 2, 40, "f32", "f32"), ("e4m3", 64, 1, 70, "f32", "f32"), ("e4m3", 128, 2, 35, "f32", "f32"),
        ("int8", 128, 1, 70, "f32", "bf16"), ("e4m3", 256, 2, 40, "bf16", "bf16"), ("int8", 256, 1, 66, "f32", "f32")]


@pytest.mark.parametrize("octaves,score", [(12, -60.0), (24, -60.0), (40, -60.0), (180, -200.0), (24, 0.0), (-24, 0.0)])
@pytest.mark.parametrize("case", FEW + MANY, ids=lambda c: "-".join(map(str, c)))
def test_one_block_of_other_scale(case, octaves, score):
    # The first block lies `octaves` above (below) the others; weighted e^-60 it cannot matter to any row.
    code, d, group, nq, qd, od = case
    rg = np.random.default_rng(octaves + d + nq)
    lens = [701, 33, 0]
    base = -80 if octaves > 100 else 0
    s = _make(rg, lens, d, code, lambda at, n: (np.where(at < BLOCK, base + octaves, base), np.where(at < BLOCK, score, 0.0)))
    q = _queries(rg, len(lens), HEADS * group, nq, d, qd)
    out, lse = _attend(s, q, lens, od)
    _check(s, q, lens, out, lse, od)


@pytest.mark.parametrize("octaves", [6, 12, 18, 24, 100])
@pytest.mark.parametrize("case", [c for c in FEW + MANY if c[3] > 1], ids=lambda c: "-".join(map(str, c)))
def test_the_newest_token_is_large(case, octaves):
    # The rows in front of it do not see it, but share its block: their own codes there are small or zero.
    code, d, group, nq, qd, od = case
    rg = np.random.default_rng(octaves + d + nq)
    lens = [700, 90, 1]
    s = _make(rg, lens, d, code, lambda at, n: (np.where(at == n - 1, octaves, 0), np.zeros(n)))
    q = _queries(rg, len(lens), HEADS * group, nq, d, qd)
    for window in (0, 50):
        out, lse = _attend(s, q, lens, od, window=window)
        _check(s, q, lens, out, lse, od, window=window)


@pytest.mark.parametrize("octaves", [12, 18, 30])
@pytest.mark.parametrize("case", [c for c in FEW + MANY if c[3] > 1], ids=lambda c: "-".join(map(str, c)))
def test_the_newest_key_is_large(case, octaves):
    # Its own row goes by that key alone; the rows in front of it go by the others, which lie far below it.
    code, d, group, nq, qd, od = case
    rg = np.random.default_rng(octaves + d + nq)
    lens = [700, 90, 1]
    s = _make(rg, lens, d, code, lambda at, n: (np.zeros(n), np.zeros(n)), lambda at, n: np.where(at == n - 1, octaves, 0))
    q = _queries(rg, len(lens), HEADS * group, nq, d, qd)
    out, lse = _attend(s, q, lens, od)
    _check(s, q, lens, out, lse, od)


@pytest.mark.parametrize("case", FEW + MANY, ids=lambda c: "-".join(map(str, c)))
def test_scales_that_wander_and_values_that_are_all_zero(case):
    code, d, group, nq, qd, od = case
    rg = np.random.default_rng(d + nq)
    lens = [1100, 64]

    def shape(at, n):
        octaves = np.round(50 * np.sin(at // BLOCK / 7.0))
        return np.where((at // 40) % 3 == 1, -1000, octaves), 20 * np.cos(at / 90.0)      # a third of the values are zero
    s = _make(rg, lens, d, code, shape)
    q = _queries(rg, len(lens), HEADS * group, nq, d, qd)
    for causal in (True, False):
        out, lse = _attend(s, q, lens, od, causal=causal)
        _check(s, q, lens, out, lse, od, causal=causal)
    s.cache.v.zero_()
    out, lse = _attend(s, q, lens, od)
    assert bool((out == 0).all())
    _check(s, q, lens, out, lse, od)


@pytest.mark.parametrize("case", FEW + MANY, ids=lambda c: "-".join(map(str, c)))
def test_values_near_the_largest(case):
    # Values up to 2^126: sums of weights times codes stay within fp32 in their own unit.
    code, d, group, nq, qd, od = case
    rg = np.random.default_rng(d + nq + 1)
    lens = [900]
    s = _make(rg, lens, d, code, lambda at, n: (np.full(n, 123), np.zeros(n)))
    q = _queries(rg, 1, HEADS * group, nq, d, qd)
    out, lse = _attend(s, q, lens, od)
    assert bool(torch.isfinite(out).all())
    _check(s, q, lens, out, lse, od)


LONG = [("int8", 64, 1, 2, "f32", "f32"), ("e4m3", 128, 4, 1, "bf16", "bf16"), ("e4m3", 64, 4, 3, "bf16", "bf16"),
        ("int8", 64, 2, 40, "bf16", "bf16"), ("e4m3", 128, 2, 150, "bf16", "bf16"), ("e4m3", 128, 1, 70, "f32", "f32"),
        ("int8", 256, 1, 66, "bf16", "bf16")]


@pytest.mark.parametrize("octaves", [-70, 30, 90])
@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(map(str, c)))
def test_sequences_cut_between_many_ctas(case, octaves):
    # Their records meet with units that lie far apart, some without an addend: the first third of the values is zero, the
    # next one lies `octaves` above the last and weighs e^-40 of it.
    code, d, group, nq, qd, od = case
    rg = np.random.default_rng(abs(octaves) + d + nq)
    lens = [9001, 700]

    def shape(at, n):
        third = 3 * at // n
        return np.choose(third, [-1000, octaves, 0]), np.choose(third, [1.0, -40.0, 0.0])
    s = _make(rg, lens, d, code, shape)
    q = _queries(rg, len(lens), HEADS * group, nq, d, qd)
    for kw in ({}, dict(window=6500)):
        out, lse = _attend(s, q, lens, od, **kw)
        _check(s, q, lens, out, lse, od, **kw)


@pytest.mark.parametrize("power", [22, 40, 70])
@pytest.mark.parametrize("case", FEW + MANY + LONG, ids=lambda c: "-".join(map(str, c)))
def test_scores_of_any_size(case, power):
    # Queries times 2^power: a row is the value of its largest score, where that is ahead by more than the scores' errors.
    code, d, group, nq, qd, od = case
    rg = np.random.default_rng(power + d + nq)
    lens = [2500, 200, 3]
    s = _make(rg, lens, d, code, lambda at, n: (10 * np.sin(at // BLOCK), np.zeros(n)), lambda at, n: 3 * at / n)
    q = _queries(rg, len(lens), HEADS * group, nq, d, qd) * 2.0 ** power
    out, lse = _attend(s, q, lens, od)
    assert not bool(torch.isnan(out).any()) and not bool(torch.isnan(lse).any())
    checked = 0
    for i, n in enumerate(lens):
        pages = s.dtable[i, :-(-n // BLOCK)].long()
        see = torch.arange(n, device="cuda")[None] <= n - nq + torch.arange(nq, device="cuda")[:, None]
        for j in range(HEADS):
            k, v = ((getattr(s.cache, m)[pages, j].view(torch.float8_e4m3fn if code == "e4m3" else torch.int8).float().double() *
                     getattr(s.cache, m + "_scale")[pages, j].double()[:, None, None]).reshape(-1, d)[:n] for m in ("k", "v"))
            x = q[i, j * group:j * group + group].double()
            score = (x @ k.T / d ** 0.5).masked_fill(~see, -torch.inf)
            size = (x.abs() @ k.abs().T / d ** 0.5).masked_fill(~see, 0.0).amax(-1)
            two = score.topk(2, -1)
            top, at = two.values[..., 0], two.indices[..., 0]
            some = ~torch.isinf(top)
            es = ((2 * d / 16 + 8) * 2.0 ** -23 + 2.0 ** -21) * size
            got, have = out[i, j * group:j * group + group].double(), lse[i, j * group:j * group + group].double()
            assert bool(((have - top).abs() <= es + 10.0)[some].all())        # the sum of weights adds ln n at most
            ahead = some & (top - two.values[..., 1] > 2 * es + 60.0)
            ref = v[at]
            assert bool(((got - ref).abs() <= (HALF[od] + 2.0 ** -11) * ref.abs() + 1e-20)[ahead].all())
            checked += int(ahead.sum())
    assert checked > 0
