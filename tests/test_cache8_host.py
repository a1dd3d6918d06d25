"""Argument checks of the 8-bit cache's entry points (CPU: nothing is launched)."""
import ctypes

import pytest
import torch

import kv_cache_vector_rope_b200 as tq

INVALID, UNSUPPORTED, WORKSPACE = tq.TQ_ERR_INVALID_ARG, tq.TQ_ERR_UNSUPPORTED, tq.TQ_ERR_WORKSPACE


def _cache(d=128, heads=8, block=64, code=0, n=100, k=0x10000, v=0x20000, ks=0x30000, vs=0x40000):
    return tq._Cache8(d, heads, block, code, n, k, v, ks, vs)


def _rows(fn, c, dtype=1, k=0x1000, kts=1024, khs=128, v=0x2000, vts=1024, vhs=128, n=4, batch=2, cu=0x100, start=0x200,
          table=0x300, stride=10):
    return fn(ctypes.byref(c), dtype, k, kts, khs, v, vts, vhs, n, batch, cu, start, table, stride, None, None)


@pytest.mark.parametrize("fn", [tq._lib.tq_cache8_write, tq._lib.tq_cache8_read])
def test_rows_host_validation(fn):
    assert _rows(fn, _cache(), n=0) == tq.TQ_OK and _rows(fn, _cache(), batch=0) == tq.TQ_OK     # nothing to do
    for bad in (dict(d=100), dict(d=0), dict(d=272), dict(block=48), dict(block=0), dict(code=2), dict(heads=0), dict(n=0),
                dict(n=1 << 31), dict(k=0), dict(vs=0), dict(k=0x10040), dict(ks=0x30002)):
        assert _rows(fn, _cache(**bad)) == INVALID, bad
    for bad in (dict(dtype=2), dict(n=-1), dict(n=1 << 31), dict(batch=-1), dict(cu=0), dict(start=0), dict(stride=0),
                dict(stride=1 << 26), dict(k=0x1008), dict(kts=1028), dict(vhs=-128), dict(table=0, stride=51)):
        assert _rows(fn, _cache(), **bad) == INVALID, bad
        assert tq.tq_last_error_string()


def test_write_needs_both_and_read_outputs_must_not_overlap():
    w, r = tq._lib.tq_cache8_write, tq._lib.tq_cache8_read
    assert _rows(w, _cache(), v=0) == INVALID and _rows(r, _cache(), k=0, v=0) == INVALID
    assert _rows(r, _cache(), kts=128, khs=128) == INVALID
    assert "overlap" in tq.tq_last_error_string()
    assert _rows(r, _cache(), vts=1016) == INVALID


def _norm(d=128, rot=128, n=4, hq=8, hkv=2, dtype=1, q=0x1000, qts=1280, qhs=128, k=0x2000, qo=0x3000, qots=1024,
          qohs=128, ko=0x4000, kots=256, qw=0x5000, kw=0x6000, eps=1e-6, pos=0x7000, base=1e4):
    return tq._lib.tq_qk_norm_rope(d, rot, n, hq, hkv, dtype, q, qts, qhs, k, 1280, 128, qo, qots, qohs, ko, kots, 128, qw,
                                   kw, eps, pos, base, None, None)


def test_norm_rope_host_validation():
    assert _norm(n=0) == tq.TQ_OK and _norm(hq=0, hkv=0) == tq.TQ_OK
    for bad in (dict(d=100), dict(d=264), dict(rot=12), dict(rot=136), dict(rot=-8), dict(n=-1), dict(hq=-1), dict(dtype=3),
                dict(eps=-1.0), dict(eps=float("nan")), dict(base=0.0), dict(base=float("inf")), dict(q=0), dict(ko=0),
                dict(q=0x1004), dict(qts=1282), dict(qhs=-128), dict(qots=1020), dict(qohs=64), dict(kots=128),
                dict(qw=0x5004)):
        assert _norm(**bad) == INVALID, bad


def _attend(c=None, qd=1, qbs=4096, qhs=128, qrs=4096, batch=2, hq=32, nq=1, lens=0x200, table=0x300, stride=10, causal=1,
            window=0, scale=0.1, q=0x1000, out=0x2000, od=1, obs=4096, ohs=128, ors=4096, ws=0x100000, wsb=1 << 30):
    c = c or _cache()
    return tq._lib.tq_cache8_attention(ctypes.byref(c), q, qd, qbs, qhs, qrs, batch, hq, nq, lens, table, stride, causal,
                                       window, scale, out, od, obs, ohs, ors, None, ws, wsb, None, None)


def test_attention_host_validation():
    assert _attend(batch=0) == tq.TQ_OK
    for bad in (dict(qd=2), dict(od=5), dict(batch=-1), dict(hq=0), dict(hq=12), dict(nq=0), dict(nq=1 << 26), dict(window=-1),
                dict(window=5, causal=0), dict(scale=float("nan")), dict(scale=float("inf")), dict(q=0), dict(out=0),
                dict(lens=0), dict(stride=0), dict(table=0, stride=51), dict(q=0x1008), dict(qhs=100), dict(nq=2, qrs=-4096),
                dict(obs=64), dict(ohs=64), dict(nq=2, ors=128), dict(ws=0x100010)):
        assert _attend(**bad) == INVALID, bad
    assert _attend(c=_cache(d=96)) == UNSUPPORTED
    assert _attend(ws=0) == WORKSPACE and _attend(wsb=1000) == WORKSPACE
    assert "workspace" in tq.tq_last_error_string()


def test_attention_refuses_sequences_that_32_bits_cannot_count():
    assert _attend(_cache(block=128, n=1 << 24), stride=(1 << 23) + 1) == UNSUPPORTED
    assert "2^30" in tq.tq_last_error_string()


def test_sizes():
    assert tq.tq_cache8_bytes(128, 8, 64, 10) == 2 * 10 * 8 * (64 * 128 + 4)
    assert tq.tq_cache8_bytes(100, 8, 64, 10) == -1
    f = tq._lib.tq_cache8_attention_workspace_bytes
    assert f(ctypes.byref(_cache()), 2, 32, 1) > 0 and f(ctypes.byref(_cache(block=5)), 2, 32, 1) == 0


def _refuses(what, f, *a, **k):
    with pytest.raises(ValueError, match=what):
        f(*a, **k)


def test_binding_refuses_before_anything_is_launched():
    c = tq.alloc_cache8(4, 2, 16, 64, device="cpu")
    assert c.nbytes() == tq.tq_cache8_bytes(64, 2, 16, 4)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    x, cu, start, table = torch.zeros(3, 2, 64), i32(0, 3), i32(0), torch.zeros(1, 4, dtype=torch.int32)
    for f in (tq.tq_cache8_write, tq.tq_cache8_read):
        _refuses("CUDA", f, c, x, x, cu, start)
        _refuses("tensor", f, c, "x", x, cu, start)
        _refuses("heads and d", f, c, x[:, :1], x, cu, start)
        _refuses("heads and d", f, c, x, x.bfloat16(), cu, start)
        _refuses("unit stride", f, c, x.transpose(1, 2).contiguous().transpose(1, 2), x, cu, start)
        _refuses("cu_tokens is None", f, c, x, x, None, start)
        _refuses("start", f, c, x, x, cu, start[0])
    _refuses("k and v are needed", tq.tq_cache8_write, c, x, None, cu, start)
    _refuses("both None", tq.tq_cache8_read, c, None, None, cu, start)
    bad = tq.Cache8(c.k, c.v, c.k_scale, c.v_scale[:2], "e4m3")
    _refuses("scales", tq.tq_cache8_read, bad, x, x, cu, start)
    _refuses("code", tq.tq_cache8_read, tq.Cache8(c.k, c.v, c.k_scale, c.v_scale, "e5m2"), x, x, cu, start)
    q, ws = torch.zeros(1, 4, 1, 64), torch.zeros(1 << 20, dtype=torch.uint8)
    _refuses("CUDA", tq.tq_cache8_attention, c, q, start, q, ws, table)
    _refuses("same shape", tq.tq_cache8_attention, c, q, start, q[0], ws, table)
    _refuses("q's d", tq.tq_cache8_attention, c, q[..., :32], start, q[..., :32], ws, table)
    _refuses("lse_out", tq.tq_cache8_attention, c, q, start, q, ws, table, lse_out=torch.zeros(4))
    _refuses("seq_lens is None", tq.tq_cache8_attention, c, q, None, q, ws, table)
    _refuses("go together", tq.tq_qk_norm_rope, x, None, None, x)
    _refuses("output as its input", tq.tq_qk_norm_rope, x, None, x[:2], None)
    _refuses("one dtype", tq.tq_qk_norm_rope, x, None, x.bfloat16(), None)
    _refuses("weights", tq.tq_qk_norm_rope, x, None, x, None, q_weight=torch.ones(32))
    _refuses("one of them at least", tq.tq_qk_norm_rope, None, None, None, None)
    _refuses("CUDA", tq.tq_qk_norm_rope, x, x, x, x)
    with pytest.raises(TypeError):
        tq._bind.cache8_rows(1, 2)
