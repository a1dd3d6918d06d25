"""Queries and keys that are not finite, through norm and rotation: where they must not go.

Exact comparisons: without a weight an element that is not turned is copied, with one its row's factor is NaN or zero by
the formula, and a row without such a value has the bits that it has by itself.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_cache8 import DT, _i32

pytestmark = pytest.mark.gpu
tq = pytest.importorskip("kv_cache_vector_rope_b200")


def _rows(seed, n, h, d, dtype):
    """Normal rows with a zero of either sign; and where something is put: in each row r of a token another element."""
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal((n, h, d))).to(DT[dtype]).cuda()
    x[:, :, 3] = 0.0
    x[:, :, d - 2] = -0.0
    return x


def _bits(t):
    return t.contiguous().view(torch.int32 if t.dtype is torch.float32 else torch.int16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,pos", [(128, 64, True), (128, 128, False), (80, 48, True), (64, 0, True), (256, 8, True), (8, 8, False)])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_elements_that_are_not_turned_are_copied(d, rot, pos, dtype, bad):
    x = _rows(d + rot, 9, 40, d, dtype)
    first = rot if pos else 0                                     # elements from here on are not turned
    put = [first + i % (d - first) for i in range(40)]
    for i, e in enumerate(put):
        x[:, i, e] = bad
    p = _i32(list(range(1000, 1009))) if pos else None
    q, k = torch.empty_like(x[:, :29]), torch.empty_like(x[:, 29:])
    tq.tq_qk_norm_rope(x[:, :29], x[:, 29:], q, k, positions=p, rot_dim=rot)
    y = torch.cat([q, k], 1)
    finite = torch.isnan(x[..., first:]) | (_bits(y[..., first:]).view_as(x[..., first:]) == _bits(x[..., first:]).view_as(x[..., first:]))
    assert bool(finite.all())
    assert torch.equal(torch.isnan(y[..., first:]), torch.isnan(x[..., first:]))
    assert bool(torch.isfinite(y[..., :first]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot,pos", [(128, 64, True), (128, 128, True), (128, 128, False), (72, 16, True), (256, 128, True)])
def test_a_norm_with_a_value_that_is_not_finite(d, rot, pos, dtype):
    # An infinity: the row's factor is 0, so 0 * inf = NaN where it is (and where it is turned into), zeros elsewhere. NaN:
    # the whole row. Rows beside them keep their bits.
    n, h = 5, 24
    x = _rows(d, n, h, d, dtype)
    w = torch.from_numpy(np.random.default_rng(1).standard_normal(d)).float().cuda()
    p = _i32([7, 0, 1 << 20, 3, 99]) if pos else None
    clean = torch.empty_like(x)
    tq.tq_qk_norm_rope(x, None, clean, None, w, positions=p, rot_dim=rot)
    spoilt = x.clone()
    half, turned = rot // 2, rot if pos else 0
    for i in range(0, h, 3):
        spoilt[:, i, (5 * i) % d] = float("inf") if i % 2 else -float("inf")
        spoilt[:, i + 1, (7 * i) % d] = float("nan")
    y = torch.empty_like(x)
    tq.tq_qk_norm_rope(spoilt, None, y, None, w, positions=p, rot_dim=rot)
    for i in range(0, h, 3):
        assert torch.equal(_bits(y[:, i + 2]), _bits(clean[:, i + 2]))
        assert bool(torch.isnan(y[:, i + 1]).all())
        e = (5 * i) % d
        into = {e, (e + half) % turned if e < turned else e}
        want = torch.zeros(d, dtype=torch.bool, device="cuda")
        want[list(into)] = True
        assert torch.equal(torch.isnan(y[:, i]), want.expand(n, d))
        assert bool((y[:, i][~want.expand(n, d)] == 0).all())
