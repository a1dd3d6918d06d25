"""Pins of the 8-bit cache's oracle (CPU): the code formats, the block scale, a growing block, attention's masks."""
import numpy as np
import torch

from oracle import cache8 as o8


def test_e4m3_values_and_rounding_are_those_of_the_format():
    v = o8.e4m3_values()
    ref = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, ref, equal_nan=True)
    assert np.nanmax(v) == 448.0 and v[1] == 2.0 ** -9
    rg = np.random.default_rng(0)
    x = np.concatenate([rg.uniform(-448, 448, 20000), rg.standard_normal(20000) * 0.01, v[~np.isnan(v)],
                        0.5 * (v[:126] + v[1:127]), [0.0, -0.0, 2.0 ** -11, 2.0 ** -10, -2.0 ** -10]])
    x = x.astype(np.float32)
    got = o8.encode(x.astype(np.float64), "e4m3")
    assert np.array_equal(got, torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert list(o8.encode(np.array([1e9, -np.inf, np.nan]), "e4m3")) == [0x7e, 0xfe, 0]
    assert list(o8.encode(np.array([0.5, 1.5, 2.5, -0.5, 300.0, np.nan]), "int8").view(np.int8)) == [0, 2, 2, 0, 127, 0]


def test_block_scale_is_the_smallest_power_of_two_that_holds_the_block():
    for code, top in (("e4m3", 448.0), ("int8", 127.0)):
        for amax in (1.0, top, top * (1 + 2.0 ** -20), 1e-20, 3.0e38, 2.0 ** 127, 0.0, 1e-40):
            s = float(o8.block_scale(amax, code))
            assert np.log2(s) == np.rint(np.log2(s)) and s >= 2.0 ** -100
            assert amax <= top * s
            assert s == 2.0 ** -100 or amax > top * s / 2


def test_a_growing_block_keeps_what_it_holds_within_half_a_step():
    rg = np.random.default_rng(1)
    for code in ("e4m3", "int8"):
        c = {"k": np.full((1, 1, 16, 16), 0xff, np.uint8), "v": np.full((1, 1, 16, 16), 0xff, np.uint8),
             "k_scale": np.full((1, 1), np.nan, np.float32), "v_scale": np.full((1, 1), np.nan, np.float32), "code": code}
        x = rg.standard_normal((16, 1, 16)) * 2.0 ** np.arange(16)[:, None, None]
        for t in range(16):
            o8.write(c, x[t:t + 1], x[t:t + 1], [0, 1], [t], [[0]])
        k, v = o8.read(c, [0, 16], [0], [[0]])
        assert np.array_equal(k, v)
        s = float(c["k_scale"][0, 0])
        assert s == o8.block_scale(np.abs(x).max(), code)
        if code == "int8":
            # Each growth by 2^j rounds once more: at most half a step of every scale passed, less than one in all.
            assert np.abs(k - x).max() < s
        else:
            assert np.all(np.abs(k - x) <= np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** -9 * s))
        assert np.array_equal(o8.block_scale(np.abs(x[:3]).max(), code) <= s, True)


def test_attention_masks():
    rg = np.random.default_rng(2)
    c = {"code": "int8"}
    for m in ("k", "v"):
        c[m] = rg.integers(0, 256, (4, 2, 16, 16)).astype(np.uint8)
        c[m + "_scale"] = np.full((4, 2), 2.0 ** -6, np.float32)
    q = rg.standard_normal((2, 4, 3, 16))
    table = np.array([[2, 0], [1, 3]])
    out, lse, _, _, _ = o8.attention(c, q, [2, 20], table)
    assert np.all(out[0, :, 0] == 0) and np.all(lse[0, :, 0] == -np.inf)       # three rows, two keys
    assert np.allclose(out[0, :2, 1], o8.values(c["v"][2, 0, 0], "int8") * 2.0 ** -6)
    full, _, _, _, _ = o8.attention(c, q, [2, 20], table, causal=False)
    assert np.allclose(full[1, :, 2], out[1, :, 2])
    near, _, _, _, _ = o8.attention(c, q, [2, 20], table, window=1)
    assert np.allclose(near[1, 0, 1], o8.values(c["v"][3, 0, 2], "int8") * 2.0 ** -6)   # key 18 alone
    wide, _, _, _, _ = o8.attention(c, q, [2, 20], table, window=100)
    assert np.allclose(wide, out)


def test_norm_rope_turns_by_position_and_keeps_the_norm():
    rg = np.random.default_rng(3)
    x = rg.standard_normal((5, 2, 16))
    pos = np.array([0, 1, 7, 100000, 3])
    y = o8.norm_rope(x, None, 1e-6, pos, 10000.0, 16)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
    assert np.allclose(y[0], x[0])
    assert np.allclose(y[1, 0, 0], x[1, 0, 0] * np.cos(1) - x[1, 0, 8] * np.sin(1))
    z = o8.norm_rope(x, np.full(16, 2.0), 0.0, None, 10000.0, 16)
    assert np.allclose((z * z).mean(-1), 4.0)
    part = o8.norm_rope(x, None, 1e-6, pos, 10000.0, 8)
    assert np.array_equal(part[..., 8:], x[..., 8:]) and not np.allclose(part[2, ..., :8], x[2, ..., :8])
