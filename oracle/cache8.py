"""The 8-bit block-scaled paged KV cache, in plain fp64 NumPy.

gist.science "TurboESM ..." section 2A (RoPE first) and 2E (online softmax
over the packed cache); 7minutos.es Etapa 1 (a token's codes are computed when
it enters the cache). Definitions:

  norm_rope  y = x / sqrt(mean x^2 + eps) * w, then pairs (i, i + r/2) turned
             by pos * base^(-2i/r), i < r/2
  scale      of a block: 2^e, the smallest e >= -100 with amax <= M 2^e,
             M = 448 (e4m3) or 127 (int8)
  code       nearest representable to x / scale, ties to even; a stored value
             is code * scale
  write      a block that holds tokens keeps the larger of its old scale and
             the one its new tokens need; held codes are rounded once more when
             the scale grows
  attention  row i of nq at position len - nq + i; causal, window; a row that
             sees nothing gives zeros and lse = -inf

A cache is a dict with "k", "v" (uint8 [n_blocks, heads, block, d]),
"k_scale", "v_scale" (float32 [n_blocks, heads]) and "code" ("e4m3", "int8").
"""
from __future__ import annotations

import numpy as np

MOST = {"e4m3": 448.0, "int8": 127.0}
LARGEST = 2.0 ** 127
E_MIN = -100


def e4m3_values() -> np.ndarray:
    """Value of each e4m3 byte: sign, 4 exponent bits (bias 7), 3 mantissa bits; 0x7f and 0xff are NaN."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where(b & 128, -v, v)
    v[(b & 127) == 127] = np.nan
    return v


def values(codes: np.ndarray, code: str) -> np.ndarray:
    if code == "int8":
        return codes.view(np.int8).astype(np.float64)
    return e4m3_values()[codes]


def encode(y: np.ndarray, code: str) -> np.ndarray:
    """Bytes of values already divided by the scale: nearest, ties to even, saturating; NaN becomes zero."""
    y = np.where(np.isnan(y), 0.0, np.clip(y, -MOST[code], MOST[code]))
    if code == "int8":
        return np.rint(y).astype(np.int8).view(np.uint8)
    table = e4m3_values()[:127]                                  # ascending magnitudes
    mid = 0.5 * (table[1:] + table[:-1])
    a = np.abs(y)
    at = np.searchsorted(mid, a, side="left")                    # ties fall to the lower byte ...
    tie = (at < 126) & (a == mid[np.minimum(at, 125)])
    at = at + (tie & (at % 2 == 1))                              # ... unless it is odd
    return (at | np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def block_scale(amax, code: str) -> np.ndarray:
    e = np.full(np.shape(amax), E_MIN, dtype=np.int64)
    amax = np.asarray(amax, dtype=np.float64)
    for k in range(E_MIN, 128):
        e = np.where(amax > MOST[code] * 2.0 ** k, k + 1, e)
    return 2.0 ** e.astype(np.float64)


def write(cache: dict, k: np.ndarray, v: np.ndarray, cu, start, table) -> None:
    code, blk = cache["code"], cache["k"].shape[2]
    for name, x in (("k", k), ("v", v)):
        codes, scales = cache[name], cache[name + "_scale"]
        for b in range(len(start)):
            p, row = int(start[b]), int(cu[b])
            while row < cu[b + 1]:
                page, r0 = int(table[b][p // blk]), p % blk
                n = min(blk - r0, int(cu[b + 1]) - row)
                new = x[row:row + n].astype(np.float64).transpose(1, 0, 2)          # [heads, n, d]
                mag = np.abs(new)
                amax = np.where(mag <= LARGEST, mag, 0.0).max(axis=(1, 2))
                s = block_scale(amax, code)
                if r0:
                    old = scales[page].astype(np.float64)
                    s = np.maximum(s, old)
                    held = values(codes[page, :, :r0], code) * (old / s)[:, None, None]
                    grown = s > old
                    codes[page, grown, :r0] = encode(held, code)[grown]
                with np.errstate(invalid="ignore"):
                    codes[page, :, r0:r0 + n] = encode(new / s[:, None, None], code)
                scales[page] = s
                p, row = p + n, row + n


def read(cache: dict, cu, start, table) -> tuple[np.ndarray, np.ndarray]:
    """Rows [cu[-1], heads, d] in fp64."""
    blk = cache["k"].shape[2]
    out = []
    for name in ("k", "v"):
        rows = np.zeros((int(cu[-1]), cache["k"].shape[1], cache["k"].shape[3]))
        for b in range(len(start)):
            for i in range(int(cu[b + 1]) - int(cu[b])):
                p = int(start[b]) + i
                page = int(table[b][p // blk])
                rows[int(cu[b]) + i] = (values(cache[name][page, :, p % blk], cache["code"]) *
                                        cache[name + "_scale"][page].astype(np.float64)[:, None])
        out.append(rows)
    return out[0], out[1]


def norm_rope(x: np.ndarray, weight, eps: float, positions, base: float, rot: int) -> np.ndarray:
    """x [tokens, heads, d] in fp64."""
    x = x.astype(np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    if positions is not None and rot:
        h = rot // 2
        a = np.asarray(positions, dtype=np.float64)[:, None] * base ** (-2.0 * np.arange(h) / rot)
        c, s = np.cos(a)[:, None], np.sin(a)[:, None]
        lo, hi = x[..., :h].copy(), x[..., h:rot].copy()
        x = x.copy()
        x[..., :h], x[..., h:rot] = lo * c - hi * s, lo * s + hi * c
    return x


def attention(cache: dict, q: np.ndarray, lens, table, causal=True, window=0, scale=None):
    """q [batch, hq, nq, d] -> out, lse, and what error bounds need: spread (softmax mean of |v|), size
    (scale * max over seen keys of sum |q_i k_i|), top (largest code times the largest value scale, [batch, hq, 1])."""
    b, hq, nq, d = q.shape
    h, blk = cache["k"].shape[1], cache["k"].shape[2]
    g = hq // h
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    out, spread = np.zeros(q.shape), np.zeros(q.shape)
    lse, size, top = np.full((b, hq, nq), -np.inf), np.zeros((b, hq, nq)), np.zeros((b, hq, 1))
    for i in range(b):
        n = int(lens[i])
        if n == 0:
            continue
        first = max(0, n - nq + 1 - window) // blk if window else 0            # pages before it may be gone
        pages = np.asarray(table[i][first:-(-n // blk)], dtype=np.int64)
        gone = (pages < 0) | (pages >= cache["k"].shape[0])
        pages = np.where(gone, 0, pages)
        at = np.arange(first * blk, n)
        for j in range(h):
            k, v = (np.nan_to_num(values(cache[m][pages, j], cache["code"])) *
                    cache[m + "_scale"][pages, j].astype(np.float64)[:, None, None] for m in ("k", "v"))
            k, v = k.reshape(-1, d)[:len(at)], v.reshape(-1, d)[:len(at)]
            lost = np.repeat(gone, blk)[:len(at)]
            top[i, j * g:j * g + g] = MOST[cache["code"]] * cache["v_scale"][pages, j].max()
            for r in range(nq):
                pos = n - nq + r if causal else n - 1
                see = (at <= pos) & ~lost
                if window:
                    see &= at > pos - window
                if not see.any():
                    continue
                for a in range(j * g, j * g + g):
                    s = scale * (k[see] @ q[i, a, r])
                    m = s.max()
                    p = np.exp(s - m)
                    out[i, a, r] = p @ v[see] / p.sum()
                    spread[i, a, r] = p @ np.abs(v[see]) / p.sum()
                    lse[i, a, r] = m + np.log(p.sum())
                    size[i, a, r] = abs(scale) * (np.abs(k[see]) @ np.abs(q[i, a, r])).max()
    return out, lse, spread, size, top
