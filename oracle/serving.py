"""Reference definitions of the INT8 product, the paged 8-bit key/value cache
and attention over it (numpy; the fp32 steps in numpy float32, everything else
in fp64 or exact integers).

TEST INFRASTRUCTURE ONLY, like the rest of this package.

Readings:

* INT8 product: exact integer sums, one rounding to fp32, then the two scale
  multiplies and the bias add in fp32.
* Append: one scale per block and head from the absolute maximum of what the
  block receives, never smaller than the scale of codes that stay in it; codes
  that stay are coded again when the scale grows; elements that are not finite
  are left out of the maximum, infinities saturate, NaN is coded as 0.
* Attention: softmax over the visible stored values; a row that sees nothing
  gives zeros and a log-sum of -inf.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np

from .reference import TINY_AMAX, e4m3_decode, e4m3_encode

QMAX = {"int8": np.float32(127.0), "fp8": np.float32(448.0)}


def int8_gemm(a: np.ndarray, sa: np.ndarray, b: np.ndarray, sb: np.ndarray,
              bias: Optional[np.ndarray] = None) -> np.ndarray:
    """fp32 [M, N] of int8 codes a [M, K], b [N, K] before the output rounding."""
    # int64 sums by fp64 products: every partial sum is below 2^53
    acc = (a.astype(np.float64) @ b.astype(np.float64).T).astype(np.int64)
    y = acc.astype(np.float32) * sa.astype(np.float32)[:, None] * sb.astype(np.float32)[None, :]
    return y if bias is None else y + bias.astype(np.float32)[None, :]


def kv_encode(y: np.ndarray, fmt: str) -> np.ndarray:
    """Codes of fp32 values in code units."""
    y = np.where(np.isnan(y), np.float32(0), np.clip(y, -QMAX[fmt], QMAX[fmt]))
    if fmt == "int8":
        return np.rint(y).astype(np.int8)
    return e4m3_encode(y.astype(np.float64))


def kv_decode(codes: np.ndarray, fmt: str) -> np.ndarray:
    return codes.astype(np.float64) if fmt == "int8" else e4m3_decode(codes)


def _slices(n: int, length: int, tokens: int, cap: int):
    """(page, first offset, end offset, first new row) of each touched block."""
    p = max(0, length - n)
    end = min(length, cap)
    while p < end:
        e = min(end, (p // tokens + 1) * tokens)
        yield p // tokens, p % tokens, e - (p // tokens) * tokens, p - (length - n)
        p = e


def kv_append(cache, k: np.ndarray, v: np.ndarray, table: np.ndarray, lens: Sequence[int],
              cu: Sequence[int], fmt: str):
    """New cache (k, k_scale, v, v_scale) after appending float rows k, v
    [total, heads, dim]; k codes [blocks, heads, T, D], v [blocks, heads, D, T]."""
    kc, ks, vc, vs = (x.copy() for x in cache)
    blocks, _, tokens, _ = kc.shape
    one = np.float32(1)
    for codes, scales, rows, trans in ((kc, ks, k, False), (vc, vs, v, True)):
        for b, length in enumerate(lens):
            for page, o0, o1, row in _slices(cu[b + 1] - cu[b], int(length), tokens,
                                             table.shape[1] * tokens):
                blk = int(table[b, page])
                if not 0 <= blk < blocks:
                    continue
                for h in range(codes.shape[1]):
                    x = rows[cu[b] + row:cu[b] + row + o1 - o0, h].astype(np.float32)  # [new, D]
                    side = codes[blk, h].T if trans else codes[blk, h]                 # [T, D] view
                    mag = np.abs(x[np.isfinite(x)])
                    amax = np.float32(mag.max()) if mag.size else np.float32(0)
                    s = np.float32(amax / QMAX[fmt]) if amax >= TINY_AMAX else np.float32(0)
                    old = scales[blk, h] if o0 else np.float32(0)
                    s = max(s, old)
                    inv = np.float32(one / s) if s > 0 else np.float32(0)
                    if o0 and s > old:
                        ratio = np.float32(old * inv)
                        side[:o0] = kv_encode(kv_decode(side[:o0], fmt).astype(np.float32) * ratio, fmt)
                    with np.errstate(invalid="ignore"):
                        side[o0:o1] = kv_encode(x * inv, fmt)
                    scales[blk, h] = s
    return kc, ks, vc, vs


def kv_attention(q: np.ndarray, cache, table: np.ndarray, lens: Sequence[int], cu: Sequence[int],
                 fmt: str, scale: float, causal: bool = True, window: int = 0):
    """(out, lse, spread, reach) in fp64 for queries q [total, heads, dim]: the
    result, log sum exp, sum_t p_t |V_t| per output (the size rounding errors
    are relative to) and the largest sum_d |q_d K_td| of each row."""
    kc, ks, vc, vs = cache
    blocks, kv, tokens, dim = kc.shape
    total, heads, _ = q.shape
    out, lse = np.zeros(q.shape), np.full((total, heads), -math.inf)
    spread, reach = np.zeros(q.shape), np.zeros((total, heads))
    for b, length in enumerate(lens):
        n, length = cu[b + 1] - cu[b], int(length)
        for i in range(n):
            pos = length - n + i
            hi = min(length, pos + 1) if causal else length
            lo = max(0, pos - window + 1) if window else 0
            seen = [p for p in range(lo, min(hi, table.shape[1] * tokens))
                    if 0 <= int(table[b, p // tokens]) < blocks]
            if not seen:
                continue
            blk = np.array([int(table[b, p // tokens]) for p in seen])
            off = np.array([p % tokens for p in seen])
            for h in range(kv):
                kk = kv_decode(kc[blk, h, off], fmt) * ks[blk, h].astype(np.float64)[:, None]
                vv = kv_decode(vc[blk, h, :, off], fmt) * vs[blk, h].astype(np.float64)[:, None]
                for g in range(heads // kv):
                    hq = h * (heads // kv) + g
                    x = q[cu[b] + i, hq].astype(np.float64)
                    s = scale * (kk @ x)
                    top = s.max()
                    p = np.exp(s - top)
                    z = p.sum()
                    out[cu[b] + i, hq] = (p @ vv) / z
                    spread[cu[b] + i, hq] = (p @ np.abs(vv)) / z
                    lse[cu[b] + i, hq] = top + math.log(z)
                    reach[cu[b] + i, hq] = scale * (np.abs(kk) @ np.abs(x)).max()
    return out, lse, spread, reach
