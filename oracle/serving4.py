"""Reference definitions of the serving operators around 4-bit data: RMS norm with
the residual's addition and a quantized output, the MXFP4 product, the paged MXFP4
key/value cache and attention over it (numpy; the fp32 steps in numpy float32,
everything else in fp64).

TEST INFRASTRUCTURE ONLY, like the rest of this package.

Readings:

* Norm: the mean of the squares and the reciprocal root are fp64, rounded once; the
  two products of an element are fp32; the sum with the residual is rounded to the
  storage type, and the norm is taken of what is stored.
* A scale byte of 255 is NaN.
* Append: elements that are not finite are left out of the block's maximum,
  infinities saturate, NaN is coded as 0.
* Attention: softmax over the visible stored values; a row that sees nothing gives
  zeros and a log-sum of -inf.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np

from .reference import QSpec, decode_input, dequantize_mxfp4, quantize_mxfp4, quantize_rows


def round_to(x: np.ndarray, dtype: str) -> np.ndarray:
    """fp32 values rounded to a storage type, as raw storage."""
    x = np.asarray(x, np.float32)
    if dtype == "f32":
        return x
    if dtype == "f16":
        return x.astype(np.float16)
    b = x.view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)     # finite inputs


def rmsnorm(raw: np.ndarray, dtype: str, weight: np.ndarray, eps: float,
            residual: Optional[np.ndarray] = None):
    """(y fp32 [rows, K], raw sum or None) of raw rows; weight fp32 [K]."""
    total = None
    if residual is not None:
        a, b = (decode_input(r, dtype).astype(np.float32) for r in (raw, residual))
        raw = total = round_to(a + b, dtype)
    h = decode_input(raw, dtype)                                       # fp64, exact
    mean = np.array([math.fsum(r) for r in h * h]) / h.shape[1] + float(np.float32(eps))
    with np.errstate(divide="ignore"):
        r = np.where(mean > 0, 1.0 / np.sqrt(mean), 0.0).astype(np.float32)
    y = h.astype(np.float32) * r[:, None] * weight.astype(np.float32)
    return y, total


def rmsnorm_quantize(raw, dtype, weight, eps, q: QSpec, residual=None):
    """(codes, scales, raw sum or None)."""
    y, total = rmsnorm(raw, dtype, weight, eps, residual)
    codes, scales = quantize_mxfp4(y, "f32") if q.fmt == "mxfp4" else quantize_rows(y, "f32", q)
    return codes, scales, total


def mxfp4_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """fp64 values of codes [..., K/2] with scale bytes [..., K/32]; 255 is NaN."""
    x = dequantize_mxfp4(codes.reshape(-1, codes.shape[-1]), scales.reshape(-1, scales.shape[-1]))
    nan = np.repeat(scales.reshape(-1, scales.shape[-1]) == 255, 32, axis=-1)
    return np.where(nan, np.nan, x).reshape(*codes.shape[:-1], -1)


def mxfp4_gemm(a, sa, b, sb, bias=None):
    """(fp64 [M, N], sum |a b| [M, N])."""
    x, w = mxfp4_values(a, sa), mxfp4_values(b, sb)
    y = x @ w.T
    return (y if bias is None else y + bias.astype(np.float64)), np.abs(x) @ np.abs(w).T


def kv_encode(x: np.ndarray):
    """MXFP4 of fp32 values [..., D]: codes [..., D/2], scale bytes [..., D/32]."""
    shape = x.shape
    x = np.where(np.isnan(x), np.float32(0), x).astype(np.float32).reshape(-1, 32)
    inf = np.isinf(x)
    codes, scales = quantize_mxfp4(np.where(inf, np.float32(0), x), "f32")
    for nib, at in ((0, slice(0, None, 2)), (4, slice(1, None, 2))):    # saturate
        full = np.where(np.signbit(x[:, at]), 15, 7) << nib
        codes = np.where(inf[:, at], (codes & (0xF0 >> nib)) | full, codes).astype(np.uint8)
    return codes.reshape(*shape[:-1], -1), scales.reshape(*shape[:-1], -1)


def kv_append(cache, k: np.ndarray, v: np.ndarray, table: np.ndarray, lens: Sequence[int],
              cu: Sequence[int]):
    """New cache (k, k_scale, v, v_scale) after appending float rows k, v [total, heads,
    dim]; codes [blocks, heads, T, D/2], scales [blocks, heads, D/32, T]."""
    kc, ks, vc, vs = (x.copy() for x in cache)
    blocks, _, tokens, _ = kc.shape
    for codes, scales, rows in ((kc, ks, k), (vc, vs, v)):
        for b, length in enumerate(lens):
            n = cu[b + 1] - cu[b]
            for i in range(n):
                pos = int(length) - n + i
                if not 0 <= pos < table.shape[1] * tokens:
                    continue
                blk = int(table[b, pos // tokens])
                if 0 <= blk < blocks:
                    codes[blk, :, pos % tokens], scales[blk, :, :, pos % tokens] = kv_encode(rows[cu[b] + i])
    return kc, ks, vc, vs


def kv_attention(q: np.ndarray, cache, table: np.ndarray, lens: Sequence[int], cu: Sequence[int],
                 scale: float, causal: bool = True, window: int = 0):
    """(out, lse, spread, reach) in fp64 for queries q [total, heads, dim]: the
    result, log sum exp, sum_t p_t |V_t| per output (the size rounding errors
    are relative to) and the largest scale * sum_d |q_d K_td| of each row."""
    kc, ks, vc, vs = cache
    blocks, kv, tokens, _ = kc.shape
    k, v = (mxfp4_values(c, s.transpose(0, 1, 3, 2)) for c, s in ((kc, ks), (vc, vs)))
    total, heads, _ = q.shape
    out, lse = np.zeros(q.shape), np.full((total, heads), -math.inf)
    spread, reach = np.zeros(q.shape), np.zeros((total, heads))
    g = heads // kv
    for b, length in enumerate(lens):
        n, length = cu[b + 1] - cu[b], int(length)
        for i in range(n):
            pos = length - n + i
            hi = min(length, pos + 1) if causal else length
            lo = max(0, pos - window + 1) if window else 0
            p = np.arange(lo, max(lo, min(hi, table.shape[1] * tokens)))
            blk = table[b, p // tokens].astype(np.int64)
            there = (blk >= 0) & (blk < blocks)
            blk, off = blk[there], p[there] % tokens
            if not blk.size:
                continue
            for h in range(kv):
                kk, vv = k[blk, h, off], v[blk, h, off]
                x = q[cu[b] + i, h * g:(h + 1) * g].astype(np.float64)            # [g, D]
                s = scale * (x @ kk.T)
                top = s.max(1, keepdims=True)
                e = np.exp(s - top)
                z = e.sum(1, keepdims=True)
                at = (cu[b] + i, slice(h * g, (h + 1) * g))
                out[at], spread[at] = (e @ vv) / z, (e @ np.abs(vv)) / z
                lse[at] = (top + np.log(z))[:, 0]
                reach[at] = scale * (np.abs(x) @ np.abs(kk).T).max(1)
    return out, lse, spread, reach
