"""fp64 definitions of the block-scaled 8-bit KV cache and of attention with
block scales, capped and distance-biased scores — TEST INFRASTRUCTURE ONLY.

Plain numpy loops over requests, blocks and heads; shares no code with the
CUDA path.  README core feature 3 names the compressed cache, nothing more:
the block scales, the cap and the bias follow the C header's formulas.
"""
from __future__ import annotations

import numpy as np

import oracle

FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}


def fp8_table(fmt: str) -> np.ndarray:
    """The values of all 256 codes (NaN and infinities included)."""
    return np.array([oracle.widen8(c, fmt) for c in range(256)])


def fp8_encode(x, fmt: str) -> np.ndarray:
    """Codes of fp64 values: to the nearest finite value of the format, ties
    to the even code, saturating; NaN to the positive NaN code 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    top = 0x7e if fmt == "e4m3" else 0x7b  # code of MAX
    values = fp8_table(fmt)[:top + 1]      # non-negative finite values, ascending
    with np.errstate(invalid="ignore"):
        a = np.minimum(np.abs(x), FP8_MAX[fmt])
    a = np.where(np.isnan(x), 0.0, a)
    hi = np.minimum(np.searchsorted(values, a, side="left"), top)
    lo = np.maximum(hi - 1, 0)
    below, above = a - values[lo], values[hi] - a
    pick_lo = (below < above) | ((below == above) & (lo % 2 == 0))
    code = np.where(pick_lo, lo, hi).astype(np.uint8)
    code = code | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7f), code)


def _widen16(x, dtype: str) -> np.ndarray:
    """fp16 / bf16 storage (torch or numpy) as exact fp64 values."""
    u = oracle._as_u16(x)
    if dtype == "f16":
        return u.view(np.float16).astype(np.float64)
    return (u.astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def _rows(b, kv_indptr, kv_indices, last_page_len, page_size):
    """Pool rows of request b's tokens, in order."""
    n = int(kv_indptr[b + 1]) - int(kv_indptr[b])
    length = (n - 1) * page_size + int(last_page_len[b]) if n > 0 else 0
    t = np.arange(length)
    return np.asarray(kv_indices, dtype=np.int64)[int(kv_indptr[b]) + t // page_size] * page_size \
        + t % page_size


def scale_for(a: float, fmt: str) -> float:
    """The smallest power of two in [2^-60, 2^60] with a <= MAX * scale."""
    s = 2.0 ** -60
    while a > FP8_MAX[fmt] * s and s < 2.0 ** 60:
        s *= 2.0
    return s


def kv_append(x, codes, scales, qo_indptr, kv_indptr, kv_indices, last_page_len, *, page_size,
              scale_block, dtype, fmt):
    """Quantise each request's last tokens into copies of ``codes`` (uint8
    ``[pages, P, Hkv, D]``) and ``scales`` (``[pages * P / scale_block,
    Hkv]``); ``x`` is ``[total_q, Hkv, D]`` in 16 bits.  Returns both."""
    shape = codes.shape
    hkv, d = shape[2], shape[3]
    codes = np.array(codes, dtype=np.uint8).reshape(-1, hkv, d)
    scales = np.array(scales, dtype=np.float64).reshape(-1, hkv)
    table = fp8_table(fmt)
    values = _widen16(x, dtype).reshape(-1, hkv, d)
    for b in range(len(last_page_len)):
        rows = _rows(b, kv_indptr, kv_indices, last_page_len, page_size)
        first = len(rows) - (int(qo_indptr[b + 1]) - int(qo_indptr[b]))
        for s0 in range(first // scale_block * scale_block, len(rows), scale_block):
            old = np.arange(s0, max(s0, min(first, s0 + scale_block)))
            new = np.arange(max(s0, first), min(s0 + scale_block, len(rows)))
            if len(new) == 0:
                continue
            block = rows[new[0]] // scale_block
            for h in range(hkv):
                y = values[int(qo_indptr[b]) + new - first, h]
                mag = np.abs(y[np.isfinite(y)])
                s = scale_for(float(mag.max()) if mag.size else 0.0, fmt)
                if len(old):
                    was = scales[block, h]
                    s = max(s, was)
                    if s > was:
                        kept = table[codes[rows[old], h]]
                        codes[rows[old], h] = fp8_encode(kept * (was / s), fmt)
                scales[block, h] = s
                codes[rows[new], h] = fp8_encode(y / s, fmt)
    return codes.reshape(shape), scales


def cached_rows(pool, rows, *, dtype, fmt=None, scales=None, scale_block=0, scale=1.0):
    """fp64 keys or values of pool rows: 16-bit pools, 8-bit pools with one
    scale, or 8-bit pools with block scales."""
    hkv, d = pool.shape[2], pool.shape[3]
    if fmt is None:
        return _widen16(pool, dtype).reshape(-1, hkv, d)[rows]
    x = fp8_table(fmt)[oracle._as_u8(pool).reshape(-1, hkv, d)[rows]]
    if scales is None:
        return x * scale
    s = scales.detach().cpu().numpy() if hasattr(scales, "detach") else np.asarray(scales)
    return x * s.astype(np.float64).reshape(-1, hkv)[rows // scale_block][..., None]


def kv_read(pool, scales, kv_indptr, kv_indices, last_page_len, *, page_size, scale_block, dtype,
            fmt, new=None):
    """fp64 values of each request's last ``new[b]`` tokens (all by default),
    requests end to end: [total, Hkv, D], before rounding to ``dtype``."""
    out = []
    for b in range(len(last_page_len)):
        rows = _rows(b, kv_indptr, kv_indices, last_page_len, page_size)
        n = len(rows) if new is None else int(new[b])
        out.append(cached_rows(pool, rows[len(rows) - n:], dtype=dtype, fmt=fmt, scales=scales,
                               scale_block=scale_block))
    return np.concatenate(out)


def _rotate(x, pos, theta):
    """Rotate-half rotary positions of [n, heads, D] rows at positions [n]."""
    d = x.shape[-1] // 2
    ang = np.asarray(pos, dtype=np.float64)[:, None, None] * theta ** (-np.arange(d) / d)
    lo, hi = x[..., :d], x[..., d:]
    return np.concatenate([lo * np.cos(ang) - hi * np.sin(ang),
                           hi * np.cos(ang) + lo * np.sin(ang)], axis=-1)


def attention(q, k_pool, v_pool, kv_indptr, kv_indices, last_page_len, *, num_qo_heads,
              num_kv_heads, page_size, dtype, sm_scale, qo_indptr=None, causal=True, fmt=None,
              k_scales=None, v_scales=None, scale_block=0, k_scale=1.0, v_scale=1.0,
              logit_cap=0.0, alibi_slopes=None, rope_theta=0.0):
    """Attention with the options of ``pa_attention_options``, in fp64.

    Decode without ``qo_indptr`` (one query token per request, the last one),
    else prefill / append.  Returns o [rows, Hq, D] and lse [rows, Hq].
    """
    batch = len(last_page_len)
    qv = _widen16(q, dtype).reshape(-1, num_qo_heads, q.shape[-1])
    if qo_indptr is None:
        qo_indptr = np.arange(batch + 1)
    o, lse = np.zeros(qv.shape), np.full(qv.shape[:2], -np.inf)
    g = num_qo_heads // num_kv_heads
    if alibi_slopes is not None:
        alibi_slopes = np.asarray(alibi_slopes.detach().cpu() if hasattr(alibi_slopes, "detach")
                                  else alibi_slopes, dtype=np.float64)
    for b in range(batch):
        rows = _rows(b, kv_indptr, kv_indices, last_page_len, page_size)
        q0, q1 = int(qo_indptr[b]), int(qo_indptr[b + 1])
        if len(rows) == 0 or q0 == q1:
            continue
        k = cached_rows(k_pool, rows, dtype=dtype, fmt=fmt, scales=k_scales,
                        scale_block=scale_block, scale=k_scale)
        v = cached_rows(v_pool, rows, dtype=dtype, fmt=fmt, scales=v_scales,
                        scale_block=scale_block, scale=v_scale)
        pos = len(rows) - (q1 - q0) + np.arange(q1 - q0)
        t = np.arange(len(rows))
        qb = qv[q0:q1]
        if rope_theta:
            qb, k = _rotate(qb, pos, rope_theta), _rotate(k, t, rope_theta)
        for h in range(num_qo_heads):
            with np.errstate(invalid="ignore"):
                s = sm_scale * (qb[:, h] @ k[:, h // g].T)
            if logit_cap:
                s = logit_cap * np.tanh(s / logit_cap)
            if alibi_slopes is not None:
                s = s - alibi_slopes[h] * (pos[:, None] - t)
            if causal:
                s = np.where(t <= pos[:, None], s, -np.inf)
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            lse[q0:q1, h] = (m + np.log(p.sum(axis=1, keepdims=True)))[:, 0]
            o[q0:q1, h] = p @ v[:, h // g] / p.sum(axis=1, keepdims=True)
    return o, lse
