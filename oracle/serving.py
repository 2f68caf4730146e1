"""fp64 reference of the serving operators around the decode: the cache append with
position rotation, decode over a sliding window and sinks, and decode of a batch that
shares a prefix (test infrastructure; see package docstring).

The attention functions also return what a rounding bound needs: per output the sum
``sum_t p_t |row_t|`` that rounded weights can move it by, and per row the largest
``|scale| sum_j |q_j row_t,j|`` over its tokens, which bounds a score's rounding.
"""
from __future__ import annotations

import numpy as np

from .mla_oracle import bf16_to_f64, gather_rows


def _attend(q, rows, scale, d_v):
    """q [H, D] over rows [n, D] (n >= 1): out, lse, sum p|v|, max_t |scale| sum |q||row|."""
    s = scale * (q @ rows.T)
    m = s.max(axis=1, keepdims=True)
    e = np.exp(s - m)
    l = e.sum(axis=1, keepdims=True)
    p = e / l
    v = rows[:, :d_v]
    return p @ v, (m + np.log(l))[:, 0], p @ np.abs(v), (abs(scale) * (np.abs(q) @ np.abs(rows).T)).max(axis=1)


def _outputs(q, d_v):
    B, SQ, H, _ = q.shape
    return (np.zeros((B, SQ, H, d_v)), np.full((B, SQ, H), -np.inf), np.zeros((B, SQ, H, d_v)), np.zeros((B, SQ, H)))


def mla_decode_window_ref(q, kv_cache, block_table, cache_seqlens, softmax_scale, window, sinks=0, *, d_v=512,
                          page_size=64):
    """Query i of sequence b sits at p = T_b - s_q + i and sees the cached tokens t <= p with
    t < sinks or t > p - window.  A query that sees none gives out = 0, lse = -inf.
    q [B, s_q, H, D]; table entries of pages without a visible token are not looked at."""
    res = _outputs(q, d_v)
    B, SQ = q.shape[:2]
    for b in range(B):
        T = int(cache_seqlens[b])
        for i in range(SQ):
            p = T - SQ + i
            t = np.arange(max(p + 1, 0))
            t = t[(t < sinks) | (t > p - window)]
            if not t.size:
                continue
            if block_table is None:
                rows = bf16_to_f64(kv_cache[b][t])
            else:
                rows = bf16_to_f64(kv_cache[np.asarray(block_table[b], dtype=np.int64)[t // page_size], t % page_size])
            for r, x in zip(res, _attend(bf16_to_f64(q[b, i]), rows, softmax_scale, d_v)):
                r[b, i] = x
    return res


def mla_decode_shared_ref(q, kv_cache, prefix_table, prefix_len, block_table, cache_seqlens, softmax_scale, *, d_v=512,
                          page_size=64):
    """Each sequence's cache is the prefix's tokens, then its own; query i sees the first
    P + T_b - s_q + 1 + i of them."""
    res = _outputs(q, d_v)
    B, SQ = q.shape[:2]
    pre = gather_rows(kv_cache, np.asarray(prefix_table)[None], 0, int(prefix_len), page_size)
    for b in range(B):
        T = int(cache_seqlens[b])
        rows = np.concatenate([pre, gather_rows(kv_cache, block_table, b, T, page_size)])
        for i in range(SQ):
            n = len(rows) - SQ + 1 + i
            if n <= 0:
                continue
            for r, x in zip(res, _attend(bf16_to_f64(q[b, i]), rows[:n], softmax_scale, d_v)):
                r[b, i] = x
    return res


def rotate_ref(x, cos_sin, interleaved):
    """x [..., 64] with pair i turned by the angle of (cos_sin[..., i], cos_sin[..., 32 + i])."""
    x, cs = bf16_to_f64(x), np.asarray(cos_sin, dtype=np.float64)
    z = cs[..., :32] + 1j * cs[..., 32:]
    if interleaved:
        v = (x[..., 0::2] + 1j * x[..., 1::2]) * z
        return np.stack([v.real, v.imag], -1).reshape(x.shape)
    v = (x[..., :32] + 1j * x[..., 32:]) * z
    return np.concatenate([v.real, v.imag], -1)


def mla_append_ref(c_kv, k_rope, q_rope, cos_sin, cu_tokens, cache_seqlens, pos_offset, block_table, interleaved, *,
                   page_size=64):
    """What the append writes: a list of (page or sequence, row in it, token, row values [576]
    in fp64) and q_out [N, H, 64] in fp64 (None without q_rope; NaN for padding tokens)."""
    writes = []
    q_out = None if q_rope is None else np.full(q_rope.shape, np.nan)
    for b in range(len(cache_seqlens)):
        lo, hi = int(cu_tokens[b]), int(cu_tokens[b + 1])
        for n in range(lo, hi):
            r = int(cache_seqlens[b]) - (hi - lo) + (n - lo)
            cs = cos_sin[r + (0 if pos_offset is None else int(pos_offset[b]))]
            row = np.concatenate([bf16_to_f64(c_kv[n]), rotate_ref(k_rope[n], cs, interleaved)])
            where = (b, r) if block_table is None else (int(block_table[b][r // page_size]), r % page_size)
            writes.append((*where, n, row))
            if q_rope is not None:
                q_out[n] = rotate_ref(q_rope[n], cs[None], interleaved)
    return writes, q_out
