"""Decode over a shared prefix, attention weights of cached tokens, and
eviction by them, in float64 and one (sequence, head) at a time.

Test infrastructure: only the tests may import this module.  The caches are
logical ones (see kv_cache); per-token scales come as [nb][Hkv][2][P].
"""
from __future__ import annotations

import math

import numpy as np

from .attention import decode_positions
from .kv_cache import BF16, bf16_bits_to_f32, codec, gather_scales, gather_tokens

P = 16


def tokens(k_cache, v_cache, k_scale, v_scale, table_row, pos, kv, cache_dtype, scale_cache=None, num_blocks=None):
    """Dequantized K and V [n][D] of the given positions, and which of them
    sit in a page with a valid block id (the others come as zeros)."""
    nb = k_cache.shape[0] if num_blocks is None else num_blocks
    row = np.asarray(table_row)
    good = (row >= 0) & (row < nb)
    safe = np.where(good, row, 0)
    kk, vv = gather_tokens(k_cache, v_cache, safe, pos, kv)
    if cache_dtype == BF16:
        k, v = bf16_bits_to_f32(kk).astype(np.float64), bf16_bits_to_f32(vv).astype(np.float64)
    else:
        k, v = codec(cache_dtype).decode(kk).astype(np.float64), codec(cache_dtype).decode(vv).astype(np.float64)
        if scale_cache is not None:
            k = k * gather_scales(scale_cache[:, :, 0], safe, pos, kv).astype(np.float64)[:, None]
            v = v * gather_scales(scale_cache[:, :, 1], safe, pos, kv).astype(np.float64)[:, None]
        else:
            k, v = k * float(k_scale[kv]), v * float(v_scale[kv])
    live = good[np.asarray(pos) // P]
    return np.where(live[:, None], k, 0.0), np.where(live[:, None], v, 0.0), live


def softmax_rows(q, k, live, sm_scale):
    """Probabilities [rows][n] over the live tokens; a row without any is zero."""
    p = np.zeros((q.shape[0], k.shape[0]))
    if live.any():
        s = (q @ k[live].T) * sm_scale
        e = np.exp(s - s.max(axis=1, keepdims=True))
        p[:, live] = e / e.sum(axis=1, keepdims=True)
    return p


def group_of(b, group_starts):
    for i in range(len(group_starts) - 1):
        if group_starts[i] <= b < group_starts[i + 1]:
            return i
    return None


def shared_prefix_decode(q, k_cache, v_cache, k_scale, v_scale, prefix_table, prefix_lens, group_starts, block_table,
                         seq_lens, sm_scale, cache_dtype):
    """(out [B][Hq][D], sum_j p_j |v_j| of the same shape)."""
    q = np.asarray(q, np.float64)
    B, Hq, D = q.shape
    H = k_cache.shape[1]
    g = Hq // H
    out, mag = np.zeros(q.shape), np.zeros(q.shape)
    for kv in range(H):
        pre = [tokens(k_cache, v_cache, k_scale, v_scale, prefix_table[i], np.arange(n), kv, cache_dtype)
               for i, n in enumerate(prefix_lens)]
        for b in range(B):
            k, v, live = tokens(k_cache, v_cache, k_scale, v_scale, block_table[b], np.arange(seq_lens[b]), kv, cache_dtype)
            i = group_of(b, group_starts)
            if i is not None:
                k, v, live = (np.concatenate([x, y]) for x, y in zip(pre[i], (k, v, live)))
            rows = slice(kv * g, (kv + 1) * g)
            p = softmax_rows(q[b, rows], k, live, sm_scale)
            out[b, rows], mag[b, rows] = p @ v, p @ np.abs(v)
    return out, mag


def decode_weights(q, k_cache, v_cache, k_scale, v_scale, block_table, seq_lens, weights, decay, sm_scale, window,
                   cache_dtype, scale_cache=None):
    """(out, sum p |v|, updated weights [B][H][W], sum over heads of p (sum_d |q_d k_jd|)
    sm_scale as a bound of the scores' size, per row: [B][Hq])."""
    q = np.asarray(q, np.float64)
    B, Hq, D = q.shape
    H = k_cache.shape[1]
    g = Hq // H
    out, mag, acc = np.zeros(q.shape), np.zeros(q.shape), np.array(weights, np.float64)
    size = np.zeros((B, Hq))
    for b in range(B):
        L = int(seq_lens[b])
        pos = decode_positions(L, window)
        for kv in range(H):
            acc[b, kv, :L] *= decay
            if pos.size == 0:
                continue
            k, v, live = tokens(k_cache, v_cache, k_scale, v_scale, block_table[b], pos, kv, cache_dtype, scale_cache)
            rows = slice(kv * g, (kv + 1) * g)
            p = softmax_rows(q[b, rows], k, live, sm_scale)
            out[b, rows], mag[b, rows] = p @ v, p @ np.abs(v)
            acc[b, kv, pos] += p.sum(axis=0)
            size[b, rows] = (np.abs(q[b, rows]) @ np.abs(k).T).max(axis=1) * sm_scale
    return out, mag, acc, size


def kept_positions(w, L, keep, sink, recent):
    """Ascending positions that one (sequence, head) keeps, by sorting."""
    n = min(L, keep)
    s = min(sink, n)
    r = min(recent, n - s)

    def order(j):
        x = float(w[j])
        return (1, 0.0, j) if math.isnan(x) else (0, -x, j)

    best = sorted(range(s, L - r), key=order)[:n - s - r]
    return list(range(s)) + sorted(best) + list(range(L - r, L))


def evict(weights, k_cache, v_cache, block_table, seq_lens, keep_lens, dst_table, dst_weights, kept, sink, recent,
          scale_cache=None):
    """In place on copies: (k_cache, v_cache, scale_cache, dst_weights, dst_lens, kept)."""
    k_cache, v_cache, dst_weights, kept = k_cache.copy(), v_cache.copy(), dst_weights.copy(), kept.copy()
    k0, v0 = k_cache.copy(), v_cache.copy()
    s0 = None if scale_cache is None else scale_cache.copy()
    scale_cache = None if scale_cache is None else scale_cache.copy()
    lens = []
    for b, L in enumerate(seq_lens):
        for h in range(weights.shape[1]):
            at = kept_positions(weights[b, h], int(L), int(keep_lens[b]), sink, recent)
            dst_weights[b, h] = 0.0
            for i, j in enumerate(at):
                src, dst = block_table[b][j // P], dst_table[b][i // P]
                kept[b, h, i] = j
                dst_weights[b, h, i] = weights[b, h, j]
                k_cache[dst, h, i % P] = k0[src, h, j % P]
                v_cache[dst, h, :, i % P] = v0[src, h, :, j % P]
                if s0 is not None:
                    scale_cache[dst, h, :, i % P] = s0[src, h, :, j % P]
        lens.append(min(int(L), int(keep_lens[b])))
    return k_cache, v_cache, scale_cache, dst_weights, np.array(lens, np.int32), kept
