"""float64 reference of the attention and eviction operators: attention of new
tokens over the paged FP8 cache, the attention weight each position received,
the choice of the positions to keep, their move, and packed prompt attention."""

from __future__ import annotations

import numpy as np

from . import formats


def slot_of(row: np.ndarray, j: int, block_size: int, num_slots: int) -> int:
    """Slot of position j under one row of a block table, -1 outside the pool."""
    b = int(row[j // block_size])
    if b < 0:
        return -1
    s = b * block_size + j % block_size
    return s if s < num_slots else -1


def spread_scales(scales: np.ndarray, heads: int, head_dim: int) -> np.ndarray:
    """Per-tensor, per-head or per-channel scales as [heads, head_dim]."""
    s = np.asarray(scales, np.float64).reshape(-1)
    if s.size == heads * head_dim:
        return s.reshape(heads, head_dim)
    return np.broadcast_to(s.reshape(-1, 1), (heads, head_dim))


def attend(q, k, v, limit, scale):
    """q [n, H, D] against k, v [L, Hk, D]; token i sees the positions j < limit[i].
    Returns out [n, H, D], lse [n, H], p [n, H, L], and for error bounds
    sum_j p_j |v_j| [n, H, D] and the largest scale * sum_c |q_c k_jc| of a seen position [n, H]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n, H, D = q.shape
    L, Hk = k.shape[:2]
    out, absv = np.zeros((n, H, D)), np.zeros((n, H, D))
    lse, smax, p_all = np.full((n, H), -np.inf), np.zeros((n, H)), np.zeros((n, H, L))
    seen = np.arange(L)[None, :] < np.asarray(limit).reshape(n, 1)
    for h in range(H):
        kh, vh = k[:, h // (H // Hk)], v[:, h // (H // Hk)]
        s = np.where(seen, q[:, h] @ kh.T * scale, -np.inf)
        a = np.where(seen, np.abs(q[:, h]) @ np.abs(kh).T * scale, 0.0)
        some = seen.any(1)
        m = np.where(some, s.max(1, initial=-np.inf), 0.0)
        e = np.exp(s - m[:, None])
        l = e.sum(1)
        p = e / np.where(some, l, 1.0)[:, None]
        lse[some, h] = (m + np.log(np.where(some, l, 1.0)))[some]
        out[:, h], absv[:, h] = p @ vh, p @ np.abs(vh)
        smax[:, h], p_all[:, h] = a.max(1, initial=0.0), p
    return out, lse, p_all, absv, smax


def kv_attention(q, k_cache, v_cache, table, block_size, q_starts, kv_lens, k_scales, v_scales, fmt, scale,
                 weights_in=None):
    """Per sequence: a dict with tokens (start, end) and attend()'s results, the weights [Hk, n positions], and for
    error bounds the sum of |v| over the positions [Hk, D]."""
    num_slots, Hk, D = k_cache.shape
    H = q.shape[1]
    ks, vs = spread_scales(k_scales, Hk, D), spread_scales(v_scales, Hk, D)
    got = []
    for b, L in enumerate(int(x) for x in kv_lens):
        t0, t1 = int(q_starts[b]), int(q_starts[b + 1])
        slots = np.array([slot_of(table[b], j, block_size, num_slots) for j in range(L)], np.int64).reshape(-1)
        live = np.flatnonzero(slots >= 0)
        k = formats.decode(k_cache[slots[live]], fmt).astype(np.float64) * ks
        v = formats.decode(v_cache[slots[live]], fmt).astype(np.float64) * vs
        # positions outside the pool are left out: the limit counts the live ones before it
        limit = [int(np.searchsorted(live, L - (t1 - t0) + i + 1)) for i in range(t1 - t0)]
        out, lse, p, absv, smax = attend(np.asarray(q[t0:t1], np.float64), k, v, limit, scale)
        w = np.zeros((Hk, L)) if weights_in is None else np.asarray(weights_in[b, :, :L], np.float64).copy()
        w[:, live] += p.reshape(t1 - t0, Hk, H // Hk, live.size).sum((0, 2))
        got.append({"tokens": (t0, t1), "out": out, "lse": lse, "absv": absv, "smax": smax, "weights": w,
                    "sumv": np.abs(v).sum(0)})
    return got


def evict_select(weights, kv_lens, keep, first, recent):
    """kept [batch, keep] (-1 behind the last) and kept_lens [batch]."""
    weights = np.asarray(weights, np.float32)
    batch = weights.shape[0]
    kept, lens = np.full((batch, keep), -1, np.int64), np.zeros(batch, np.int64)
    for b in range(batch):
        n = int(kv_lens[b])
        idx = np.arange(n)
        if n > keep:
            with np.errstate(invalid="ignore"):
                score = weights[b, :, :n].astype(np.float64).sum(0).astype(np.float32).astype(np.float64)
            forced = (idx < first) | (idx >= n - recent)
            # order: forced positions, then by score (NaN last), then by position
            nan = np.isnan(score)
            idx = np.lexsort((idx, -np.where(nan, 0.0, score), nan, ~forced))[:keep]
        kept[b, :idx.size], lens[b] = np.sort(idx), idx.size
    return kept, lens


def compact(cache, src_table, dst_table, block_size, kept, kept_lens):
    """The cache with row i under dst_table taken from row kept[b, i] under src_table."""
    out, num_slots = cache.copy(), cache.shape[0]
    for b in range(kept.shape[0]):
        for i in range(min(int(kept_lens[b]), kept.shape[1], dst_table.shape[1] * block_size)):
            j = int(kept[b, i])
            if not 0 <= j < src_table.shape[1] * block_size:
                continue
            s = slot_of(src_table[b], j, block_size, num_slots)
            d = slot_of(dst_table[b], i, block_size, num_slots)
            if s >= 0 and d >= 0:
                out[d] = cache[s]
    return out
