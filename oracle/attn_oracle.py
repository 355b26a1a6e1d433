"""Plain binary64 forms of the operators around the quantised projections: rotary positions,
low-rank adapters, block means, the choice of key blocks and attention over them.

Written from the formulas, one row, pair or block at a time; slow on purpose.  Inputs are numpy
arrays of any float type (exact in binary64); outputs are binary64 and unrounded, except the block
means, which the definition rounds once to binary32.
"""

from __future__ import annotations

import numpy as np

BLOCK_Q, BLOCK_K = 128, 64


def rope(x, positions, inv_freq, pair_axis=None, interleaved=True, scale=1.0, inverse=False):
    """x [rows, heads, dim], positions [rows, axes] or [rows] integers."""
    x = np.asarray(x, dtype=np.float64)
    pos = np.asarray(positions).reshape(x.shape[0], -1)
    n = len(inv_freq)
    y = x.copy()
    for p in range(n):
        axis = 0 if pair_axis is None else int(pair_axis[p])
        # the angle is a binary64 product by definition; its sine and cosine go by numpy
        a = pos[:, axis].astype(np.float64) * np.float64(inv_freq[p])
        c, s = (np.cos(a) * scale)[:, None], (np.sin(a) * scale)[:, None]
        if inverse:
            s = -s
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + n)
        u, v = x[:, :, i], x[:, :, j]
        y[:, :, i] = u * c - v * s
        y[:, :, j] = u * s + v * c
    return y


def lora_add(y, x, a, b, seg_start, seg_adapter, scale=None, out=None):
    """(out, t_abs): out as the operator gives it, unrounded; rows outside every request are
    `out`'s (or y's).  t_abs[m][n] bounds the terms summed for an element: sum_r |B| sum_k |A||x|."""
    y, x, a, b = (np.asarray(v, dtype=np.float64) for v in (y, x, a, b))
    got = (y if out is None else np.asarray(out, dtype=np.float64)).copy()
    size = np.zeros_like(got)
    for lo, hi, i in zip(seg_start[:-1], seg_start[1:], seg_adapter):
        got[lo:hi] = y[lo:hi]
        if i >= 0:
            s = 1.0 if scale is None else float(scale[i])
            got[lo:hi] += s * ((x[lo:hi] @ a[i].T) @ b[i].T)
            size[lo:hi] = abs(s) * ((np.abs(x[lo:hi]) @ np.abs(a[i]).T) @ np.abs(b[i]).T)
    return got, size


def block_means(x, lens=None, size=BLOCK_K):
    """x [B, L, H, D] -> binary32 [B, H, blocks, D]."""
    x = np.asarray(x, dtype=np.float64)
    B, L, H, D = x.shape
    out = np.zeros((B, H, -(-L // size), D), dtype=np.float32)
    for b in range(B):
        end = L if lens is None else int(lens[b])
        for j in range(-(-end // size)):
            rows = x[b, j * size : min((j + 1) * size, end)]
            out[b, :, j] = (rows.sum(0) / rows.shape[0]).astype(np.float32)
    return out


def seen_keys(row, q_len, k_len, causal):
    """How many leading keys a query row sees."""
    return max(0, min(k_len, row + 1 + k_len - q_len)) if causal else k_len


def block_select(q, means, count, keys, first=0, last=0, causal=False, q_len=None, k_len=None):
    q = np.asarray(q, dtype=np.float64)
    B, Lq, Hq, _ = q.shape
    group = Hq // means.shape[1]
    nq = -(-Lq // BLOCK_Q)
    out = np.full((B, Hq, nq, count), -1, dtype=np.int32)
    qm = block_means(q, q_len, BLOCK_Q)
    for b in range(B):
        ql = Lq if q_len is None else int(q_len[b])
        kl = keys if k_len is None else int(k_len[b])
        for i in range(-(-ql // BLOCK_Q)):
            n = -(-seen_keys(min((i + 1) * BLOCK_Q, ql) - 1, ql, kl, causal) // BLOCK_K)
            for h in range(Hq):
                score = [float(np.dot(qm[b, h, i].astype(np.float64), means[b, h // group, j].astype(np.float64)))
                         for j in range(n)]
                always = [j < first or j >= n - last for j in range(n)]
                rank = sorted(range(n), key=lambda j: (not always[j], np.isnan(score[j]),
                                                       0.0 if always[j] or np.isnan(score[j]) else -score[j], j))
                chosen = sorted(rank[:count])
                out[b, h, i, : len(chosen)] = chosen
    return out


def block_attention(q, k, v, blocks, scale=None, causal=False, q_len=None, k_len=None, out=None, lse=None):
    """(out, lse, size): size[b, i, h, d] = sum_j p_ij |v_jd| / sum_j p_ij."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    B, Lq, Hq, D = q.shape
    Lk, group = k.shape[1], Hq // k.shape[2]
    scale = D ** -0.5 if scale is None else scale
    o = np.zeros_like(q) if out is None else np.asarray(out, dtype=np.float64).copy()
    z = np.full((B, Hq, Lq), -np.inf) if lse is None else np.asarray(lse, dtype=np.float64).copy()
    size = np.zeros_like(q)
    for b in range(B):
        ql = Lq if q_len is None else int(q_len[b])
        kl = Lk if k_len is None else int(k_len[b])
        for h in range(Hq):
            for i in range(-(-ql // BLOCK_Q)):
                at = [j * BLOCK_K + e for j in blocks[b, h, i] if 0 <= j * BLOCK_K < kl
                      for e in range(min(BLOCK_K, kl - j * BLOCK_K))]
                at = np.array(at, dtype=np.int64)
                for r in range(i * BLOCK_Q, min((i + 1) * BLOCK_Q, ql)):
                    mine = at[at < seen_keys(r, ql, kl, causal)]
                    if mine.size == 0:
                        o[b, r, h], z[b, h, r] = 0.0, -np.inf
                        continue
                    s = scale * (k[b, mine, h // group] @ q[b, r, h])
                    p = np.exp(s - s.max())
                    o[b, r, h] = p @ v[b, mine, h // group] / p.sum()
                    size[b, r, h] = p @ np.abs(v[b, mine, h // group]) / p.sum()
                    z[b, h, r] = s.max() + np.log(p.sum())
    return o, z, size
