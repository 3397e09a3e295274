"""Plain 64-bit forms of the operators around the decode step: prompt
attention, absorbed queries, gathered attention weights and cache eviction.
Test infrastructure only: numpy, one sequence and head at a time, written from
the definitions in include/mlra_serving.h.

Beside each result stand the sums that a bound on a kernel's error is made of,
so that the tests' tolerances come from the inputs and the number formats.
"""
from __future__ import annotations

import numpy as np

PAGE = 64
LOG2E = 1.4426950408889634


def rope(x, pos, base=10000.0):
    """Interleaved pairs of the last axis turned by pos * base^(-2i/d_r); pos broadcasts against x[..., 0]."""
    d = x.shape[-1]
    ang = np.asarray(pos, dtype=np.float64)[..., None] * base ** (-np.arange(0, d, 2) / d)
    c, s = np.cos(ang), np.sin(ang)
    out = np.empty_like(x, dtype=np.float64)
    out[..., 0::2] = x[..., 0::2] * c - x[..., 1::2] * s
    out[..., 1::2] = x[..., 0::2] * s + x[..., 1::2] * c
    return out


def cached(pool, row, n):
    """The first n tokens of the sequence whose page-table row is `row`."""
    return pool[row[:-(-n // PAGE)]].reshape(-1, pool.shape[-1])[:n]


def prompt(q_nope, q_rope, cu_q, k_nope, v, cu_k, rope_cache, page_table, scale):
    """(out, lse, spread, rot): attention of packed prompts.  spread = sum_j p_j |v_j| of each output, rot =
    the largest scale * sum |q_rot| |k| over a row's keys, dot = the largest scale * sum |q| |k| over all dims."""
    T, H, _ = q_nope.shape
    group = H // k_nope.shape[1]
    out = np.zeros((T, H, v.shape[2]))
    lse = np.full((T, H), -np.inf)
    spread, rot, dot = np.zeros_like(out), np.zeros((T, H)), np.zeros((T, H))
    for b in range(len(cu_q) - 1):
        lk = cu_k[b + 1] - cu_k[b]
        keys = cached(rope_cache, page_table[b], lk)
        for i in range(cu_q[b], cu_q[b + 1]):
            pos = lk - cu_q[b + 1] + i
            n = max(0, pos + 1)
            if n == 0:
                continue
            for h in range(H):
                q = rope(q_rope[i, h], pos)
                k, val = k_nope[cu_k[b]:cu_k[b] + n, h // group], v[cu_k[b]:cu_k[b] + n, h // group]
                x = scale * (k @ q_nope[i, h] + keys[:n] @ q)
                p = np.exp(x - x.max())
                lse[i, h] = (x.max() + np.log(p.sum())) * LOG2E
                p /= p.sum()
                out[i, h], spread[i, h] = p @ val, p @ np.abs(val)
                rot[i, h] = scale * (np.abs(keys[:n]) @ np.abs(q)).max()
                dot[i, h] = rot[i, h] + scale * (np.abs(k) @ np.abs(q_nope[i, h])).max()
    return out, lse, spread, rot, dot


def absorb(q_nope, q_rope, q_pos, W_UK, scale):
    """(q_abs, size): the absorbed query and the sum of absolute products behind each of its values."""
    lat, size = np.einsum("bhd,hdc->bhc", q_nope, W_UK), np.einsum("bhd,hdc->bhc", np.abs(q_nope), np.abs(W_UK))
    pairs = np.abs(q_rope).reshape(*q_rope.shape[:-1], -1, 2).sum(-1).repeat(2, -1)
    f = scale * LOG2E
    return f * np.concatenate((lat, rope(q_rope, q_pos[:, None])), -1), f * np.concatenate((size, pairs), -1)


def weights(q_abs, lse, latent, rope_cache, page_table, seq_lens, n_branch):
    """(p, size) per sequence: the attention weight of each of its tokens, summed over heads and branches, and the
    same sum with each term times the sum of absolute products in its exponent."""
    d_c = latent.shape[-1]
    out = []
    for b, n in enumerate(seq_lens):
        c, k = cached(latent, page_table[b], n), cached(rope_cache, page_table[b], n)
        p, size = np.zeros(n), np.zeros(n)
        for r in range(n_branch):
            cols = slice(r * d_c // n_branch, (r + 1) * d_c // n_branch)
            key, q = np.concatenate((c[:, cols], k), 1), np.concatenate((q_abs[b][:, cols], q_abs[b][:, d_c:]), 1)
            for h in range(q.shape[0]):
                if lse[b, r, h] == -np.inf:
                    continue
                w = np.exp2(key @ q[h] - lse[b, r, h])
                p += w
                size += w * (np.abs(key) @ np.abs(q[h]) + abs(lse[b, r, h]))
        out.append((p, size))
    return out


def evict(weights_, page_table, seq_lens, evict_pages, recent):
    """Per sequence: (moves [(from slot, to slot)], new weights row, new table row, new length)."""
    slots = weights_.shape[1]
    out = []
    for w, row, n, pages in zip(weights_, page_table, seq_lens, evict_pages):
        free = PAGE * pages
        order = sorted(range(max(0, n - recent)),
                       key=lambda t: (-np.inf if np.isnan(w[t]) else w[t], -t))
        gone = set(order[:free])
        src = [t for t in range(free) if t not in gone]
        dst = [t for t in range(free, n) if t in gone]
        new = w[:n].copy()
        new[dst] = w[src]
        out.append((list(zip(src, dst)), np.concatenate((new[free:], np.zeros(slots - (n - free), new.dtype))),
                    np.concatenate((row[pages:], np.full(pages, -1, row.dtype))), n - free))
    return out
