"""CPU fp64 oracle for attention over a paged key/value cache — test infrastructure only.

Key j of sequence b is row j % page_size of page block_table[b][j // page_size]
of the [pages, page_size, H_kv, D] caches.  Query i of the sequence's n new
tokens stands at position p = kv_len - n + i and sees keys
max(0, p - left) <= j <= min(kv_len - 1, p + right) (a negative side is
unlimited, causal makes right 0).  A row that sees none has O = 0, L = -inf.
"""
from __future__ import annotations

import math

import torch

from .attention import F64, as_f64


def slots(block_table_row, positions, page_size):
    """Flat cache rows (page * page_size + row) of key positions."""
    t = torch.as_tensor(block_table_row).to(torch.int64)
    p = torch.as_tensor(positions).to(torch.int64)
    return t[p // page_size] * page_size + p % page_size


def append(cache, rows, block_table, kv_lens, cu_seqlens):
    """The cache [pages, page_size, H_kv, D] with the new tokens' rows [T, H_kv, D] in their slots."""
    c = cache.clone()
    flat = c.reshape(-1, *c.shape[2:])
    for b, (t0, t1) in enumerate(zip(cu_seqlens[:-1], cu_seqlens[1:])):
        if t1 > t0:
            at = torch.arange(int(kv_lens[b]) - (t1 - t0), int(kv_lens[b]))
            flat[slots(block_table[b], at, c.shape[1])] = rows[t0:t1].to(c.dtype)
    return flat.view(c.shape)


def attend(q, k_cache, v_cache, block_table, kv_lens, cu_seqlens, causal=True, window=None, scale=None):
    """O [T, H, D], L [H, T], and per-row sums used by error bounds: W = sum_j p_j |v_j| [T, H, D]."""
    q = as_f64(q)
    T, H, D = q.shape
    hk = k_cache.shape[2]
    G = H // hk
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    left, right = (-1, -1) if window is None else window
    if causal:
        right = 0
    o, w = torch.zeros(T, H, D, dtype=F64), torch.zeros(T, H, D, dtype=F64)
    lse = torch.full((H, T), -math.inf, dtype=F64)
    for b, (t0, t1) in enumerate(zip(cu_seqlens[:-1], cu_seqlens[1:])):
        n, kv = t1 - t0, int(kv_lens[b])
        if n == 0 or kv == 0:
            continue
        p = torch.arange(kv - n, kv)
        lo = 0 if left < 0 else max(0, int(p[0]) - left)  # keys before it are never touched
        j = torch.arange(lo, kv)
        at = slots(block_table[b], j, k_cache.shape[1])
        k = as_f64(k_cache.reshape(-1, hk, D)[at])
        v = as_f64(v_cache.reshape(-1, hk, D)[at])
        seen = torch.ones(n, kv - lo, dtype=torch.bool)
        if left >= 0:
            seen &= j[None, :] >= p[:, None] - left
        if right >= 0:
            seen &= j[None, :] <= p[:, None] + right
        for h in range(H):
            s = scale * q[t0:t1, h] @ k[:, h // G].T
            s = s.masked_fill(~seen, -math.inf)
            m = s.amax(1, keepdim=True)
            e = torch.where(seen, torch.exp(s - m.clamp(min=-1e300)), torch.zeros_like(s))
            z = e.sum(1, keepdim=True)
            ok = z > 0
            pr = torch.where(ok, e / z.clamp(min=1e-300), torch.zeros_like(e))
            o[t0:t1, h] = pr @ v[:, h // G]
            w[t0:t1, h] = pr @ v[:, h // G].abs()
            lse[h, t0:t1] = torch.where(ok, m + z.clamp(min=1e-300).log(), torch.full_like(m, -math.inf))[:, 0]
    return o, lse, w
