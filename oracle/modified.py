"""CPU fp64 oracle for attention with modified scores — test infrastructure only.

One sequence at a time: q [n, H, D] at positions ``pos_q`` [n], k and v [m, H_kv, D]
at positions ``pos_k`` [m], ``seen`` [n, m] the visible pairs.

  x_ij = scale q_i . k_j
  s_ij = cap tanh(x_ij / cap) - slopes[h] |pos_q[i] - pos_k[j]|     (cap None: x_ij)
  P = softmax of the visible scores,  O = P V,  L = ln sum exp(s)
  dV = P^T dO,  dP = dO V^T,  dS = P o (dP - rowsum(P o dP)),
  dX = dS o (1 - tanh^2(x / cap)),  dQ = scale dX K,  dK = scale dX^T Q

A row that sees no key has O = 0, L = -inf and no gradient.  Each head also yields
the matrices that error bounds are made of.
"""
from __future__ import annotations

import math

import torch

from .attention import F64, as_f64, softmax_rows


def visible(n: int, causal: bool, window=None, prefix: int = 0) -> torch.Tensor:
    """[n, n]: key j to row i iff i - left <= j and (j <= i + right or j < prefix)."""
    i, j = torch.arange(n)[:, None], torch.arange(n)[None, :]
    left, right = (-1, -1) if window is None else window
    right = 0 if causal else right
    seen = torch.ones(n, n, dtype=torch.bool) if right < 0 else (j <= i + right) | (j < prefix)
    return seen if left < 0 else seen & (j >= i - left)


def head(q, k, v, seen, pos_q, pos_k, scale, softcap=None, slope=None, do=None):
    """One head: a dict of o, lse and, with ``do``, dq, dk, dv (this head's share); and p, s, x, ds, f."""
    q, k, v = as_f64(q), as_f64(k), as_f64(v)
    x = scale * q @ k.T
    t = torch.zeros_like(x) if softcap is None else torch.tanh(x / softcap)
    s = x if softcap is None else softcap * t
    bias = torch.zeros_like(x)
    if slope is not None:
        bias = -float(slope) * (pos_q.to(F64)[:, None] - pos_k.to(F64)[None, :]).abs()
    s = (s + bias).masked_fill(~seen, -math.inf)
    p, lse = softmax_rows(s)
    r = {"x": x, "s": s, "bias": bias, "p": p, "lse": lse, "o": p @ v, "f": 1 - t * t}
    if do is not None:
        do = as_f64(do)
        dp = do @ v.T
        r["dp"] = dp
        r["g"] = dp - (p * dp).sum(-1, keepdim=True)
        r["ds"] = p * r["g"] * r["f"]
        r["dq"], r["dk"], r["dv"] = scale * r["ds"] @ k, scale * r["ds"].T @ q, p.T @ do
    return r


def sequence(q, k, v, seen, pos_q, pos_k, scale, softcap=None, slopes=None, do=None):
    """All heads: list of ``head`` results of query head h on K/V head h // (H / H_kv)."""
    H, hk = q.shape[1], k.shape[1]
    return [head(q[:, h], k[:, h // (H // hk)], v[:, h // (H // hk)], seen, pos_q, pos_k, scale, softcap,
                 None if slopes is None else slopes[h], None if do is None else do[:, h]) for h in range(H)]
