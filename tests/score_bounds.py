"""Error bounds of attention with modified scores, element by element, from the roundings the kernels make.

u is half a step of the 16-bit type.  First order in each error, the product of two covered by a factor 1.1.

A score's error e_ij: products of D terms summed in fp32, truncated at worst, scale sum_d |q_d k_d| (D + 4) 2^-23;
under a cap, its arithmetic: 2^-19 of the score where |x| <= 1.25 cap (a minimax polynomial with a relative error
under 2^-20, and fp32's roundings), 2^-20 of the cap beyond (the derivative of tanh is at most 1, so the
product's error does not grow); the bias and the sums with the row's maximum or L: 2^-22 (|s| +
|bias| + |L|); its exponential, 2^-21.

A weight p_ij is off by e_ij p_ij, and by the row's sum: c_i p_ij with c_i = sum_j p_ij e_ij + n 2^-24 (fp32 sums of n
terms).  O: P is rounded to 16 bits (u p_ij; in fp16 also half a subnormal step, 2^-25, of weights relative to the
row's maximum, where their sum is 1 at least: 2^-25 sum_j |v_j| e^(max s - L)), V's product sums in fp32 (n 2^-24),
and O is rounded once (u |O|, fp16's subnormals 2^-25).  L: c_i + 2^-22 |L| + 2^-21.

Backward: P = exp(s - L) is off by (e_ij + errL_i) p_ij and rounded (u p_ij; fp16 2^-25).  Delta_i as from the stored O (the kernels do better: test_scores_edges.py has that bound):
sum_d |dO_d| (errO_d + D 2^-24 |O_d|); dP: D 2^-23 sum_d |dO_d v_d|; g = dP - Delta, so dS = p g f is off by
  (e_ij + errL_i + u) |dS_ij| + p_ij f_ij (err dP + err Delta) + p_ij |g_ij| errf_ij + 2^-25 (fp16),
errf = 2 |t| err t + 2^-22 with err t = (error of the product) / cap + 2^-19 |t|.  The products over n rows or keys sum in
fp32: n 2^-23 of their absolute terms.
"""
import math

import torch

from oracle.attention import as_f64

F = 1.1


def score_error(r, q, k, scale, softcap):
    D = q.shape[-1]
    ex = abs(scale) * (D + 4) * 2.0 ** -23 * (as_f64(q).abs() @ as_f64(k).abs().T)
    e = ex + 2.0 ** -21
    if softcap is not None:
        e = e + 2.0 ** -19 * torch.minimum(r["x"].abs(), torch.full_like(ex, softcap))
    s = torch.where(torch.isfinite(r["s"]), r["s"], torch.zeros_like(r["s"]))
    l = torch.where(torch.isfinite(r["lse"]), r["lse"], torch.zeros_like(r["lse"]))
    return ex, e + 2.0 ** -22 * (s.abs() + r["bias"].abs() + l.abs()[:, None])


def forward_bounds(r, q, k, v, scale, softcap, dtype):
    """(bound of O, bound of L, score errors) of one head."""
    u = torch.finfo(dtype).eps / 2
    n = r["p"].shape[1]
    ex, e = score_error(r, q, k, scale, softcap)
    p, va = r["p"], as_f64(v).abs()
    c = (p * e).sum(1) + n * 2.0 ** -24
    tol = (p * (u + e)) @ va + (c[:, None] + n * 2.0 ** -24) * (p @ va) + u * r["o"].abs() + 1e-12
    if dtype == torch.float16:
        top = torch.where(torch.isfinite(r["lse"]), r["s"].amax(1) - r["lse"], torch.full_like(r["lse"], -math.inf))
        seen = (r["s"] > -math.inf).double()
        tol = tol + 2.0 ** -25 * (1 + (seen @ va) * torch.exp(top)[:, None])
    lse = torch.where(torch.isfinite(r["lse"]), r["lse"], torch.zeros_like(r["lse"]))
    return F * tol, F * (c + 2.0 ** -22 * lse.abs() + 2.0 ** -21), (ex, e)


def backward_bounds(r, q, k, v, do, scale, softcap, dtype):
    """Bounds of this head's dQ, dK, dV before they are summed and stored (add u |result|)."""
    u = torch.finfo(dtype).eps / 2
    sub = 2.0 ** -25 if dtype == torch.float16 else 0.0
    n, D = r["p"].shape[1], q.shape[-1]
    tol_o, tol_l, (ex, e) = forward_bounds(r, q, k, v, scale, softcap, dtype)
    qa, ka, va, da = (as_f64(x).abs() for x in (q, k, v, do))
    p, g, f = r["p"], r["g"].abs(), r["f"]
    ep = e + tol_l[:, None]
    seen = (r["s"] > -math.inf).double()
    delta = (da * (tol_o + D * 2.0 ** -24 * r["o"].abs())).sum(1)
    dp = D * 2.0 ** -23 * (da @ va.T)
    ds = (ep + u) * r["ds"].abs() + p * f * (dp + delta[:, None]) + sub * seen
    if softcap is not None:
        t = torch.sqrt((1 - f).clamp(min=0))
        ds = ds + p * g * (2 * t * (ex / softcap + 2.0 ** -19 * t + 2.0 ** -21) + 2.0 ** -22)
    acc = n * 2.0 ** -23
    dsa = r["ds"].abs()
    dq = abs(scale) * ((ds + acc * dsa) @ ka)
    dk = abs(scale) * ((ds + acc * dsa).T @ qa)
    dv = (p * (ep + u + acc) + sub * seen).T @ da
    return F * dq + 1e-12, F * dk + 1e-12, F * dv + 1e-12
