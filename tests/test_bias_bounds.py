"""The error of distance biases that fa.h states: a one-sided block's arithmetic replayed in fp32 on the CPU, and far
keys under negative slopes on the GPU."""
import math

import numpy as np
import pytest
import torch

from tests.test_paged_scores import words_of
from tests.test_rope import ints, on_gpu, paged_setup
from tests.test_scores import rnd

F = np.float32
LOG2E = F(1.4426950408889634)
SCALES = [32 ** -0.5, 64 ** -0.5, 128 ** -0.5, 16 ** -0.5, 1.0, 0.037, 1e-3, 7.0, 1e4, -0.125]
CAPS = [50.0, 30.0, 20.0, 15.0, 5.0, 1.0, 0.01, 1e-4, 1e-10, 1000.0, 1e5, 1e10]


@pytest.mark.parametrize("cap", [None] + CAPS)
def test_bias_of_a_one_sided_block(cap):
    """Column and row parts as the forward kernels form them, for slopes that are not steep: 2^-21 of the bias, and
    2^-15 beside it."""
    g = np.random.default_rng(2)
    n = 200000
    slope = np.concatenate([g.random(n) * 1.03, 2.0 ** -(8 * g.random(n))]).astype(F)
    sign = np.where(g.random(2 * n) < 0.5, F(1), F(-1))
    near = np.floor(2.0 ** (20 * g.random(2 * n))).astype(np.int64)  # distance of the block's last column
    col = g.integers(0, 64, 2 * n)
    d0 = -(near + 63)
    s2 = (sign * slope * LOG2E).astype(F)
    units = [F(F(x) * LOG2E) for x in SCALES if x * LOG2E >= 1e-4] if cap is None else [F(cap * 1.4426950408889634074)]
    for unit in units:
        per = F(1) / unit
        su = (s2 * per).astype(F)
        fixed = ((su * d0.astype(F)).astype(F) * unit).astype(F)
        y = (su * col.astype(F)).astype(F)
        total = y.astype(np.float64) * np.float64(unit) + fixed.astype(np.float64)
        exact = (sign * slope).astype(np.float64) * math.log2(math.e) * (d0 + col)
        allowed = 2.0 ** -21 * np.abs(exact) + 2.0 ** -15 * math.log2(math.e)
        assert bool((np.abs(total - exact) <= allowed).all())


@pytest.fixture(scope="module")
def fa():
    import exact_attention_18_gb300 as m
    m.load_library()
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("softcap", [None, 20.0])
def test_far_keys_of_a_negative_slope(fa, softcap, dtype, D):
    """Scores of 0 under slopes that favour the farthest keys: L_i = ln sum_k e^(s k) over the i + 1 distances k, to
    2^-21 of the bias s i, 2^-15, and L's own roundings; O, whose weights are off by that much twice over."""
    S, H, n = 7777, 4, 300
    slopes = torch.tensor([-0.74557686, -1.03, -0.25, -1.5])
    q, k = torch.zeros(1, H, S, D, dtype=dtype), rnd((1, 1, S, D), 2, dtype)
    v = rnd((1, 1, S, D), 3, dtype)
    kw = dict(causal=True, softcap=softcap, slopes=slopes.cuda())
    u, sub = torch.finfo(dtype).eps / 2, 2.0 ** -25 if dtype == torch.float16 else 0.0
    o, lse = fa.forward(q.cuda(), k.cuda(), v.cuda(), **kw)
    kc, vc, table, cu = paged_setup([S], [n], 1, D, 64, dtype, 5)
    rows = (table[0][:-(-S // 64)].long()[:, None] * 64 + torch.arange(64)).reshape(-1)[:S]
    kc.view(-1, 1, D)[rows], vc.view(-1, 1, D)[rows] = k[0].transpose(0, 1), v[0].transpose(0, 1)
    kg, vg = on_gpu(kc, vc)
    chunks = []
    for m in (n, 3):
        out = fa.forward_paged(q[0, :, -m:].transpose(0, 1).contiguous().cuda(), kg, vg, ints(table), ints([S]),
                               ints([0, m]), m, S, **kw)
        chunks.append((m, out))
    assert fa.fa_check_device_errors(None) == 0
    i = torch.arange(S, dtype=torch.float64)
    for h in range(H):
        s = -float(slopes[h])
        tail = torch.exp(-s * (i + 1))
        ref = s * i + torch.log((1 - tail) / (1 - math.exp(-s)))
        off = 2.0 ** -21 * s * i + 2.0 ** -15 * max(1.0, s)
        tol = off + 3 * 2.0 ** -24 * ref + 2.0 ** -20
        vis = 64  # keys beyond weigh less than e^-16 of the first, and are added to the bound
        w = torch.exp(-s * torch.arange(vis, dtype=torch.float64))
        seen = (torch.arange(vis)[None, :] <= i[:, None]).double()
        p = seen * w / (seen * w).sum(1, keepdim=True)
        vv = v[0, 0, :vis].double()
        want, terms = p @ vv, p @ vv.abs()
        far = math.exp(-s * vis) / (1 - math.exp(-s)) * 8 * (i >= vis)
        for rows, lo, oo in ((i.long(), lse[0, h], o[0, h]), *((i[-m:].long(), x[1][h], x[0][:, h]) for m, x in chunks)):
            assert bool(((lo.cpu().double() - ref[rows]).abs() <= tol[rows]).all()), f"L h={h}"
            bound = u * want[rows].abs() + 1.1 * (u + 2 * off[rows] + 2.0 ** -18)[:, None] * terms[rows] \
                + far[rows][:, None] + sub * (1 + vv.abs().sum(0))
            assert bool(((oo.cpu().double() - want[rows]).abs() <= bound).all()), f"O h={h}"


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_gradient_of_a_negative_slope(fa, D):
    """dV = P^T dO with |L| up to 6000: each weight is off by 2^-20 |L| and half a 16-bit step, the sum over n rows by
    n 2^-23 of its terms."""
    S, H, dt = 2000, 2, torch.float16
    slopes = torch.tensor([-3.0, -0.7])
    q, k = torch.zeros(1, H, S, D, dtype=dt), rnd((1, H, S, D), 2, dt)
    v, do = rnd((1, H, S, D), 3, dt), rnd((1, H, S, D), 4, dt)
    g = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.forward(*g[:3], causal=True, slopes=slopes.cuda())
    dq, dk, dv = fa.backward(*g[:3], o, g[3], lse, causal=True, slopes=slopes.cuda())
    assert fa.fa_check_device_errors(None) == 0
    u, d = torch.finfo(dt).eps / 2, torch.arange(S)[:, None] - torch.arange(S)[None, :]
    for h in range(H):
        s = torch.where(d >= 0, -float(slopes[h]) * d.double(), torch.full((S, S), -math.inf, dtype=torch.float64))
        l = torch.logsumexp(s, 1)
        p, da = torch.exp(s - l[:, None]), do[0, h].double()
        want = p.T @ da
        tol = 1.1 * (p * (2.0 ** -20 * l[:, None] + u + S * 2.0 ** -23) + 2.0 ** -25 * (d >= 0)).T @ da.abs()
        tol += u * want.abs() + 2.0 ** -25
        assert bool(((dv[0, h].cpu().double() - want).abs() <= tol).all()), f"dV h={h}"
        assert not bool(dq.isnan().any()) and not bool(dk.isnan().any())


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("n", [12, 150, 1400])
def test_tree_whose_slots_are_far_from_its_positions(fa, n, D):
    """Drafted tokens in any order of the slots: a row's nearest keys lie hundreds of slots away, and their bias is off
    by no more for it.  Scores of 0; each row sees all positions up to its own: L_i = ln sum_d e^(-s d)."""
    f, H, dt = 300, 4, torch.float16
    kv = f + n
    slopes = torch.tensor([1.0, 0.73, 1.03, 0.31])
    kc, vc, table, cu = paged_setup([kv], [n], 1, D, 16, dt, 5)
    kg, vg = on_gpu(kc, vc)
    depth = torch.randperm(n, generator=torch.Generator().manual_seed(7))
    bits = depth[None, :] <= depth[:, None]
    words = -(-n // 32)
    o, lse = fa.forward_paged(torch.zeros(n, H, D, dtype=dt, device="cuda"), kg, vg, ints(table), ints([kv]), ints(cu), n,
                              kv, slopes=slopes.cuda(), tree=words_of(bits, words).cuda(),
                              positions=(f + depth).to(torch.int32).cuda())
    assert fa.fa_check_device_errors(None) == 0
    for h in range(H):
        s = float(slopes[h])
        ref = torch.log((1 - torch.exp(-s * (f + depth + 1).double())) / (1 - math.exp(-s)))
        tol = 2.0 ** -15 * max(1.0, s) + 2.0 ** -20
        assert bool(((lse[h].cpu().double() - ref).abs() <= tol).all()), f"L h={h}"
