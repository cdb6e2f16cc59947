"""Caps and slopes at the ends of their ranges together, on every kernel that forms modified scores.

Slopes this steep leave a row the keys at its smallest (a negative slope: largest) visible distance.  Bounds: O is a
mean of values summed in fp32 (n 2^-23 of their absolute terms) and rounded once; L is the bias, off by at most 2^-21
of itself, plus the logarithm of the number of keys, 2^-21 of fp32's arithmetic and the cap.

Keys at one distance share a row by what fp32 makes of them.  Where the product of slope and distance is halfway
between two fp32 numbers, the score beside it decides which one it is, so two such keys may be a step apart (here above
2^70).  And a chunk's keys may lie in the parts of several CTAs, joined by their fp32 L: a part with c of the keys has
L = m + log2 c, which rounds to m for every c here, and the parts count alike.  So where several keys are tied O is held
to their hull alone: within the largest |v_j - O| of theirs."""
import math

import pytest
import torch

from oracle import modified, paged
from tests.test_paged_scores import make_tree, words_of
from tests.test_rope import ints, on_gpu, paged_setup
from tests.test_scores import rnd

pytestmark = pytest.mark.gpu

CAPS = [1e-10, 5e-5, 1e-4]
SLOPES = [1e29, 5e30, -1e29, -5e30]  # times 170 keys: below 1e33


@pytest.fixture(scope="module")
def fa():
    import exact_attention_18_gb300 as m
    m.load_library()
    return m


def check(o, lse, rs, v, group, cap, dtype):
    """o [n, H, D], lse [H, n] against the oracle's heads; v [m, H_kv, D]."""
    u, o, lse = torch.finfo(dtype).eps / 2, o.cpu().double(), lse.cpu().double()
    for h, r in enumerate(rs):
        n = r["p"].shape[1]
        terms = r["p"] @ v[:, h // group].double().abs()
        tol = u * r["o"].abs() + (n * 2.0 ** -23 + 4 * cap) * terms + 2.0 ** -25
        tied = r["p"] > 0
        far = ((v[:, h // group].double()[None] - r["o"][:, None]).abs() * tied[:, :, None]).amax(1)
        tol = torch.where((tied.sum(1) > 1)[:, None], tol + far, tol)
        assert bool(((o[:, h] - r["o"]).abs() <= tol).all()), f"O h={h}"
        some = torch.isfinite(r["lse"])
        assert torch.equal(torch.isneginf(lse[h]), ~some), f"L h={h}"
        tol = 2.0 ** -21 * (1 + r["lse"][some].abs()) + 4 * cap
        assert bool(((lse[h][some] - r["lse"][some]).abs() <= tol).all()), f"L h={h}"


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("slope", SLOPES)
@pytest.mark.parametrize("cap", CAPS)
def test_whole_sequences(fa, cap, slope, D):
    """Fixed length and packed, one-sided and two-sided.  A positive slope leaves a row its own key: P is 1 there, so
    dV is dO to the bit, and dQ, dK are what two fp32 sums of dO . V differ by (D 2^-23 of the absolute terms each)."""
    S, H, hk, scale = 170, 4, 2, D ** -0.5
    q, k, v, do = (rnd((1, h, S, D), i, torch.float16) for i, h in enumerate((H, hk, hk, H)))
    q[:, :, ::7] = 0
    slopes = torch.full((H,), slope)
    at = torch.arange(S)
    for causal in (True, False):
        kw = dict(causal=causal, softcap=cap, slopes=slopes.cuda())
        g = [x.cuda() for x in (q, k, v, do)]
        o, lse = fa.forward(*g[:3], **kw)
        rows = [x[0].transpose(0, 1).contiguous() for x in (q, k, v, do)]
        gp, cu = [x.cuda() for x in rows], ints([0, S])
        op, lp = fa.forward_varlen(*gp[:3], cu, S, **kw)
        assert fa.fa_check_device_errors(None) == 0
        rs = modified.sequence(*rows[:3], modified.visible(S, causal), at, at, scale, cap, slopes)
        check(o[0].transpose(0, 1), lse[0], rs, rows[2], H // hk, cap, q.dtype)
        check(op, lp, rs, rows[2], H // hk, cap, q.dtype)
        if slope < 0:
            continue
        dq, dk, dv = (x.cpu() for x in fa.backward_varlen(*gp[:3], op, gp[3], lp, cu, S, **kw))
        assert fa.fa_check_device_errors(None) == 0
        want = rows[3].float().view(S, hk, H // hk, D).sum(2).half()
        assert torch.equal(dv, want)
        va = rows[2].double().abs().repeat_interleave(H // hk, 1)
        off = 2 * scale * D * 2.0 ** -23 * (rows[3].double().abs() * va).sum(-1)  # [S, H]
        assert bool((dq.double().abs() <= off[..., None] * 8 + 2.0 ** -24).all())
        assert bool((dk.double().abs() <= off.view(S, hk, -1).sum(-1)[..., None] * 8 + 2.0 ** -24).all())
        assert float(max(rows[0].abs().max(), rows[1].abs().max())) < 8


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("slope", SLOPES)
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("n", [2, 150])
@pytest.mark.parametrize("tree", [False, True])
def test_over_the_cache(fa, tree, n, cap, slope, D):
    """Few rows and chunks, trees whose rows need not see their own key."""
    kv, H, hk, page = 170, 4, 2, 16
    kc, vc, table, cu = paged_setup([kv], [n], hk, D, page, torch.float16, 5)
    kg, vg = on_gpu(kc, vc)
    q = rnd((n, H, D), 6, torch.float16)
    q[::7] = 0
    slopes = torch.full((H,), slope)
    where = torch.arange(kv)
    pos, seen, extra = where[kv - n:], where[None, :] <= where[kv - n:, None], {}
    if tree:
        bits, depth = make_tree(n, "random", 3)
        pos = (kv - n + depth).clamp(kv - n, kv - 1)
        where = torch.cat((where[:kv - n], pos))
        seen = torch.cat((torch.ones(n, kv - n, dtype=torch.bool), bits), 1)
        extra = dict(tree=words_of(bits, 5).cuda(), positions=pos.to(torch.int32).cuda())
    o, lse = fa.forward_paged(q.cuda(), kg, vg, ints(table), ints([kv]), ints(cu), n, kv, softcap=cap,
                              slopes=slopes.cuda(), **extra)
    assert fa.fa_check_device_errors(None) == 0
    at = paged.slots(table[0], torch.arange(kv), page)
    k, v = kc.reshape(-1, hk, D)[at], vc.reshape(-1, hk, D)[at]
    check(o, lse, modified.sequence(q, k, v, seen, pos, where, 1 / math.sqrt(D), cap, slopes), v, H // hk, cap, q.dtype)
