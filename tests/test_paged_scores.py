"""Modified scores and drafted trees over a paged cache on the GPU, against the fp64 oracle (bounds in
score_bounds.py; a unit that several CTAs share joins fp32 partials, which the bounds' 2^-24 a key covers)."""
import math

import pytest
import torch

from oracle import modified, paged
from tests.score_bounds import forward_bounds
from tests.test_paged import poison
from tests.test_rope import DT, ints, on_gpu, paged_setup, rnd
from tests.test_scores import alibi, inside

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_18_gb300 as m
    m.load_library()
    return m


MODS = {"cap": dict(softcap=5.0, gain=4.0), "bias": dict(bias=True), "both": dict(softcap=30.0, bias=True, gain=8.0)}


def make_tree(n, kind, seed):
    """(bits [n, n], depth [n]) of n drafted tokens."""
    g = torch.Generator().manual_seed(seed)
    bits, depth = torch.zeros(n, n, dtype=torch.bool), torch.zeros(n, dtype=torch.int64)
    if kind == "random":  # any bits, rows without one among them; depths anywhere, beyond the ends too
        bits = torch.rand(n, n, generator=g) < 0.3
        bits[torch.rand(n, generator=g) < 0.2] = False
        return bits, torch.randint(-3, n + 3, (n,), generator=g)
    for i in range(n):
        if kind == "chain":
            p = i - 1
        else:
            p = (i - 1) // 3 if i else -1
        if p >= 0:
            bits[i], depth[i] = bits[p], depth[p] + 1
        bits[i, i] = True
    return bits, depth


def words_of(bits, words):
    """int32 rows of a bool matrix."""
    full = torch.zeros(bits.shape[0], 32 * words, dtype=torch.int64)
    full[:, :bits.shape[1]] = bits
    x = (full.view(-1, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(x >= 2 ** 31, x - 2 ** 32, x).to(torch.int32)


def case(fa, lens, q_lens, H, hk, D, page, dtype, softcap=None, bias=False, gain=1.0, causal=True, window=None,
         tree=None, junk=True, max_q=None, max_k=None, slack=0, seed=0, **kw):
    dt = DT[dtype]
    kc, vc, table, cu = paged_setup(lens, q_lens, hk, D, page, dt, sum(lens) + seed)
    std = math.sqrt(gain)
    kc = (kc.float() * std).to(dt)
    T = cu[-1]
    q = rnd((T, H, D), sum(lens) + 1, torch.float32).mul(std).to(dt)
    slopes = alibi(H) if bias else None
    clean = (kc, vc, table)
    if junk:
        reach = window if tree is None or window is None else (window[0], 0)
        kc, vc, table = poison(kc, vc, table, lens, cu, reach)
    args = {}
    trees = []
    if tree is not None:
        words = -(-max(q_lens) // 32) + slack
        rows, pos = torch.full((T, words), -1, dtype=torch.int32), torch.zeros(T, dtype=torch.int32)
        for b, n in enumerate(q_lens):
            bits, depth = make_tree(n, tree, seed + b)
            trees.append((bits, depth))
            pad = torch.ones(n, 32 * words, dtype=torch.bool)  # bits past the new tokens are not used
            pad[:, :n] = bits
            rows[cu[b]:cu[b + 1]] = words_of(pad, words)
            pos[cu[b]:cu[b + 1]] = (lens[b] - n + depth).to(torch.int32)
        args = dict(tree=rows.cuda(), positions=pos.cuda())
    kcg, vcg = on_gpu(kc, vc)
    o, lse = fa.forward_paged(q.cuda(), kcg, vcg, ints(table), ints(lens), ints(cu), max_q or max(q_lens + [1]),
                              max_k or max(lens), causal=causal, window=window, softcap=softcap,
                              slopes=None if slopes is None else slopes.cuda(), **args, **kw)
    assert fa.fa_check_device_errors(None) == 0, fa.fa_last_error_detail()
    kc, vc, table = clean
    oc, lc = o.cpu(), lse.cpu()
    left, right = (-1, -1) if window is None else window
    for b, (t0, t1) in enumerate(zip(cu[:-1], cu[1:])):
        n, kv = t1 - t0, lens[b]
        if n == 0:
            continue
        at = paged.slots(table[b], torch.arange(kv), page)
        k, v = kc.reshape(-1, hk, D)[at], vc.reshape(-1, hk, D)[at]
        pos, where = torch.arange(kv - n, kv), torch.arange(kv)
        seen = torch.ones(n, kv, dtype=torch.bool)
        if tree is not None:
            bits, depth = trees[b]
            pos = (kv - n + depth).clamp(kv - n, kv - 1)
            where = torch.cat((where[:kv - n], pos))
        if left >= 0:
            seen &= where[None, :] >= pos[:, None] - left
        if tree is not None:
            seen[:, kv - n:] = bits
        elif causal or right >= 0:
            seen &= where[None, :] <= pos[:, None] + (0 if causal else right)
        rs = modified.sequence(q[t0:t1], k, v, seen, pos, where, 1 / math.sqrt(D), softcap, slopes)
        for h, r in enumerate(rs):
            g = h // (H // hk)
            tol_o, tol_l, _ = forward_bounds(r, q[t0:t1, h], k[:, g], v[:, g], 1 / math.sqrt(D), softcap, dt)
            inside(oc[t0:t1, h], r["o"], tol_o, f"O b={b} h={h}")
            got, some = lc[h, t0:t1].double(), torch.isfinite(r["lse"])
            assert torch.equal(torch.isneginf(got), ~some), f"L b={b} h={h}: rows that see no key"
            inside(got[some], r["lse"][some], tol_l[some], f"L b={b} h={h}")
            assert bool((oc[t0:t1, h][~some] == 0).all())
    return o, lse


@pytest.mark.parametrize("mods", MODS)
@pytest.mark.parametrize("D,page,dtype", [(16, 16, "fp16"), (32, 64, "bf16"), (64, 16, "fp16"), (128, 64, "bf16")])
@pytest.mark.parametrize("H,hk", [(4, 4), (8, 2), (9, 3)])
def test_decoding(fa, D, page, dtype, H, hk, mods):
    case(fa, [1, 17, 300, 128, 1029], [1] * 5, H, hk, D, page, dtype, **MODS[mods])


@pytest.mark.parametrize("mods", MODS)
@pytest.mark.parametrize("D,G", [(64, 4), (64, 16), (128, 8), (32, 8)])
@pytest.mark.parametrize("window", [None, (100, 0), (3, 0)])
def test_drafted(fa, D, G, mods, window):
    """A few new tokens a sequence: 16, 32 and 64 rows of the few-row kernel."""
    case(fa, [5, 270, 513, 1500], [4, 1, 3, 2], 2 * G, 2, D, 16, "fp16", window=window, **MODS[mods])


@pytest.mark.parametrize("mods", MODS)
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("causal,window", [(True, None), (True, (70, 0)), (False, None), (False, (50, 31))])
def test_chunks(fa, D, mods, causal, window):
    """The tile kernel, one to four tiles a unit."""
    case(fa, [130, 700, 333], [130, 200, 65], 4, 2, D, 32, "bf16", causal=causal, window=window, **MODS[mods])


@pytest.mark.parametrize("D", [64, 128])
def test_mixed(fa, D):
    """Both kernels in one call, bounds loose."""
    case(fa, [600, 33, 1100, 90, 5], [200, 1, 300, 0, 2], 8, 2, D, 16, "fp16", softcap=9.0, bias=True, gain=3.0,
         max_q=900, max_k=5000)


TREES = [([17], [13]), ([64, 300, 90], [64, 5, 33]), ([7, 200], [7, 100]), ([1, 150, 1000], [1, 31, 65]),
         ([420, 130], [129, 128])]


@pytest.mark.parametrize("kind", ["tree", "random", "chain"])
@pytest.mark.parametrize("lens,q_lens", TREES, ids=lambda x: "-".join(map(str, x)))
@pytest.mark.parametrize("D,H,hk", [(64, 4, 2), (128, 8, 1), (16, 2, 2)])
def test_trees(fa, D, H, hk, lens, q_lens, kind):
    case(fa, lens, q_lens, H, hk, D, 16, "fp16", tree=kind, seed=3)


@pytest.mark.parametrize("kind", ["tree", "random"])
@pytest.mark.parametrize("mods", MODS)
@pytest.mark.parametrize("window", [None, (40, 0), (0, 0), (300, -1)])
@pytest.mark.parametrize("D,H,hk", [(64, 4, 4), (64, 16, 2), (128, 8, 2), (32, 4, 1)])
def test_tree_scores(fa, D, H, hk, window, mods, kind):
    """Distances and windows by the tokens' positions."""
    case(fa, [40, 333, 129], [20, 45, 2], H, hk, D, 16, "bf16", tree=kind, window=window, slack=1, **MODS[mods])


def test_tree_mixed_kernels(fa):
    """Short and long trees in one call, and a sequence without new tokens."""
    case(fa, [500, 90, 700, 64], [100, 3, 0, 8], 16, 2, 128, 64, "bf16", tree="tree", softcap=20.0, bias=True)


@pytest.mark.parametrize("D,n", [(64, 6), (64, 150), (128, 150)])
def test_chain_is_causal(fa, D, n):
    """A chain of drafted tokens is a causal chunk, to the bit."""
    a = case(fa, [400, n], [n, n], 4, 2, D, 32, "fp16", tree="chain", softcap=10.0, bias=True)
    b = case(fa, [400, n], [n, n], 4, 2, D, 32, "fp16", softcap=10.0, bias=True)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_long_cache_split_over_ctas(fa):
    case(fa, [9000, 4097], [1, 3], 8, 1, 64, 128, "fp16", softcap=8.0, bias=True, gain=3.0)
    case(fa, [5000], [40], 8, 1, 128, 128, "bf16", tree="tree", softcap=8.0, gain=3.0)


def test_graph_and_streams(fa):
    """A captured tree call beside eager ones, replayed with changed contents."""
    lens, q_lens, H, hk, D = [300, 90], [12, 40], 8, 2, 64
    kc, vc, table, cu = paged_setup(lens, q_lens, hk, D, 16, torch.float16, 5)
    q = rnd((cu[-1], H, D), 6, torch.float16).cuda()
    kc, vc = on_gpu(kc, vc)
    rows, pos = [], []
    for b, n in enumerate(q_lens):
        bits, depth = make_tree(n, "tree", b)
        rows.append(words_of(bits, 2))
        pos.append((lens[b] - n + depth).to(torch.int32))
    kw = dict(tree=torch.cat(rows).cuda(), positions=torch.cat(pos).cuda(), softcap=12.0, slopes=alibi(H).cuda())
    args = (kc, vc, ints(table), ints(lens), ints(cu), 40, 300)
    want = fa.forward_paged(q, *args, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    qg = q.clone()
    with torch.cuda.graph(graph):
        got = fa.forward_paged(qg, *args, **kw)
    side = torch.cuda.Stream()
    for i in range(3):
        qg.copy_(q * (1 if i != 1 else 0))
        torch.cuda.synchronize()
        graph.replay()
        other = fa.forward_paged(q, *args, stream=side, **kw)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, other))
        assert all(torch.equal(x, y) for x, y in zip(want, got)) == (i != 1)


def test_arguments_are_checked(fa):
    lens, q_lens, H, hk, D = [50], [8], 4, 2, 64
    kc, vc, table, cu = paged_setup(lens, q_lens, hk, D, 16, torch.float16, 5)
    q = rnd((8, H, D), 6, torch.float16).cuda()
    kc, vc = on_gpu(kc, vc)
    args = (q, kc, vc, ints(table), ints(lens), ints(cu), 8, 50)
    tree, pos = torch.ones(8, 1, dtype=torch.int32, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    for kw in (dict(softcap=0.0), dict(softcap=-2.0), dict(slopes=torch.ones(3, device="cuda")),
               dict(slopes=torch.ones(4)), dict(slopes=torch.ones(4, device="cuda").half()), dict(tree=tree),
               dict(positions=pos), dict(tree=tree, positions=pos[:7]), dict(tree=tree[:7], positions=pos),
               dict(tree=tree.long(), positions=pos), dict(tree=tree, positions=pos.long()),
               dict(tree=tree, positions=pos, causal=False), dict(tree=tree, positions=pos, window=(4, 2)),
               dict(tree=tree.cpu(), positions=pos), dict(tree=tree.expand(8, 3)[:, ::2], positions=pos)):
        with pytest.raises(ValueError):
            fa.forward_paged(*args, **kw)
    with pytest.raises(fa.FAError):
        fa.forward_paged(*args, softcap=math.inf)
    wide = (q, kc, vc, ints(table), ints(lens), ints(cu), 8, 50)
    with pytest.raises(fa.FAError):  # rows without words
        fa.forward_paged(*wide, tree=torch.ones(8, 0, dtype=torch.int32, device="cuda"), positions=pos)
    with pytest.raises(TypeError):
        fa.forward_paged(*args, slopes=[1.0] * 4)
