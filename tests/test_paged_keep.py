"""paged_keep on the GPU, and a cycle of drafting with it: positions, append, tree, keep, next token."""
import math

import pytest
import torch

from oracle import modified, paged
from tests.score_bounds import forward_bounds
from tests.test_paged_scores import make_tree, words_of
from tests.test_rope import DT, ints, on_gpu, paged_setup, rnd
from tests.test_scores import alibi, inside

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_18_gb300 as m
    m.load_library()
    return m


def expected(cache, table, lens, cu, paths):
    out = cache.clone(memory_format=torch.contiguous_format)
    src, dst = cache.reshape(-1, *cache.shape[2:]), out.view(-1, *cache.shape[2:])
    for b, path in enumerate(paths):
        f = lens[b] - (cu[b + 1] - cu[b])
        at = paged.slots(table[b], torch.arange(max(lens[b], 1)), cache.shape[1])
        for i, t in enumerate(path):
            dst[at[f + i]] = src[at[f + t]]
    return out


def keep(fa, kc, vc, table, lens, cu, paths, wide=0, max_q=None):
    cols = max([len(p) for p in paths] + [1]) + wide
    path = torch.full((len(paths), cols), 1 << 30, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    fa.paged_keep(kc, vc, ints(table), ints(lens), ints(cu), max_q or max(b - a for a, b in zip(cu[:-1], cu[1:])),
                  path.cuda(), ints([len(p) for p in paths]))


PATHS = [[0, 2, 3, 7], [0], [], [1, 2], list(range(12)), list(range(0, 38, 2)), [4, 9, 10, 11, 12, 13, 14, 15, 16, 20]]


@pytest.mark.parametrize("D,hk,page,dtype", [(16, 1, 16, "fp16"), (64, 3, 32, "bf16"), (128, 8, 16, "bf16"),
                                             (32, 2, 256, "fp16")])
@pytest.mark.parametrize("hnd", [False, True])
def test_moves(fa, D, hk, page, dtype, hnd):
    """Sources that are slots of earlier ones, tokens that stay, pages that end between, nothing to keep; values
    that no arithmetic may touch."""
    q_lens = [8, 5, 4, 3, 12, 40, 21]
    lens = [8, 21, 4, 19, 60, 300, 37]
    kc, vc, table, cu = paged_setup(lens, q_lens, hk, D, page, DT[dtype], 9, hnd=hnd)
    kc[:, 0, 0, 0], vc[:, 1, 0, 1] = float("nan"), -0.0
    want = [expected(x, table, lens, cu, PATHS) for x in (kc, vc)]
    kg, vg = on_gpu(kc, vc)
    keep(fa, kg, vg, table, lens, cu, PATHS, wide=3, max_q=100)
    assert fa.fa_check_device_errors(None) == 0, fa.fa_last_error_detail()
    for got, w in zip((kg, vg), want):
        assert torch.equal(got.cpu().view(torch.int16) if got.is_contiguous() else got.cpu().contiguous().view(torch.int16),
                           w.contiguous().view(torch.int16))


def test_offsets_past_32_bits(fa):
    """Pages more than 2^32 bytes apart."""
    page, hk, D = 16, 1, 16
    gap = 1 << 31  # elements
    pool = torch.empty(2 * gap + page * hk * D, dtype=torch.float16, device="cuda")
    kc = pool.as_strided((3, page, hk, D), (gap, hk * D, D, 1))
    vpool = torch.empty_like(pool)
    vc = vpool.as_strided(kc.shape, kc.stride())
    table, lens, cu = torch.tensor([[1, 2]], dtype=torch.int32), [32], [0, 20]
    for x, s in ((kc, 1), (vc, 2)):
        x.copy_(rnd(kc.shape, s, torch.float16))
    want = [expected(x.cpu(), table, lens, cu, [[0, 5, 18]]) for x in (kc, vc)]
    keep(fa, kc, vc, table, lens, cu, [[0, 5, 18]])
    assert fa.fa_check_device_errors(None) == 0
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])


@pytest.mark.parametrize("bad", ["order", "twice", "range", "negative", "long", "wide", "kv", "max", "table"])
def test_bad_paths_are_left_alone(fa, bad):
    """What contradicts the call is reported, and its sequence keeps its rows; the other one moves."""
    lens, q_lens, hk, D, page = [40, 50], [10, 10], 2, 64, 16
    kc, vc, table, cu = paged_setup(lens, q_lens, hk, D, page, torch.float16, 4)
    kg, vg = on_gpu(kc, vc)
    path = {"order": [0, 3, 2], "twice": [0, 3, 3], "range": [0, 4, 10], "negative": [-1, 4, 5]}.get(bad, [0, 4, 5])
    path = torch.tensor([path, [0, 4, 5]], dtype=torch.int32)
    n, lens_g, max_q = [3, 3], list(lens), 10
    if bad == "long":
        n[0] = 11
        path = torch.arange(12, dtype=torch.int32).repeat(2, 1)
    if bad == "wide":
        n[0] = 4
    if bad == "kv":
        lens_g[0] = 9
    if bad == "max":
        cu, max_q = [0, 10, 16], 9
    if bad == "table":
        table = table.clone()
        table[0, 1:3] = 1 << 20
    want = expected(kc, table, lens, cu, [[], [0, 4, 5] if bad != "long" else [0, 1, 2]])
    fa.paged_keep(kg, vg, ints(table), ints(lens_g), ints(cu), max_q, path.cuda(), ints(n))
    assert fa.fa_check_device_errors(None) == 1
    assert torch.equal(kg.cpu(), want)
    assert fa.fa_check_device_errors(None) == 0


def test_arguments_are_checked(fa):
    kc, vc, table, cu = paged_setup([40], [10], 2, 64, 16, torch.float16, 4)
    kc, vc = on_gpu(kc, vc)
    good = [kc, vc, ints(table), ints([40]), ints(cu), 10, torch.zeros(1, 3, dtype=torch.int32, device="cuda"), ints([1])]
    fa.paged_keep(*good)
    for i, x in ((6, good[6].long()), (6, good[6][0]), (6, torch.zeros(2, 3, dtype=torch.int32, device="cuda")),
                 (7, ints([1, 1])), (7, good[7].long()), (1, vc[..., :32]), (6, good[6].cpu())):
        bad = list(good)
        bad[i] = x
        with pytest.raises(ValueError):
            fa.paged_keep(*bad)
    with pytest.raises(fa.FAError):
        fa.paged_keep(*good[:5], -1, *good[6:])
    fa.paged_keep(*good[:6], torch.zeros(1, 0, dtype=torch.int32, device="cuda"), ints([0]))  # nothing to keep


@pytest.mark.parametrize("D,H,hk,dtype", [(64, 4, 2, "fp16"), (128, 16, 2, "bf16")])
def test_a_cycle_of_drafting(fa, D, H, hk, dtype):
    """Trees of drafted tokens are rotated by their depths and appended, attended to, an accepted path is kept, and
    the next token attends to what was kept: as if only the path had ever been appended."""
    dt, page = DT[dtype], 16
    ctx, n = [37, 100], [13, 30]
    lens = [c + m for c, m in zip(ctx, n)]
    kc, vc, table, cu = paged_setup(lens, n, hk, D, page, dt, 11)
    T = cu[-1]
    x = rnd((T, H + 2 * hk, D), 12, torch.float32).to(dt).cuda()
    q, k, v = x[:, :H], x[:, H:H + hk], x[:, H + hk:]
    trees = [make_tree(m, "tree", 0) for m in n]
    rows = torch.cat([words_of(b, 1) for b, _ in trees]).cuda()
    pos = torch.cat([c + d for c, (_, d) in zip(ctx, trees)]).to(torch.int32).cuda()
    steps = fa.rope_steps(fa.rope_inv_freq(D)[0])
    kg, vg = on_gpu(kc, vc)
    kv, cug, tab = ints(lens), ints(cu), ints(table)
    slopes = alibi(H).cuda()
    q_rot = fa.paged_append(k, v, kg, vg, tab, kv, cug, max(n), q=q, positions=pos, steps=steps)
    o, lse = fa.forward_paged(q_rot, kg, vg, tab, kv, cug, max(n), max(lens), softcap=20.0, slopes=slopes, tree=rows,
                              positions=pos)
    paths = [[0, 3, 10], [0, 2, 8, 26]]
    path = torch.tensor([p + [0] * (4 - len(p)) for p in paths], dtype=torch.int32, device="cuda")
    m = ints([len(p) for p in paths])
    fa.paged_keep(kg, vg, tab, kv, cug, max(n), path, m)
    kv2 = kv - ints(n) + m + 1  # and one token more
    x2 = rnd((2, H + 2 * hk, D), 13, torch.float32).to(dt).cuda()
    one = ints([0, 1, 2])
    q2 = fa.paged_append(x2[:, H:H + hk], x2[:, H + hk:], kg, vg, tab, kv2, one, 1, q=x2[:, :H], steps=steps)
    o2, lse2 = fa.forward_paged(q2, kg, vg, tab, kv2, one, 1, max(lens), softcap=20.0, slopes=slopes)
    assert fa.fa_check_device_errors(None) == 0, fa.fa_last_error_detail()
    # the same with only the path appended, token by token as a chunk
    k3, v3 = on_gpu(kc, vc)
    sel = torch.tensor([cu[b] + t for b, p in enumerate(paths) for t in p], device="cuda")
    cu3 = ints([0, len(paths[0]), len(paths[0]) + len(paths[1])])
    kv3 = kv - ints(n) + m
    q3 = fa.paged_append(k[sel], v[sel], k3, v3, tab, kv3, cu3, 4, q=q[sel], steps=steps)
    assert torch.equal(q3, q_rot[sel])
    o3, lse3 = fa.forward_paged(q3, k3, v3, tab, kv3, cu3, 4, max(lens), softcap=20.0, slopes=slopes)
    q4 = fa.paged_append(x2[:, H:H + hk], x2[:, H + hk:], k3, v3, tab, kv2, one, 1, q=x2[:, :H], steps=steps)
    o4, lse4 = fa.forward_paged(q4, k3, v3, tab, kv2, one, 1, max(lens), softcap=20.0, slopes=slopes)
    assert torch.equal(o2, o4) and torch.equal(lse2, lse4)
    # the tree's rows of the path see what the chunk's rows see; other keys lie between, so blocks and sums differ
    for b, (t0, c) in enumerate(zip(cu[:-1], ctx)):
        at = paged.slots(table[b], torch.arange(c + len(paths[b])), page)
        kk, vv = (y.cpu().reshape(-1, hk, D)[at] for y in (k3, v3))
        i = torch.arange(c, c + len(paths[b]))
        j = torch.arange(c + len(paths[b]))
        base = 0 if b == 0 else len(paths[0])
        qq = q3[base:base + len(i)].cpu()
        rs = modified.sequence(qq, kk, vv, j[None, :] <= i[:, None], i, j, 1 / math.sqrt(D), 20.0, alibi(H))
        for h, r in enumerate(rs):
            g = h // (H // hk)
            tol_o, tol_l, _ = forward_bounds(r, qq[:, h], kk[:, g], vv[:, g], 1 / math.sqrt(D), 20.0, dt)
            tree_rows = [t0 + t for t in paths[b]]
            inside(o[tree_rows, h], r["o"], tol_o, f"tree O b={b} h={h}")
            inside(lse[h, tree_rows], r["lse"], tol_l, f"tree L b={b} h={h}")
            inside(o3[base:base + len(i), h], r["o"], tol_o, f"chunk O b={b} h={h}")


def test_graph(fa):
    """Captured and replayed with other paths in the same tensors."""
    lens, q_lens, hk, D, page = [40, 50], [10, 10], 2, 64, 16
    kc, vc, table, cu = paged_setup(lens, q_lens, hk, D, page, torch.float16, 4)
    kg, vg = on_gpu(kc, vc)
    path, n = torch.tensor([[0, 4, 5], [0, 1, 2]], dtype=torch.int32, device="cuda"), ints([3, 3])
    args = (kg, vg, ints(table), ints(lens), ints(cu), 10, path, n)
    fa.paged_keep(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.paged_keep(*args)
    for paths in ([[0, 4, 5], [2, 3, 9]], [[1, 2, 3], [0]]):
        kg.copy_(kc), vg.copy_(vc)
        path.zero_()
        for b, p in enumerate(paths):
            path[b, :len(p)] = torch.tensor(p, dtype=torch.int32, device="cuda")
        n.copy_(ints([len(p) for p in paths]))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kg.cpu(), expected(kc, table, lens, cu, paths))
        assert torch.equal(vg.cpu(), expected(vc, table, lens, cu, paths))
