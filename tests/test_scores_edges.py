"""Modified scores, trees and paged_keep where a call can go wrong beside its numbers: waits that run out, calls at
once on two streams and threads, absent parts of the raw calls, values behind masks, neighbours full of NaN, lengths
at the ends of their ranges, wide groups, sliced arguments, empty calls.  Bounds in score_bounds.py."""
import ctypes
import threading

import pytest
import torch

from oracle import modified, paged
from tests.score_bounds import forward_bounds
from tests.test_paged_scores import case, make_tree, words_of
from tests.test_rope import ints, on_gpu, paged_setup
from tests.test_scores import alibi, check_sequence, fixed_case, inside, rnd

pytestmark = pytest.mark.gpu

FA_ERR_TIMEOUT = 6


@pytest.fixture(scope="module")
def fa():
    import exact_attention_18_gb300 as m
    m.load_library()
    return m


def stream_ptr():
    return torch.cuda.current_stream().cuda_stream


class ShortLimit:
    def __init__(self, fa):
        self.fa = fa

    def __enter__(self):
        assert self.fa.fa_check_device_errors(None) == 0
        self.fa.fa_set_wait_limit_ns(1)
        return self

    def __exit__(self, *exc):
        self.status = self.fa.fa_check_device_errors(None)
        self.fa.fa_set_wait_limit_ns(0)


@pytest.mark.parametrize("D", [64, 128])
def test_waits_that_run_out(fa, D):
    """Pipeline waits with a limit of a nanosecond: the calls return, report it, and the next ones are right."""
    q, k, v, do = (rnd((2, 4, 1500, D), i, torch.float16).cuda() for i in range(4))
    kw = dict(causal=True, softcap=20.0, slopes=alibi(4).cuda())
    o, lse = fa.forward(q, k, v, **kw)
    grads = fa.backward(q, k, v, o, do, lse, **kw)
    with ShortLimit(fa) as a:
        fa.forward(q, k, v, **kw)
    with ShortLimit(fa) as b:
        fa.backward(q, k, v, o, do, lse, **kw)
    lens, n = [1600, 300], [200, 40]
    kc, vc, table, cu = paged_setup(lens, n, 2, D, 16, torch.float16, 5)
    kc, vc = on_gpu(kc, vc)
    qp = rnd((cu[-1], 4, D), 6, torch.float16).cuda()
    rows = torch.cat([words_of(make_tree(m, "tree", 0)[0], 7) for m in n]).cuda()
    pos = torch.cat([L - m + make_tree(m, "tree", 0)[1] for L, m in zip(lens, n)]).to(torch.int32).cuda()
    args = (kc, vc, ints(table), ints(lens), ints(cu), 200, 1600)
    want = fa.forward_paged(qp, *args, tree=rows, positions=pos, softcap=9.0)
    few = (qp[:2], kc, vc, ints(table), ints(lens), ints([0, 1, 2]), 1, 1600)
    one = fa.forward_paged(*few, softcap=9.0)
    with ShortLimit(fa) as c:
        fa.forward_paged(qp, *args, tree=rows, positions=pos, softcap=9.0)
    with ShortLimit(fa) as d:
        fa.forward_paged(*few, softcap=9.0)
    cu3 = ints([0, 70, 1333, 1500])
    pk = [x[0].transpose(0, 1).contiguous() for x in (q, k, v, do)]
    op, lp = fa.forward_varlen(*pk[:3], cu3, 1400, **kw)
    gp = fa.backward_varlen(*pk[:3], op, pk[3], lp, cu3, 1400, **kw)
    with ShortLimit(fa) as e:
        fa.forward_varlen(*pk[:3], cu3, 1400, **kw)
    with ShortLimit(fa) as f:
        fa.backward_varlen(*pk[:3], op, pk[3], lp, cu3, 1400, **kw)
    assert [x.status for x in (a, b, c, d, e, f)] == [FA_ERR_TIMEOUT] * 6
    again = (*fa.forward(q, k, v, **kw), *fa.backward(q, k, v, o, do, lse, **kw),
             *fa.forward_paged(qp, *args, tree=rows, positions=pos, softcap=9.0), *fa.forward_paged(*few, softcap=9.0),
             *fa.forward_varlen(*pk[:3], cu3, 1400, **kw),
             *fa.backward_varlen(*pk[:3], op, pk[3], lp, cu3, 1400, **kw))
    assert fa.fa_check_device_errors(None) == 0
    for x, y in zip(again, (o, lse, *grads, *want, *one, op, lp, *gp)):
        assert torch.equal(x, y)


def test_threads_and_streams_at_once(fa):
    """Two threads, a stream each, calls of every kind: the bits of the calls made alone."""
    lens, n, H, hk, D = [700, 90], [60, 3], 4, 2, 64
    kc, vc, table, cu = paged_setup(lens, n, hk, D, 16, torch.bfloat16, 5)
    kc, vc = on_gpu(kc, vc)
    qp = rnd((cu[-1], H, D), 6, torch.bfloat16).cuda()
    q, k, v, do = (rnd((1, H, 900, D), i, torch.bfloat16).cuda() for i in range(4))
    slopes = alibi(H).cuda()
    rows = torch.cat([words_of(make_tree(m, "tree", 0)[0], 2) for m in n]).cuda()
    pos = torch.cat([L - m + make_tree(m, "tree", 0)[1] for L, m in zip(lens, n)]).to(torch.int32).cuda()
    args = (qp, kc, vc, ints(table), ints(lens), ints(cu), 60, 700)

    def everything(cap, stream=None):
        o, lse = fa.forward(q, k, v, causal=True, softcap=cap, slopes=slopes, stream=stream)
        g = fa.backward(q, k, v, o, do, lse, causal=True, softcap=cap, slopes=slopes, stream=stream)
        t = fa.forward_paged(*args, softcap=cap, tree=rows, positions=pos, stream=stream)
        return (o, lse, *g, *t)

    want = [everything(c) for c in (5.0, 40.0)]
    torch.cuda.synchronize()
    got, streams = [[], []], [torch.cuda.Stream() for _ in range(2)]

    def work(i):
        for _ in range(5):
            got[i].append(everything((5.0, 40.0)[i], streams[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert fa.fa_check_device_errors(None) == 0
    for i in range(2):
        assert len(got[i]) == 5
        for res in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(res, want[i]))


def test_raw_calls_without_scores(fa):
    """scores == NULL, forward and backward, fixed and packed: the plain calls' bits where those run the same
    kernels, and their values where not; a tree without scores."""
    B, H, S, D = 1, 2, 200, 64
    q, k, v, do = (rnd((B, H, S, D), i, torch.float16).cuda() for i in range(4))
    o, lse = fa.forward(q, k, v, causal=True)
    grads = fa.backward(q, k, v, o, do, lse, causal=True)
    o2, lse2, *g2 = (torch.empty_like(x) for x in (o, lse, *grads))
    ws = torch.empty(1 << 27, dtype=torch.uint8, device="cuda")
    assert fa.fa_fwd_scores(q.data_ptr(), k.data_ptr(), v.data_ptr(), o2.data_ptr(), lse2.data_ptr(), B, H, H, S, D,
                            True, -1, -1, None, 0.125, fa.FA_FP16, stream_ptr()) == 0
    assert fa.fa_bwd_scores(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
                            *(x.data_ptr() for x in g2), B, H, H, S, D, True, -1, -1, None, 0.125, fa.FA_FP16,
                            ws.data_ptr(), ws.nbytes, stream_ptr()) == 0
    for a, b in zip((o, lse, *grads), (o2, lse2, *g2)):
        assert torch.equal(a, b)
    T = S
    cu = ints([0, 80, T])
    qp, kp, vp, dop = (x[0].transpose(0, 1).contiguous() for x in (q, k, v, do))
    o3, lse3 = torch.empty_like(qp), torch.empty(H, T, device="cuda")
    g3 = [torch.empty_like(qp) for _ in range(3)]
    assert fa.fa_fwd_scores_varlen(qp.data_ptr(), kp.data_ptr(), vp.data_ptr(), o3.data_ptr(), lse3.data_ptr(),
                                   cu.data_ptr(), 2, 120, T, H, H, D, True, -1, -1, None, 0.125, fa.FA_FP16,
                                   stream_ptr()) == 0
    assert fa.fa_bwd_scores_varlen(qp.data_ptr(), kp.data_ptr(), vp.data_ptr(), o3.data_ptr(), dop.data_ptr(),
                                   lse3.data_ptr(), *(x.data_ptr() for x in g3), cu.data_ptr(), 2, 120, T, H, H, D,
                                   True, -1, -1, None, 0.125, fa.FA_FP16, ws.data_ptr(), ws.nbytes, stream_ptr()) == 0
    torch.cuda.synchronize()
    assert fa.fa_check_device_errors(None) == 0
    for a, e in ((0, 80), (80, T)):
        check_sequence(*(x[a:e].cpu() for x in (qp, kp, vp, dop, o3)), lse3[:, a:e].cpu(), [x[a:e].cpu() for x in g3],
                       True, None, 0, None, None, 0.125)
    lens, n, page = [50, 400], [20, 140], 16
    for D in (64, 128):
        kc, vc, table, cu = paged_setup(lens, n, 2, D, page, torch.float16, 5)
        kc, vc = on_gpu(kc, vc)
        q = rnd((cu[-1], 4, D), 6, torch.float16).cuda()
        rows = torch.cat([words_of(make_tree(m, "tree", 0)[0], 5) for m in n]).cuda()
        pos = torch.cat([L - m + make_tree(m, "tree", 0)[1] for L, m in zip(lens, n)]).to(torch.int32).cuda()
        tab, kv, cug = ints(table), ints(lens), ints(cu)
        want = fa.forward_paged(q, kc, vc, tab, kv, cug, 140, 400, tree=rows, positions=pos)
        o, lse = torch.empty_like(q), torch.empty(4, cu[-1], device="cuda")
        cache = fa.PagedCache(kc.data_ptr(), vc.data_ptr(), tab.data_ptr(), kv.data_ptr(), tab.shape[1], 0, kc.shape[0],
                              page, kc.stride(0), kc.stride(1), kc.stride(2))
        assert fa.fa_fwd_paged_tree(q.data_ptr(), o.data_ptr(), lse.data_ptr(), ctypes.byref(cache), cug.data_ptr(),
                                    pos.data_ptr(), rows.data_ptr(), 5, 5, 2, 140, 400, cu[-1], 4, 2, D, -1, None,
                                    D ** -0.5, fa.FA_FP16, ws.data_ptr(), ws.nbytes, stream_ptr()) == 0
        assert fa.fa_check_device_errors(None) == 0
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf"), 6e4])
@pytest.mark.parametrize("D", [64, 128])
def test_values_behind_the_mask(fa, D, junk):
    """Keys that no row sees: their K may hold anything, and rows of blocks that hold them keep their bits."""
    S, t = 300, 201
    q, k, v, do = (rnd((1, 2, S, D), i, torch.float16).cuda() for i in range(4))
    for mods in (dict(softcap=9.0), dict(slopes=alibi(2).cuda()), dict(softcap=9.0, slopes=alibi(2).cuda())):
        o, lse = fa.forward(q, k, v, causal=True, **mods)
        k2 = k.clone()
        k2[:, :, t:] = junk
        o2, lse2 = fa.forward(q, k2, v, causal=True, **mods)
        assert torch.equal(o[:, :, :t], o2[:, :, :t]) and torch.equal(lse[:, :, :t], lse2[:, :, :t])


@pytest.mark.parametrize("D", [16, 64, 128])
def test_a_sample_of_nan_between_others(fa, D):
    """Documents beside one that holds nothing but NaN keep their bits, forward and backward."""
    lens, H, hk = [70, 133, 200, 1, 64], 4, 2
    cu = [0, 70, 203, 403, 404, 468]
    q, k, v, do = (rnd((cu[-1], h, D), i, torch.bfloat16).cuda() for i, h in enumerate((H, hk, hk, H)))
    kw = dict(causal=True, softcap=8.0, slopes=alibi(H).cuda(), prefix=ints([3, 100, 50, 1, 0]))

    def run():
        o, lse = fa.forward_varlen(q, k, v, ints(cu), 200, **kw)
        return o, lse, fa.backward_varlen(q, k, v, o, do, lse, ints(cu), 200, **kw)

    o, lse, grads = run()
    for x in (q, k, v, do):
        x[70:203] = float("nan")
    o2, lse2, grads2 = run()
    assert fa.fa_check_device_errors(None) == 0
    keep = torch.cat((torch.arange(70), torch.arange(203, cu[-1]))).cuda()
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[:, keep], lse2[:, keep])
    for a, b in zip(grads, grads2):
        assert torch.equal(a[keep], b[keep])
        assert not bool(a.isnan().any())


@pytest.mark.parametrize("D", [64, 128])
def test_ends_of_ranges(fa, D):
    """Prefix lengths and window sides at the ends of their types, a slope whose bias leaves nothing but the nearest
    keys, and a scale below any sensible one."""
    q, k, v = (rnd((3, 2, 190, D), i, torch.float16).cuda() for i in range(3))
    pfx = ints([2 ** 31 - 1, -2 ** 31, 77])
    a = fa.forward(q, k, v, causal=True, softcap=9.0, prefix=pfx)
    b = fa.forward(q, k, v, causal=True, softcap=9.0, prefix=ints([190, 0, 77]))
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    c = fa.forward(q, k, v, causal=True, softcap=9.0, prefix=pfx, window=(2 ** 40, 2 ** 40))
    d = fa.forward(q, k, v, causal=True, softcap=9.0, prefix=pfx, window=(-5, -(2 ** 40)))
    assert all(torch.equal(x, y) for x, y in zip(a, c)) and all(torch.equal(x, y) for x, y in zip(a, d))
    e = fa.forward(q, k, v, causal=True, slopes=torch.full((2,), 1e30, device="cuda"))
    assert torch.equal(e[0], v)
    fixed_case(fa, 1, 2, 1, 150, D, "fp16", scale=1e-9, bias=True)
    fixed_case(fa, 1, 2, 1, 150, D, "bf16", scale=-1e-3, bias=True, causal=False)


@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("scale", [None, 0.0, -0.2])
def test_prefix_alone(fa, D, scale):
    """Plain scores under a prefix, forward and backward; scales that no unit can be made of."""
    fixed_case(fa, 2, 4, 2, 300, D, "fp16", prefix=170, scale=scale)
    fixed_case(fa, 1, 2, 1, 200, D, "bf16", prefix=65, window=(50, 0), scale=scale)


def test_long_rows(fa):
    """More keys than a tile's CTA holds at once, and distances past 2^13."""
    fixed_case(fa, 1, 2, 1, 8300, 64, "fp16", bias=True, softcap=30.0, window=(8200, 0), backward=False)
    fixed_case(fa, 1, 1, 1, 4200, 128, "bf16", bias=True, causal=False, gain=2.0)


@pytest.mark.parametrize("D,H", [(128, 64), (64, 128)])
def test_offsets_past_2_31_elements(fa, D, H):
    """A packed batch of more than 2^31 elements a tensor: its last document, forward and backward, has the bits that
    it has alone, and so has a head of a document before it."""
    n, last, lens = 1500, 700, [280000 - 2200, 1500, 700]
    T = sum(lens)
    assert T * H * D > 2 ** 31
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB of free device memory")
    g = torch.Generator("cuda").manual_seed(3)
    q, k, v, do = (torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    for x in (q, k, v, do):
        x[-(n + last):].normal_(generator=g)
    kw = dict(causal=True, window=(500, 0), softcap=20.0, slopes=alibi(H).cuda())

    def run(t, lengths):
        cu = ints([sum(lengths[:i]) for i in range(len(lengths) + 1)])
        o, lse = fa.forward_varlen(*t[:3], cu, max(lengths), **kw)
        return (o, lse, *fa.backward_varlen(*t[:3], o, t[3], lse, cu, max(lengths), **kw))

    big = run((q, k, v, do), lens)
    tail = n + last
    small = run([x[-tail:].contiguous() for x in (q, k, v, do)], [n, last])
    assert fa.fa_check_device_errors(None) == 0, fa.fa_last_error_detail()
    for name, a, b in zip(("O", "L", "dQ", "dK", "dV"), big, small):
        a = a[:, -tail:] if name == "L" else a[-tail:]
        assert torch.equal(a, b), name
        assert not bool(b.isnan().any()) and bool(b.any())
    assert not bool(big[0][:-tail].any()) and not bool(big[2][:-tail].any()) and not bool(big[4][:-tail].any())


@pytest.mark.parametrize("D", [64, 128])
def test_pages_past_2_32_bytes(fa, D):
    """Pages more than 2^32 bytes apart: the bits of the same pages side by side, few rows, chunks and trees."""
    page, hk, H, gap = 128, 1, 4, (1 << 31) + 128
    near = torch.randn(2, 3, page, hk, D, generator=torch.Generator().manual_seed(8)).half().cuda()
    pools = [torch.empty(2 * gap + page * hk * D, dtype=torch.float16, device="cuda") for _ in range(2)]
    far = [x.as_strided((3, page, hk, D), (gap, hk * D, D, 1)) for x in pools]
    for x, y in zip(far, near):
        x.copy_(y)
    table, kw = ints([[2, 0, 1]]), dict(softcap=9.0, slopes=alibi(H).cuda())
    for n, tree in ((1, False), (6, True), (150, False), (150, True)):
        q = rnd((n, H, D), n, torch.float16).cuda()
        if tree:
            bits, depth = make_tree(n, "tree", 0)
            kw.update(tree=words_of(bits, 5).cuda(), positions=(340 - n + depth).to(torch.int32).cuda())
        else:
            kw.pop("tree", None), kw.pop("positions", None)
        args = (table, ints([340]), ints([0, n]), n, 340)
        a, b = fa.forward_paged(q, *far, *args, **kw), fa.forward_paged(q, *near, *args, **kw)
        assert fa.fa_check_device_errors(None) == 0, fa.fa_last_error_detail()
        assert all(torch.equal(x, y) for x, y in zip(a, b)) and not bool(a[0].isnan().any())


@pytest.mark.parametrize("G", [64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_wide_groups(fa, D, G):
    """Up to 128 query heads to a K/V head, each with its slope."""
    case(fa, [40, 300], [1, 1], G, 1, D, 16, "fp16", softcap=9.0, bias=True)
    case(fa, [140, 20], [3, 2], G, 1, D, 16, "fp16", bias=True, tree="random")


def test_sliced_arguments(fa):
    """Trees and paths as slices of wider tensors, caches with their heads outside the rows, a table within a wider
    one."""
    lens, n, H, hk, D, page = [60, 200], [10, 70], 4, 2, 64, 16
    kc, vc, table, cu = paged_setup(lens, n, hk, D, page, torch.float16, 5, hnd=True)
    k1, v1 = on_gpu(kc, vc)
    k2, v2 = kc.cuda().contiguous(), vc.cuda().contiguous()
    q = rnd((cu[-1], H, D), 6, torch.float16).cuda()
    rows = torch.cat([words_of(make_tree(m, "tree", 0)[0], 3) for m in n]).cuda()
    pos = torch.cat([L - m + make_tree(m, "tree", 0)[1] for L, m in zip(lens, n)]).to(torch.int32).cuda()
    wide = torch.full((cu[-1], 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 2:5] = rows
    far = torch.full((2, 40), 1 << 20, dtype=torch.int32, device="cuda")
    far[:, 5:5 + table.shape[1]] = table.cuda()
    kw = dict(softcap=9.0, slopes=alibi(H).cuda(), positions=pos)
    a = fa.forward_paged(q, k1, v1, far[:, 5:5 + table.shape[1]], ints(lens), ints(cu), 70, 200, tree=wide[:, 2:5], **kw)
    b = fa.forward_paged(q, k2, v2, ints(table), ints(lens), ints(cu), 70, 200, tree=rows, **kw)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    paths = torch.full((2, 30), -9, dtype=torch.int32, device="cuda")
    paths[:, 7:10] = torch.tensor([[0, 2, 9], [1, 40, 69]], dtype=torch.int32, device="cuda")
    fa.paged_keep(k1, v1, far[:, 5:5 + table.shape[1]], ints(lens), ints(cu), 70, paths[:, 7:10], ints([3, 3]))
    fa.paged_keep(k2, v2, ints(table), ints(lens), ints(cu), 70, paths[:, 7:10].contiguous(), ints([3, 3]))
    assert fa.fa_check_device_errors(None) == 0
    assert torch.equal(k1, k2) and torch.equal(v1, v2)
    for b in range(2):
        at = paged.slots(table[b], torch.arange(lens[b]), page)
        f = lens[b] - n[b]
        for i, t in enumerate(paths[b, 7:10].tolist()):
            for x, y in ((k2, kc), (v2, vc)):
                assert torch.equal(x.cpu().reshape(-1, hk, D)[at[f + i]],
                                   y.contiguous().reshape(-1, hk, D)[at[f + t]])


def test_a_tree_longer_than_its_bound(fa):
    """More new tokens than max_seqlen_q: reported, that sequence's rows left as they were, the other one right."""
    lens, n, H, hk, D = [60, 90], [10, 30], 4, 2, 64
    kc, vc, table, cu = paged_setup(lens, n, hk, D, 16, torch.float16, 5)
    kc, vc = on_gpu(kc, vc)
    q = rnd((cu[-1], H, D), 6, torch.float16).cuda()
    rows = torch.cat([words_of(make_tree(m, "tree", 0)[0], 1) for m in n]).cuda()
    pos = torch.cat([L - m + make_tree(m, "tree", 0)[1] for L, m in zip(lens, n)]).to(torch.int32).cuda()
    good = fa.forward_paged(q, kc, vc, ints(table), ints(lens), ints(cu), 30, 90, tree=rows, positions=pos, softcap=4.0)
    o, lse = torch.full_like(q, 7.0), torch.full((H, cu[-1]), 7.0, device="cuda")
    fa.forward_paged(q, kc, vc, ints(table), ints(lens), ints(cu), 12, 90, tree=rows, positions=pos, softcap=4.0,
                     out=o, lse=lse)
    assert fa.STATUS[fa.fa_check_device_errors(None)] == "FA_ERR_INVALID_ARG"
    assert torch.equal(o[:10], good[0][:10]) and bool((o[10:] == 7.0).all()) and bool((lse[:, 10:] == 7.0).all())


@pytest.mark.parametrize("D,n", [(64, 5), (64, 150), (128, 150)])
def test_a_cache_shorter_than_its_new_tokens(fa, D, n):
    """kv_len < n: the first new tokens are no keys; a chunk's rows before key 0 see nothing, a tree's see by their
    bits what there is."""
    kv, H, hk, page = n - 3, 4, 2, 16
    kc, vc, table, cu = paged_setup([kv], [n], hk, D, page, torch.float16, 5)
    q = rnd((n, H, D), 6, torch.float16)
    at = paged.slots(table[0], torch.arange(kv), page)
    k, v = kc.reshape(-1, hk, D)[at], vc.reshape(-1, hk, D)[at]
    kg, vg = on_gpu(kc, vc)
    bits, depth = make_tree(n, "random", 7)
    pos = (kv - n + depth).clamp(kv - n, kv - 1)
    where = pos[n - kv:]
    args = (q.cuda(), kg, vg, ints(table), ints([kv]), ints(cu), n, kv)
    words = -(-n // 32)
    mods = dict(softcap=7.0, slopes=alibi(H).cuda())
    for tree in (False, True):
        extra = dict(tree=words_of(bits, words).cuda(), positions=pos.to(torch.int32).cuda()) if tree else {}
        o, lse = fa.forward_paged(*args, **mods, **extra)
        assert fa.fa_check_device_errors(None) == 0, fa.fa_last_error_detail()
        i = pos if tree else torch.arange(kv - n, kv)
        j = where if tree else torch.arange(kv)
        seen = bits[:, n - kv:] if tree else j[None, :] <= i[:, None]
        rs = modified.sequence(q, k, v, seen, i, j, D ** -0.5, 7.0, alibi(H))
        for h, r in enumerate(rs):
            tol_o, tol_l, _ = forward_bounds(r, q[:, h], k[:, h // 2], v[:, h // 2], D ** -0.5, 7.0, torch.float16)
            some = torch.isfinite(r["lse"])
            inside(o[:, h], r["o"], tol_o, f"O h={h}")
            assert torch.equal(torch.isneginf(lse[h].cpu()), ~some)
            inside(lse[h].cpu()[some], r["lse"][some], tol_l[some], f"L h={h}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("slope", [1.0, 1.1, 40.0, 1e6, -2.0])
def test_steep_slopes(fa, D, slope):
    """Slopes about and beyond the one from which each distance is taken by itself."""
    s = torch.tensor([slope, 0.25], dtype=torch.float32)
    fixed_case(fa, 1, 2, 1, 333, D, "fp16", slopes=s)
    fixed_case(fa, 1, 2, 1, 200, D, "bf16", slopes=s, causal=False, softcap=9.0)


@pytest.mark.parametrize("D", [64, 128])
def test_steep_slopes_in_a_cache(fa, D):
    """Rows of one tile with slopes of either kind; o = v at the row's own key where nothing else weighs."""
    lens, n, H = [400, 90], [150, 2], 4
    kc, vc, table, cu = paged_setup(lens, n, 1, D, 16, torch.float16, 5)
    kg, vg = on_gpu(kc, vc)
    q = rnd((cu[-1], H, D), 6, torch.float16)
    slopes = torch.tensor([1e25, 0.5, 3.0, 0.0])
    o, lse = fa.forward_paged(q.cuda(), kg, vg, ints(table), ints(lens), ints(cu), 150, 400, slopes=slopes.cuda())
    assert fa.fa_check_device_errors(None) == 0
    for b in range(2):
        at = paged.slots(table[b], torch.arange(lens[b]), 16)
        k, v = kc.reshape(-1, 1, D)[at], vc.reshape(-1, 1, D)[at]
        i, j = torch.arange(lens[b] - n[b], lens[b]), torch.arange(lens[b])
        qb = q[cu[b]:cu[b + 1]]
        ob, lb = o[cu[b]:cu[b + 1]].cpu(), lse[:, cu[b]:cu[b + 1]].cpu()
        assert torch.equal(ob[:, 0], v[lens[b] - n[b]:, 0])
        rs = modified.sequence(qb, k, v, j[None, :] <= i[:, None], i, j, D ** -0.5, None, slopes)
        for h, r in list(enumerate(rs))[1:]:
            tol_o, tol_l, _ = forward_bounds(r, qb[:, h], k[:, 0], v[:, 0], D ** -0.5, None, torch.float16)
            inside(ob[:, h], r["o"], tol_o, f"O b={b} h={h}")
            inside(lb[h], r["lse"], tol_l, f"L b={b} h={h}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cap", [1e-10, 1e-4, 1e10])
def test_ends_of_the_cap(fa, D, cap):
    """The smallest and largest caps, products of 0 among them: scores of +-cap and 0, or as without one."""
    q, k, v, do = (rnd((1, 2, 170, D), i, torch.float16) for i in range(4))
    q[:, :, ::7] = 0
    kw = dict(causal=True, softcap=cap)
    g = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.forward(*g[:3], **kw)
    grads = fa.backward(*g[:3], o, g[3], lse, **kw)
    tr = lambda x: x[0].cpu().transpose(0, 1)  # noqa: E731
    check_sequence(tr(q), tr(k), tr(v), tr(do), tr(o), lse[0].cpu(), [tr(x) for x in grads], True, None, 0, cap, None,
                   D ** -0.5)
    kc, vc, table, cu = paged_setup([170], [40], 2, D, 16, torch.float16, 5)
    kg, vg = on_gpu(kc, vc)
    qp = tr(q)[-40:].contiguous()
    at = paged.slots(table[0], torch.arange(170), 16)
    kk, vv = kc.reshape(-1, 2, D)[at], vc.reshape(-1, 2, D)[at]
    for n in (40, 2):
        o, lse = fa.forward_paged(qp[-n:].cuda(), kg, vg, ints(table), ints([170]), ints([0, n]), n, 170, softcap=cap)
        i, j = torch.arange(170 - n, 170), torch.arange(170)
        rs = modified.sequence(qp[-n:], kk, vv, j[None, :] <= i[:, None], i, j, D ** -0.5, cap, None)
        for h, r in enumerate(rs):
            tol_o, tol_l, _ = forward_bounds(r, qp[-n:, h], kk[:, h], vv[:, h], D ** -0.5, cap, torch.float16)
            inside(o[:, h], r["o"], tol_o, f"O h={h}")
            inside(lse[h], r["lse"], tol_l, f"L h={h}")
    assert fa.fa_check_device_errors(None) == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cu", [[0, 100, 400], [0, 300, 200, 400], [0, 100, 900], [-4, 100, 200]])
def test_offsets_that_contradict_the_call(fa, D, cu):
    """A sample longer than the bound, decreasing offsets, offsets out of the batch: reported, nothing read or
    written out of range, and the next call is right."""
    q, k, v, do = (rnd((400, 2, D), i, torch.float16).cuda() for i in range(4))
    kw = dict(causal=True, softcap=9.0, slopes=alibi(2).cuda())
    good = ints([0, 150, 400])
    o, lse = fa.forward_varlen(q, k, v, good, 250, **kw)
    grads = fa.backward_varlen(q, k, v, o, do, lse, good, 250, **kw)
    fa.forward_varlen(q, k, v, ints(cu), 250, **kw)
    assert fa.STATUS[fa.fa_check_device_errors(None)] == "FA_ERR_INVALID_ARG"
    fa.backward_varlen(q, k, v, o, do, lse, ints(cu), 250, **kw)
    assert fa.STATUS[fa.fa_check_device_errors(None)] == "FA_ERR_INVALID_ARG"
    o2, lse2 = fa.forward_varlen(q, k, v, good, 250, **kw)
    grads2 = fa.backward_varlen(q, k, v, o, do, lse, good, 250, **kw)
    assert fa.fa_check_device_errors(None) == 0
    assert all(torch.equal(a, b) for a, b in zip((o, lse, *grads), (o2, lse2, *grads2)))


def test_empty_calls(fa):
    e = lambda *s: torch.empty(*s, dtype=torch.float16, device="cuda")  # noqa: E731
    for shape in ((0, 2, 10, 64), (1, 2, 0, 64)):
        x = e(*shape)
        o, lse = fa.forward(x, x, x, softcap=2.0)
        assert o.shape == shape and all(g.shape == shape for g in fa.backward(x, x, x, o, x, lse, softcap=2.0))
    x = e(0, 2, 64)
    o, lse = fa.forward_varlen(x, x, x, ints([0, 0]), 5, softcap=2.0)
    fa.backward_varlen(x, x, x, o, x, lse, ints([0, 0]), 5, softcap=2.0)
    kc, vc, table, _ = paged_setup([20], [0], 2, 64, 16, torch.float16, 5)
    kc, vc = on_gpu(kc, vc)
    fa.forward_paged(x, kc, vc, ints(table), ints([20]), ints([0, 0]), 4, 20, softcap=2.0,
                     tree=torch.empty(0, 1, dtype=torch.int32, device="cuda"), positions=ints([]))
    fa.paged_keep(kc, vc, ints(table)[:0], ints([]), ints([0]), 4, torch.empty(0, 3, dtype=torch.int32, device="cuda"),
                  ints([]))
    assert fa.fa_check_device_errors(None) == 0


def exact_delta_bounds(r, q, k, v, do, scale, softcap, dtype):
    """backward_bounds' dQ and dK with the row's Delta summed in fp32 from P and dP instead of taken from the stored O.

    Delta' = sum_j P dP is off by sum_j p (e + errL)|dP| + p err dP + n 2^-24 p |dP|.  dS is formed with the stored O's
    Delta, off by d16, and corrected by the difference times (P o f) K: both operands' roundings then act on terms up to
    p f d16 larger, u each."""
    u, n, D = torch.finfo(dtype).eps / 2, r["p"].shape[1], q.shape[-1]
    sub = 2.0 ** -25 if dtype == torch.float16 else 0.0
    tol_o, tol_l, (ex, e) = forward_bounds(r, q, k, v, scale, softcap, dtype)
    qa, ka, va, da = (x.double().abs() for x in (q, k, v, do))
    p, g, f, dpa = r["p"], r["g"].abs(), r["f"], r["dp"].abs()
    ep = e + tol_l[:, None]
    dp = D * 2.0 ** -23 * (da @ va.T)
    d16 = (da * (tol_o + D * 2.0 ** -24 * r["o"].abs())).sum(1)[:, None]
    d32 = (p * ((ep + n * 2.0 ** -24) * dpa + dp)).sum(1)[:, None]
    ds = (ep + u) * r["ds"].abs() + p * f * (dp + d32 + 2 * u * d16) + 2 * sub * (r["s"] > -float("inf")).double() * (1 + d16)
    if softcap is not None:
        t = torch.sqrt((1 - f).clamp(min=0))
        ds = ds + p * (g + d16) * (2 * t * (ex / softcap + 2.0 ** -19 * t + 2.0 ** -21) + 2.0 ** -22)
    acc = n * 2.0 ** -23
    dsa = r["ds"].abs() + p * f * d16
    return 1.1 * abs(scale) * ((ds + acc * dsa) @ ka) + 1e-12, 1.1 * abs(scale) * ((ds + acc * dsa).T @ qa) + 1e-12


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("mods", [dict(softcap=30.0), dict(bias=True), dict(softcap=50.0, bias=True)],
                         ids=["cap", "bias", "both"])
@pytest.mark.parametrize("S", [4, 300])
def test_gradients_of_peaked_rows(fa, S, mods, dtype, D):
    """Rows whose weight lies on few keys: what dP - Delta leaves there is small against dP, and the rounding of the
    stored O has no part in dQ and dK.  The mean square error stays near the roundings of operands and results."""
    H, gain = 2, 10.0
    q, k, v, do = (rnd((1, H, S, D), 90 + i, torch.float32).mul(gain ** 0.5 if i < 2 else 1).to(dtype) for i in range(4))
    cap, slopes = mods.get("softcap"), alibi(H) if "bias" in mods else None
    kw = dict(causal=True, softcap=cap, slopes=None if slopes is None else slopes.cuda())
    gpu = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.forward(*gpu[:3], **kw)
    dq, dk, _ = fa.backward(*gpu[:3], o, gpu[3], lse, **kw)
    assert fa.fa_check_device_errors(None) == 0
    at, u = torch.arange(S), torch.finfo(dtype).eps / 2
    tr = lambda x: x[0].transpose(0, 1)  # noqa: E731
    rs = modified.sequence(tr(q), tr(k), tr(v), modified.visible(S, True), at, at, D ** -0.5, cap, slopes, tr(do))
    sub = 2.0 ** -25 if dtype == torch.float16 else 0.0
    for h, r in enumerate(rs):
        bq, bk = exact_delta_bounds(r, q[0, h], k[0, h], v[0, h], do[0, h], D ** -0.5, cap, dtype)
        inside(dq[0, h], r["dq"], bq + u * r["dq"].abs() + sub, f"dQ h={h}")
        inside(dk[0, h], r["dk"], bk + u * r["dk"].abs() + sub, f"dK h={h}")


def test_backward_of_few_rows_and_many_heads(fa):
    """One token, one head a group; the workspace's split partials hold each head's share."""
    fixed_case(fa, 2, 16, 1, 1, 64, "fp16", softcap=5.0, bias=True)
    fixed_case(fa, 1, 32, 1, 130, 128, "bf16", softcap=5.0, bias=True, prefix=64)
