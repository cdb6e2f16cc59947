"""Paged attention of batches whose sequences differ in kind: prompts of different sizes beside one another and
beside single tokens, loose bounds, and what must not reach a row from elsewhere.

Error bounds are those of tests/test_paged.py (``check``).
"""
import pytest
import torch

from oracle import paged
from tests.test_paged import case, check, fa, run  # noqa: F401  (fa is a fixture)
from tests.test_rope import ints, on_gpu, paged_setup, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture
def wait_limit(fa):  # noqa: F811
    """A pipeline wait that is never satisfied ends after 0.2 s."""
    fa.fa_set_wait_limit_ns(200_000_000)
    yield
    fa.fa_set_wait_limit_ns(0)


# ------------------------------------------------- prompts that fill different numbers of row tiles
@pytest.mark.parametrize("D", [16, 32, 64])
def test_short_prompts_of_one_and_two_tiles(fa, wait_limit, D):  # noqa: F811
    """Units of two row tiles and of one by turns, of a block or two of keys each: the tiles that share a unit's
    blocks change partners from unit to unit."""
    q_lens = [40, 20] * 32
    for _ in range(3):
        case(fa, q_lens, q_lens, 32, 8, D, 16, "bf16")


@pytest.mark.parametrize("D", [16, 32, 64])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_random_prompts(fa, wait_limit, D, seed):  # noqa: F811
    """One to four row tiles a unit in any order, one to a dozen blocks."""
    g = torch.Generator().manual_seed(seed)
    q_lens = torch.randint(17, 200, (64,), generator=g).tolist()
    lens = [n + int(x) for n, x in zip(q_lens, torch.randint(0, 2 + 300 * seed, (64,), generator=g))]
    case(fa, lens, q_lens, 32, 8, D, 16, "fp16")


@pytest.mark.parametrize("D", [16, 64])
def test_one_two_and_three_tiles_in_a_run(fa, wait_limit, D):  # noqa: F811
    """Every order of one, two, three and four row tiles, of units of one to eight blocks, few CTAs' worth."""
    g = torch.Generator().manual_seed(7)
    q_lens = [(17, 33, 65, 97)[int(x)] for x in torch.randint(0, 4, (300,), generator=g)]
    lens = [n + int(x) for n, x in zip(q_lens, torch.randint(0, 400, (300,), generator=g))]
    case(fa, lens, q_lens, 4, 1, D, 16, "bf16")


@pytest.mark.parametrize("D,tokens", [(128, 9), (128, 32), (64, 80)])
def test_tiles_without_blocks(fa, wait_limit, D, tokens):  # noqa: F811
    """Many units in a row that leave one of the CTA's tiles nothing to do (one row tile of two, three of four)."""
    g = torch.Generator().manual_seed(8)
    lens = [tokens + int(x) for x in torch.randint(0, 300, (400,), generator=g)]
    case(fa, lens, [tokens] * 400, 4, 1, D, 16, "fp16")


# ------------------------------------------------- chunks beside single tokens
@pytest.mark.parametrize("D", [64, 128])
def test_mixed_step_replayed_with_new_tables(fa, D):  # noqa: F811
    """A chunk beside single tokens, append and attention in one graph, the lengths and the block table written by a
    kernel of the graph right before: each replay moves the sequences to other pages and lengths."""
    H, hk, page, q_lens = 8, 2, 16, [150, 1, 1, 3, 1]
    cu = [0, 150, 151, 152, 155, 156]
    g = torch.Generator().manual_seed(50 + D)
    per = 40  # pages a sequence
    pages = 5 * per + 3
    kc, vc = (rnd((pages, page, hk, D), 51 + i, torch.bfloat16) for i in range(2))
    kcg, vcg = on_gpu(kc, vc)
    x = rnd((156, H + 2 * hk, D), 53, torch.bfloat16).cuda()
    lens_in, table_in = ints([0] * 5), ints(torch.zeros(5, per))
    lens, table, cug = torch.empty_like(lens_in), torch.empty_like(table_in), ints(cu)
    steps = fa.rope_steps(fa.rope_inv_freq(D)[0])

    def step():
        torch.add(lens_in, 0, out=lens)
        torch.add(table_in, 0, out=table)
        q = fa.paged_append(x[:, H:H + hk], x[:, H + hk:], kcg, vcg, table, lens, cug, 150, q=x[:, :H], steps=steps)
        return q, *fa.forward_paged(q, kcg, vcg, table, lens, cug, 150, per * page)

    def deal():
        now = [n + int(v) for n, v in zip(q_lens, torch.randint(0, 480, (5,), generator=g))]
        pick = torch.randperm(pages, generator=g)[:5 * per].view(5, per)
        lens_in.copy_(ints(now))
        table_in.copy_(ints(pick))
        return now, pick

    deal()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q, o, lse = step()
    for _ in range(6):
        now, pick = deal()
        graph.replay()
        graph.replay()  # (the second finds what the first left in the caches)
        assert fa.fa_check_device_errors(None) == 0
        check(o, lse, q.cpu(), kcg.cpu(), vcg.cpu(), pick, now, cu)


# ------------------------------------------------- what other rows must not do
def test_other_sequences_queries_do_not_reach_a_row(fa):  # noqa: F811
    """The query rows of a unit that are not its own (here the next sequence's) have no say in its rows' running
    maximum: whatever they are, the first sequence's bits stay.

    Scores 1/64 and 131/16 with this scale differ by 8 powers of two so closely that a test of the rounded sum
    lets the maximum stay and one of the rounded terms moves it, so any vote from elsewhere shows in L.
    """
    scale, low, high = float.fromhex("0x1.5b6d58p-1"), 1 / 64, 131 / 16
    hk, D, page, n = 8, 16, 128, 128 * 100
    lens, q_lens = [n, 20], [1, 8]
    kc, vc, table, cu = paged_setup(lens, q_lens, hk, D, page, torch.bfloat16, 60)
    kc.zero_()
    at = paged.slots(table[0], torch.arange(n), page)
    k = -torch.randint(1, 192, (n, hk), generator=torch.Generator().manual_seed(61)) / 64
    rise = torch.randint(0, 2, (n // 128,), generator=torch.Generator().manual_seed(62)).bool()
    k.view(-1, 128, hk)[:, 5] = torch.where(rise, high, low)[:, None]
    rows = torch.zeros(n, hk, D)
    rows[..., 0] = k
    rows.view(-1, 128, hk, D)[rise, :, :, 5] = 2.0
    kc.view(-1, hk, D)[at] = rows.bfloat16()
    q = torch.zeros(9, hk, D, dtype=torch.bfloat16)
    q[0, :, 0] = 1.0
    outs = []
    for other in (0.0, 100.0, -100.0):
        q[1:, :, 5] = other
        outs.append(run(fa, q, kc, vc, table, lens, cu, scale=scale))
        check(*outs[-1], q, kc, vc, table, lens, cu, scale=scale)
    for o, lse in outs[1:]:
        assert torch.equal(o[0], outs[0][0][0]) and torch.equal(lse[:, 0], outs[0][1][:, 0])


# ------------------------------------------------- special values that a row sees
@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("q_len", [1, 20, 40, 300])
@pytest.mark.parametrize("where", ["q", "k"])
def test_nan_under_a_scale_of_zero(fa, D, q_len, where):  # noqa: F811
    """0 times NaN: the rows concerned are NaN, whichever kernel takes them, the others the mean of their values."""
    lens, q_lens = [700, q_len + 90], [q_len, q_len]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, D, 32, torch.bfloat16, 82)
    q = rnd((cu[-1], 8, D), 83, torch.bfloat16)
    q2, k2 = q.clone(), kc.clone()
    bad = torch.zeros(cu[-1], 8, dtype=torch.bool)
    if where == "q":
        q2[q_len - 1, 1, 3] = float("nan")
        bad[q_len - 1, 1] = True
    else:
        k2.view(-1, 2, D)[paged.slots(table[0], torch.tensor([3]), 32), 0, 5] = float("nan")
        bad[:q_len, :4] = True
    o, lse = run(fa, q2, k2, vc, table, lens, cu, scale=0.0)
    bad = bad.cuda()
    assert bool(o[bad].isnan().all()) and bool(lse.T[bad].isnan().all())
    want_o, want_l = run(fa, q, kc, vc, table, lens, cu, scale=0.0)
    o[bad], lse.T[bad] = want_o[bad], want_l.T[bad]
    check(o, lse, q, kc, vc, table, lens, cu, scale=0.0)


@pytest.mark.parametrize("H,D", [(2, 64), (16, 128), (256, 64)])
def test_blocks_whose_scores_are_all_minus_infinity(fa, H, D):  # noqa: F811
    """Keys that overflowed to -infinity, whole blocks of them before others: they weigh nothing, and the rest of
    the sequence is what it is without them."""
    hk, page, blocks = 2, 128, 400
    n = 128 * blocks
    kc, vc, table, cu = paged_setup([n], [1], hk, D, page, torch.float16, 84)
    keep = torch.rand(blocks, generator=torch.Generator().manual_seed(85)) < 0.4
    keep[-1] = True
    q = rnd((1, H, D), 86, torch.float16)
    q[..., 0] = q[..., 0].abs() + 0.5
    kc[table[0, :blocks][~keep].long(), :, :, 0] = float("-inf")
    o, lse = run(fa, q, kc, vc, table, [n], cu)
    kept = table[:, :blocks][:, keep]
    check(o, lse, q, kc, vc, kept, [128 * int(keep.sum())], cu)


# ------------------------------------------------- tensors without storage
def test_tensors_without_storage_are_refused(fa):  # noqa: F811
    """Tensors that stand for others while a program is traced have no memory behind them: a Python exception, and
    the next call, which takes the same locks, works."""
    from torch._subclasses.fake_tensor import FakeTensorMode
    lens, q_lens = [40, 33], [2, 1]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 64, 16, torch.float16, 87)
    kcg, vcg = on_gpu(kc, vc)
    q = rnd((3, 4, 64), 88, torch.float16)
    qg, kg, pos = q.cuda(), rnd((3, 2, 64), 89, torch.float16).cuda(), ints([0, 1, 2])
    steps = fa.rope_steps(fa.rope_inv_freq(64)[0])
    mode = FakeTensorMode()
    fake, fake_k = mode.from_tensor(qg), mode.from_tensor(kg)
    args = (ints(table), ints(lens), ints(cu), 2)

    def traced():
        with mode:
            fa.rope(fake, fake_k, mode.from_tensor(pos), mode.from_tensor(steps))

    for call in (lambda: fa.rope(fake, kg, pos, steps), lambda: fa.rope(qg, fake_k, pos, steps),
                 lambda: fa.rope(qg, kg, pos, steps, q_out=fake), traced,
                 lambda: fa.paged_append(fake_k, kg, kcg, vcg, *args), lambda: fa.paged_append(kg, fake_k, kcg, vcg, *args),
                 lambda: fa.paged_append(kg, kg, kcg, vcg, *args, q=fake),
                 lambda: fa.forward_paged(fake, kcg, vcg, *args, 40),
                 lambda: fa.forward_paged(qg, kcg, vcg, *args, 40, out=fake)):
        with pytest.raises(Exception):
            call()
    assert torch.equal(kcg.cpu(), kc) and torch.equal(vcg.cpu(), vc)
    for _ in range(2):
        o, lse = fa.forward_paged(qg, kcg, vcg, *args, 40)
    assert fa.fa_check_device_errors(None) == 0
    check(o, lse, q, kc, vc, table, lens, cu)
    lazy = torch._lazy_clone(qg)  # shares its memory until one side is written
    qo, _ = fa.rope(lazy, kg, pos, steps, q_out=lazy)
    want, _ = fa.rope(qg, kg, pos, steps)
    assert torch.equal(qo, want) and torch.equal(qg.cpu(), q)


# ------------------------------------------------- loose bounds on the new tokens
def appended(fa, q_lens, lens, H, hk, D, max_seqlen, page=16, seed=70):  # noqa: F811
    """An append of these batches against the rotation alone, row for row and slot for slot (the same bits)."""
    T, n_pages = sum(q_lens), [-(-n // page) for n in lens]
    first = torch.tensor([0] + n_pages).cumsum(0)
    table = torch.zeros(len(lens), max(n_pages), dtype=torch.int32)
    for b, n in enumerate(n_pages):
        table[b, :n] = torch.arange(first[b], first[b] + n)
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T + 2, H + 2 * hk, D, generator=g, device="cuda").half()
    kc, vc = (torch.full((int(first[-1]), page, hk, D), 9.0, dtype=torch.float16, device="cuda") for _ in range(2))
    cu = torch.tensor([0] + q_lens).cumsum(0)
    steps = fa.rope_steps(fa.rope_inv_freq(D)[0])
    q_out = torch.full((T + 2, H, D), 7.0, dtype=torch.float16, device="cuda")
    fa.paged_append(x[:, H:H + hk], x[:, H + hk:], kc, vc, ints(table), ints(lens), ints(cu), max_seqlen, q=x[:, :H],
                    steps=steps, q_out=q_out)
    assert fa.fa_check_device_errors(None) == 0
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(q_lens))
    pos = torch.arange(T) - cu[seq + 1] + torch.tensor(lens)[seq]
    qr, kr = fa.rope(x[:T, :H], x[:T, H:H + hk], ints(pos), steps)
    assert torch.equal(q_out[:T], qr) and bool((q_out[T:] == 7).all())
    at = (first[seq] * page + pos).cuda()
    for cache, rows in ((kc, kr), (vc, x[:T, H + hk:])):
        flat = cache.view(-1, hk, D)
        assert torch.equal(flat[at], rows)
        left = torch.ones(flat.shape[0], dtype=torch.bool, device="cuda")
        left[at] = False
        assert bool((flat[left] == 9).all())


@pytest.mark.parametrize("H,hk,D", [(4, 1, 64), (32, 4, 128), (2, 2, 16)])
@pytest.mark.parametrize("q_lens", [[1] * 600, [500] + [1] * 63, [1] * 40 + [700] + [2] * 40, [0, 3, 0, 0, 900, 0, 5, 0],
                                    [0] * 30 + [250] + [0] * 30])
@pytest.mark.parametrize("bound", [None, (1 << 31) - 1])
def test_append_under_loose_bounds(fa, H, hk, D, q_lens, bound):  # noqa: F811
    """Many short sequences under a loose bound, one long beside many short ones, empty ones anywhere."""
    g = torch.Generator().manual_seed(71)
    lens = [n + int(v) for n, v in zip(q_lens, torch.randint(0, 60, (len(q_lens),), generator=g))]
    appended(fa, q_lens, lens, H, hk, D, bound or max(q_lens))


def test_append_of_a_very_large_batch_under_a_loose_bound(fa):  # noqa: F811
    """Sequences times the CTAs that the longest may need pass 2^31 here."""
    appended(fa, [1] * 47000, [1 + i % 16 for i in range(47000)], 62, 1, 128, 1 << 20)


@pytest.mark.parametrize("bound", [40, (1 << 31) - 1])
def test_append_reports_every_bad_sequence_under_a_loose_bound(fa, bound):  # noqa: F811
    """A cache length below the new tokens, or past the table, is found and left out, the others appended."""
    q_lens, lens = [40] + [1] * 60, [40] + [5] * 60
    kc, vc, table, cu = paged_setup(lens, q_lens, 1, 64, 16, torch.float16, 72)
    k, v = rnd((cu[-1], 1, 64), 73, torch.float16), rnd((cu[-1], 1, 64), 74, torch.float16)
    for b, n in ((0, 39), (7, 0), (60, -3), (33, 16 * table.shape[1] + 1)):
        now = list(lens)
        now[b] = n
        kcg, vcg = on_gpu(kc, vc)
        fa.paged_append(k.cuda(), v.cuda(), kcg, vcg, ints(table), ints(now), ints(cu), bound)
        assert fa.STATUS[fa.fa_check_device_errors(None)] == "FA_ERR_INVALID_ARG"
        want = kc.clone()
        for s in range(61):
            if s != b:
                want.view(-1, 1, 64)[paged.slots(table[s], torch.arange(lens[s] - q_lens[s], lens[s]), 16)] = \
                    k[cu[s]:cu[s + 1]]
        assert torch.equal(kcg.cpu(), want)
    for bad in (cu[:-1] + [cu[-1] + 1], [0, 40] + [41] * 60, [-1] + cu[1:], cu[:30] + [cu[30] + 5000] + cu[31:]):
        kcg, vcg = on_gpu(kc, vc)
        fa.paged_append(k.cuda(), v.cuda(), kcg, vcg, ints(table), ints([50] * 61), ints(bad), 30 if bad[1] == 40 else bound)
        assert fa.STATUS[fa.fa_check_device_errors(None)] == "FA_ERR_INVALID_ARG"


# ------------------------------------------------- loose bounds on lengths
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_lens", [[1] * 64, [3, 0, 1] * 30, [1] * 700, [150] + [1] * 63, [1] * 40 + [90, 33] + [2] * 9])
@pytest.mark.parametrize("max_q,max_k", [(1 << 29, 131072), (1 << 29, 1 << 29), (4000, None)])
def test_attention_under_loose_bounds(fa, D, q_lens, max_q, max_k):  # noqa: F811
    """The largest bounds there are, at batches of many sequences."""
    g = torch.Generator().manual_seed(75)
    lens = [n + int(x) for n, x in zip(q_lens, torch.randint(1, 150, (len(q_lens),), generator=g))]
    kc, vc, table, cu = paged_setup(lens, q_lens, 1, D, 16, torch.bfloat16, 76)
    q = rnd((cu[-1] + 1, 8, D), 77, torch.bfloat16)
    o, lse = run(fa, q, kc, vc, table, lens, cu, max_q=max_q, max_k=max_k)
    check(o, lse, q, kc, vc, table, lens, cu)


@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("H,hk", [(1, 1), (8, 1), (128, 1)])
def test_one_token_among_many_rows_without_sequence(fa, D, H, hk):  # noqa: F811
    """A padded batch of one token: by its bounds a chunk, so the kernel for chunks takes it."""
    kc, vc, table, cu = paged_setup([5000], [1], hk, D, 16, torch.bfloat16, 96)
    q = rnd((2000, H, D), 97, torch.bfloat16)
    o = torch.full((2000, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, 2000), 6.0, device="cuda")
    run(fa, q, kc, vc, table, [5000], cu, max_q=2000, max_k=100000, out=o, lse=lse)
    assert bool((o[1:] == 5).all()) and bool((lse[:, 1:] == 6).all())
    check(o, lse, q, kc, vc, table, [5000], cu)


def test_bad_lengths_behind_many_sequences_under_a_loose_bound(fa):  # noqa: F811
    """Each sequence's lengths are looked at, also where most tiles of the bound do not exist."""
    lens, q_lens = [30] * 900, [1] * 900
    kc, vc, table, cu = paged_setup(lens, q_lens, 1, 64, 16, torch.float16, 98)
    q = rnd((900, 8, 64), 99, torch.float16)
    kcg, vcg = on_gpu(kc, vc)
    for b in (0, 1, 450, 899):
        now = list(lens)
        now[b] = 1 << 20
        o, lse = fa.forward_paged(q.cuda(), kcg, vcg, ints(table), ints(now), ints(cu), 1 << 20, 1 << 29)
        assert fa.STATUS[fa.fa_check_device_errors(None)] == "FA_ERR_INVALID_ARG"
        some = [i for i in range(max(0, b - 3), min(900, b + 4)) if i != b]
        check(o[some], lse[:, some], q[some], kc, vc, table[some], [30] * len(some), list(range(len(some) + 1)))


@pytest.mark.parametrize("D", [64, 128])
def test_mixed_call_in_a_workspace_of_anything(fa, D):  # noqa: F811
    """Both kernels of a mixed call share a workspace: whatever it holds on entry, and used again and again, by calls
    of one kernel in between, the result is the same; after a call whose waits run out, too."""
    lens, q_lens = [600, 900, 50, 300], [200, 1, 4, 1]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, D, 32, torch.bfloat16, 63)
    q = rnd((cu[-1], 8, D), 64, torch.bfloat16)
    kcg, vcg = on_gpu(kc, vc)
    args = (kcg, vcg, ints(table), ints(lens))
    need = fa.fa_fwd_paged_workspace_size(4, 200, 900, 8, 2, D)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    o, lse = fa.forward_paged(q.cuda(), *args, ints(cu), 200, 900, workspace=ws)
    check(o, lse, q, kc, vc, table, lens, cu)
    one, single = q[:4].cuda(), ints([0, 1, 2, 3, 4])
    for fill in (0, 255, 127, 1, None, "single", "late", None):
        if isinstance(fill, int):
            ws.fill_(fill)
        elif fill == "single":
            fa.forward_paged(one, *args, single, 1, 900, workspace=ws)
        elif fill == "late":
            fa.fa_set_wait_limit_ns(1)
            try:
                fa.forward_paged(q.cuda(), *args, ints(cu), 200, 900, workspace=ws)
                torch.cuda.synchronize()
            finally:
                fa.fa_set_wait_limit_ns(0)
            assert fa.STATUS[fa.fa_check_device_errors(None)] == "FA_ERR_TIMEOUT"
        o2, l2 = fa.forward_paged(q.cuda(), *args, ints(cu), 200, 900, workspace=ws)
        assert fa.fa_check_device_errors(None) == 0
        assert torch.equal(o, o2) and torch.equal(lse, l2)
    with pytest.raises(fa.FAError):
        fa.forward_paged(q.cuda(), *args, ints(cu), 200, 900, workspace=ws[:-256])


@pytest.mark.parametrize("D", [64, 128])
def test_mixed_calls_on_two_streams_and_in_graphs(fa, D):  # noqa: F811
    """Mixed calls unsynchronised on two streams, each with its stream's scratch, beside two replayed graphs of the
    same calls, each with its own."""
    lens, q_lens = [2500, 900, 50, 300, 77], [200, 1, 4, 1, 1]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, D, 32, torch.bfloat16, 65)
    kcg, vcg = on_gpu(kc, vc)
    args = (kcg, vcg, ints(table), ints(lens), ints(cu), 200, 2500)
    qs = [rnd((cu[-1], 8, D), 66 + i, torch.bfloat16) for i in range(2)]
    qg = [x.cuda() for x in qs]
    want = [fa.forward_paged(x, *args) for x in qg]
    check(*want[0], qs[0], kc, vc, table, lens, cu)
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, [fa.forward_paged(qg[i], *args) for _ in range(3)]))
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for i in range(2):
            got.append((i, fa.forward_paged(qg[i], *args, stream=streams[i])))
            with torch.cuda.stream(streams[1 - i]):
                graphs[i][0].replay()
    torch.cuda.synchronize()
    assert fa.fa_check_device_errors(None) == 0
    for i, (o, lse) in got + [(i, r) for i in range(2) for r in graphs[i][1]]:
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


@pytest.mark.parametrize("order", ["rows", "heads"])
@pytest.mark.parametrize("q_len", [1, 100])
@pytest.mark.parametrize("D", [16, 64, 128])
def test_padded_strides(fa, order, q_len, D):  # noqa: F811
    """Strides that are multiples of 8 elements and of nothing else, append and attention."""
    hk, page, lens, q_lens = 3, 16, [200, 130], [q_len, 1]
    kc, vc, table, cu = paged_setup(lens, q_lens, hk, D, page, torch.float16, 68)
    n = kc.shape[0]
    if order == "rows":    # [pages, rows, heads, D] with room behind heads, rows and pages
        head, row = D + 8, hk * (D + 8) + 16
        strides = (page * row + 24, row, head, 1)
    else:                  # [pages, heads, rows, D]
        row, head = D + 8, page * (D + 8) + 40
        strides = (hk * head + 8, row, head, 1)
    caches = [torch.full((n * strides[0],), float("nan"), dtype=torch.float16, device="cuda") for _ in range(2)]
    kcg, vcg = (c.as_strided(kc.shape, strides) for c in caches)
    kcg.copy_(kc)
    vcg.copy_(vc)
    k, v, q = rnd((cu[-1], hk, D), 69, torch.float16), rnd((cu[-1], hk, D), 70, torch.float16), \
        rnd((cu[-1], 2 * hk, D), 71, torch.float16)
    args = (kcg, vcg, ints(table), ints(lens), ints(cu), q_len)
    fa.paged_append(k.cuda(), v.cuda(), *args)
    kn, vn = paged.append(kc, k, table, lens, cu), paged.append(vc, v, table, lens, cu)
    assert torch.equal(kcg.cpu(), kn) and torch.equal(vcg.cpu(), vn)
    for c, x in zip(caches, (kn, vn)):  # the room between is as it was
        assert int(c.isnan().sum()) == c.numel() - x.numel()
    o, lse = fa.forward_paged(q.cuda(), *args, 200)
    assert fa.fa_check_device_errors(None) == 0
    check(o, lse, q, kn, vn, table, lens, cu)
