"""Attention of new tokens over a paged cache on the GPU, against the fp64 oracle.

Error bound of an output element, term by term (W = sum_j p_j |v_j|):
  - P is rounded to the 16-bit type (half a step, u) before the second product: u W; for fp16 also half a
    subnormal step, 2^-25, of each 2^(s - m), whose sum is at least 1: 2^-25 sum_j |v_j| e^(max s - L);
  - a weight's exponent is off by e = scale (D + 4) 2^-23 max_ij sum_d |q_d k_d| (fp32 products and sums,
    truncated at worst) + 2^-21 (its exponential, the running sums), above and below the line: 2 e W;
  - the stored result: u |O|, and 2^-25 for fp16's subnormals.
L is off by e + 2^-22 |L| + 2^-21 (its logarithm).
"""
import math
import threading

import pytest
import torch

from oracle import paged
from oracle.attention import as_f64
from tests.test_rope import DT, ints, on_gpu, paged_setup, projection, rnd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_18_gb300 as m
    m.load_library()
    return m


def check(o, lse, q, kc, vc, table, lens, cu, causal=True, window=None, scale=None):
    D, H, hk = q.shape[2], q.shape[1], kc.shape[2]
    u = torch.finfo(q.dtype).eps / 2
    sc = 1 / math.sqrt(D) if scale is None else scale
    ro, rl, w = paged.attend(q, kc, vc, table, lens, cu, causal, window, scale)
    G = H // hk
    for b, (t0, t1) in enumerate(zip(cu[:-1], cu[1:])):
        if t1 == t0:
            continue
        lo = 0 if window is None or window[0] < 0 else max(0, lens[b] - (t1 - t0) - window[0])
        at = paged.slots(table[b], torch.arange(lo, lens[b]), kc.shape[1])
        for h in range(H):
            k = as_f64(kc.reshape(-1, hk, D)[at, h // G])
            v = as_f64(vc.reshape(-1, hk, D)[at, h // G])
            e = abs(sc) * (D + 4) * 2.0 ** -23 * float((as_f64(q[t0:t1, h]).abs() @ k.abs().T).max()) + 2.0 ** -21 \
                if len(at) else 2.0 ** -21
            ref, got = ro[t0:t1, h], o[t0:t1, h].cpu().double()
            tol = (u + 2 * e) * w[t0:t1, h] + u * ref.abs() + 1e-12
            if q.dtype == torch.float16 and len(at):
                s = sc * as_f64(q[t0:t1, h]) @ k.T
                lift = torch.exp((s.amax(1) - rl[h, t0:t1]).clamp(max=80.0))
                tol = tol + 2.0 ** -25 * (1 + v.abs().sum(0)[None, :] * torch.nan_to_num(lift, nan=0.0)[:, None])
            d = (got - ref).abs()
            assert bool((d <= tol).all()), f"O b={b} h={h}: worst error {float((d / tol).max()):.2f} of its bound"
            rl_h, got_l = rl[h, t0:t1], lse[h, t0:t1].cpu().double()
            seen = torch.isfinite(rl_h)
            assert torch.equal(torch.isneginf(got_l), ~seen), f"L b={b} h={h}: rows that see no key"
            assert bool(((got_l - rl_h).abs()[seen] <= e + 2.0 ** -21 + 2.0 ** -22 * rl_h.abs()[seen]).all()), \
                f"L b={b} h={h}"
            assert bool((got[~seen] == 0).all())


def poison(kc, vc, table, lens, cu, window=None):
    """NaN and infinity in every cache row no query sees, and table entries of unseen pages out of range."""
    kc, vc, table = kc.clone(), vc.clone(), table.clone()
    page = kc.shape[1]
    live = torch.zeros(kc.shape[0], page, dtype=torch.bool)
    for b, n in enumerate(lens):
        nq = cu[b + 1] - cu[b]
        lo = n if nq == 0 else (0 if window is None or window[0] < 0 else max(0, n - nq - window[0]))
        live.view(-1)[paged.slots(table[b], torch.arange(lo, n), page)] = True
        table[b, :lo // page] = -1
        if nq == 0:
            table[b] = -1
    kc[~live], vc[~live] = float("nan"), float("inf")
    return kc, vc, table


def run(fa, q, kc, vc, table, lens, cu, causal=True, window=None, scale=None, max_q=None, max_k=None, **kw):
    nq = [b - a for a, b in zip(cu[:-1], cu[1:])]
    kcg, vcg = on_gpu(kc, vc)
    o, lse = fa.forward_paged(q.cuda(), kcg, vcg, ints(table), ints(lens), ints(cu), max_q or max(nq + [1]),
                              max_k or max(lens), causal=causal, window=window, scale=scale, **kw)
    assert fa.fa_check_device_errors(None) == 0, fa.fa_last_error_detail()
    return o, lse


def case(fa, lens, q_lens, H, hk, D, page, dtype, causal=True, window=None, scale=None, hnd=False, std=1.0, seed=0):
    kc, vc, table, cu = paged_setup(lens, q_lens, hk, D, page, DT[dtype], sum(lens) + seed, hnd=hnd)
    q = rnd((cu[-1], H, D), sum(lens) + 1, torch.float32).mul(std).to(DT[dtype])
    kp, vp, tp = poison(kc, vc, table, lens, cu, window)
    o, lse = run(fa, q, kp, vp, tp, lens, cu, causal, window, scale)
    check(o, lse, q, kc, vc, table, lens, cu, causal, window, scale)


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens(fa, D, dtype, page):
    """Decoding: one token a sequence, lengths around page and block borders, one of length 1."""
    case(fa, [1, 127, 128, 129, 700, 15, 16, 17], [1] * 8, 8, 2, D, page, dtype)


@pytest.mark.parametrize("H,hk", [(1, 1), (5, 1), (16, 1), (17, 1), (33, 1), (65, 1), (128, 1), (14, 2), (6, 3), (9, 9)])
@pytest.mark.parametrize("D", [64, 128])
def test_group_sizes(fa, H, hk, D):
    """Rows of a unit across the kernel's four sizes, filled and not."""
    case(fa, [300, 77], [1, 1], H, hk, D, 32, "bf16")


@pytest.mark.parametrize("q_len", [2, 3, 7, 16, 31, 100])
@pytest.mark.parametrize("D,dtype", [(64, "fp16"), (128, "bf16"), (32, "bf16")])
def test_short_chunks(fa, q_len, D, dtype):
    case(fa, [q_len, 500, q_len + 128], [q_len, q_len, max(1, q_len - 2)], 6, 2, D, 16, dtype)


@pytest.mark.parametrize("lens,q_lens", [
    ([900], [700]), ([513, 2000, 64], [513, 130, 1]), ([300, 0, 40, 129], [300, 0, 40, 1]),
])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("H,hk", [(4, 4), (6, 2)])
def test_chunks(fa, lens, q_lens, D, dtype, H, hk):
    case(fa, lens, q_lens, H, hk, D, 64, dtype)


@pytest.mark.parametrize("window", [(0, 0), (1, 0), (127, 0), (128, 0), (200, 0), (5000, 0)])
@pytest.mark.parametrize("q_len", [1, 5, 200])
@pytest.mark.parametrize("D", [64, 128])
def test_windows(fa, window, q_len, D):
    """Pages before the window are not there (their entries are out of range), rows before it hold NaN."""
    case(fa, [1500, q_len, 640], [q_len, q_len, 1], 4, 2, D, 16, "bf16", window=window)


@pytest.mark.parametrize("window", [None, (-1, 3), (10, 10), (40, -1)])
@pytest.mark.parametrize("q_len", [1, 9, 150])
def test_not_causal(fa, window, q_len):
    case(fa, [400, q_len], [q_len, q_len], 4, 2, 64, 32, "fp16", causal=False, window=window)


FEW_TILES = [  # what is special, arguments of the case (G = 8: 12 tokens are one tile of rows, 30 are two)
    ("no scale", dict(scale=0.0)), ("negative", dict(scale=-0.2)), ("steep", dict(scale=1.5)),
    ("only itself", dict(window=(0, 0))), ("both sides", dict(causal=False, window=(100, 70))),
    ("right side", dict(causal=False, window=(-1, 3))), ("all", dict(causal=False)), ("large", dict(std=8.0)),
]


@pytest.mark.parametrize("D", [16, 64])
@pytest.mark.parametrize("q_len", [12, 30])
@pytest.mark.parametrize("kw", [kw for _, kw in FEW_TILES], ids=[n for n, _ in FEW_TILES])
def test_units_of_few_tiles_masks_and_scales(fa, q_len, D, kw):
    case(fa, [2500, q_len, 700], [q_len] * 3, 8, 1, D, 16, "fp16", **kw)


@pytest.mark.parametrize("D", [32, 64])
@pytest.mark.parametrize("q_len", [12, 30])
@pytest.mark.parametrize("down", [False, True])
def test_units_of_few_tiles_moving_maximum(fa, q_len, D, down):
    """Keys that grow, or shrink, along the cache: the tiles that share a unit end with maxima far apart."""
    lens, q_lens = [3000, 400], [q_len, q_len]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, D, 32, torch.float16, 90)
    at = paged.slots(table[0], torch.arange(3000), 32)
    ramp = torch.linspace(0.05, 6, 3000)
    kc.view(-1, 2, D)[at] *= (ramp.flip(0) if down else ramp)[:, None, None].half()
    q = rnd((cu[-1], 16, D), 91, torch.float16)
    o, lse = run(fa, q, kc, vc, table, lens, cu)
    check(o, lse, q, kc, vc, table, lens, cu)


@pytest.mark.parametrize("q_len", [12, 30])
def test_units_of_few_tiles_long_context(fa, q_len):
    """One sequence over all CTAs, rows that see nothing beside it, the same bits twice."""
    lens, q_lens = [60000, 5, 0], [q_len] * 3
    kc, vc, table, cu = paged_setup([60000, 5], [q_len] * 3, 1, 64, 64, torch.bfloat16, 92)
    table = torch.cat((table, torch.full((1, table.shape[1]), -1, dtype=torch.int32)))
    q = rnd((cu[-1], 8, 64), 93, torch.bfloat16)
    o, lse = run(fa, q, kc, vc, table, lens, cu)
    check(o, lse, q, kc, vc, table, lens, cu)
    o2, l2 = run(fa, q, kc, vc, table, lens, cu)
    assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("q_len", [12, 30])
def test_units_of_few_tiles_wait_runs_out(fa, q_len):
    """Tiles that wait for one another give up together, and the next call is right."""
    lens, q_lens = [3000, 1000], [q_len, q_len]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 64, 32, torch.bfloat16, 94)
    q = rnd((cu[-1], 16, 64), 95, torch.bfloat16)
    kcg, vcg = on_gpu(kc, vc)
    assert fa.fa_check_device_errors(None) == 0
    fa.fa_set_wait_limit_ns(1)
    try:
        fa.forward_paged(q.cuda(), kcg, vcg, ints(table), ints(lens), ints(cu), q_len, 3000)
        st = fa.fa_check_device_errors(None)
    finally:
        fa.fa_set_wait_limit_ns(0)
    assert fa.STATUS[st] == "FA_ERR_TIMEOUT"
    o, lse = run(fa, q, kc, vc, table, lens, cu)
    check(o, lse, q, kc, vc, table, lens, cu)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len,longest", [(1, 300), (1, 40000), (40, 300), (40, 20000), (70, 20000), (300, 400), (300, 20000)])
@pytest.mark.parametrize("where", ["q", "k"])
def test_nan_that_is_seen(fa, D, q_len, longest, where):
    """NaN in a query, or in a key it sees, reaches the rows concerned, however the context is cut, and no others."""
    lens, q_lens = [longest, q_len + 90], [q_len, q_len]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, D, 32, torch.bfloat16, 80)
    q = rnd((cu[-1], 8, D), 81, torch.bfloat16)
    q2, k2 = q.clone(), kc.clone()
    bad = torch.zeros(cu[-1], 8, dtype=torch.bool)
    if where == "q":
        q2[q_len - 1, 1, 3] = float("nan")
        bad[q_len - 1, 1] = True
    else:  # key 3 of the first sequence, first K/V head: seen by all its rows at position 3 or later
        k2.view(-1, 2, D)[paged.slots(table[0], torch.tensor([3]), 32), 0, 5] = float("nan")
        bad[:q_len, :4] = True
    o, lse = run(fa, q2, k2, vc, table, lens, cu)
    bad = bad.cuda()
    assert bool(o[bad].isnan().all()) and bool(lse.T[bad].isnan().all())
    want_o, want_l = run(fa, q, kc, vc, table, lens, cu)
    o[bad], lse.T[bad] = want_o[bad], want_l.T[bad]
    check(o, lse, q, kc, vc, table, lens, cu)


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("q_len", [9, 16, 17, 33, 48])
@pytest.mark.parametrize("window", [None, (70, -1), (1000, -1)])
def test_units_of_few_tiles(fa, q_len, D, window):
    """One to three tiles of rows a unit (G = 8): blocks taken in turns, fewer blocks than tiles, cut and whole units."""
    case(fa, [5000, 48, 1300, 64, 700, 129], [q_len] * 6, 8, 1, D, 32, "bf16", window=window)


@pytest.mark.parametrize("D", [64, 128])
def test_units_of_few_tiles_in_one_piece(fa, D):
    """More units than CTAs, so that most are not cut, of one and two tiles each, in both orders."""
    lens = [200 + 61 * i for i in range(12)]
    case(fa, lens, [70 if i % 3 else 150 for i in range(12)], 16, 16, D, 64, "fp16")


@pytest.mark.parametrize("q_len", [1, 40, 200])
@pytest.mark.parametrize("D", [16, 128])
def test_rows_that_see_nothing(fa, q_len, D):
    """An empty cache, and more new tokens than keys: O = 0, L = -inf, other sequences as ever."""
    kc, vc, table, cu = paged_setup([q_len // 2 + 1, 300], [q_len, q_len, q_len], 2, D, 16, torch.bfloat16, 3)
    table = torch.cat((torch.full((1, table.shape[1]), -1, dtype=torch.int32), table))
    lens = [0, q_len // 2 + 1, 300]
    q = rnd((cu[-1], 4, D), 4, torch.bfloat16)
    o, lse = run(fa, q, kc, vc, table, lens, cu)
    check(o, lse, q, kc, vc, table, lens, cu)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
@pytest.mark.parametrize("q_len", [1, 130])
def test_scales(fa, scale, q_len):
    case(fa, [333, 1000], [q_len, q_len], 4, 2, 64, 32, "fp16", scale=scale)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len", [1, 150])
def test_rising_maximum(fa, D, q_len):
    """Keys that grow along the cache move the running maximum again and again."""
    lens, q_lens = [2000], [q_len]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, D, 32, torch.float16, 5)
    at = paged.slots(table[0], torch.arange(2000), 32)
    kc.view(-1, 2, D)[at] *= torch.linspace(0.05, 6, 2000)[:, None, None].half()
    q = rnd((q_len, 8, D), 6, torch.float16)
    o, lse = run(fa, q, kc, vc, table, lens, cu)
    check(o, lse, q, kc, vc, table, lens, cu)


@pytest.mark.parametrize("form", ["hnd", "pool"])
@pytest.mark.parametrize("q_len", [1, 140])
def test_strides(fa, form, q_len):
    if form == "hnd":
        return case(fa, [700, 90], [q_len, 1], 4, 2, 128, 64, "bf16", hnd=True)
    lens, q_lens = [300, 200], [q_len, q_len]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 64, 16, torch.float16, 7, shared=True)
    pool = torch.stack((kc, vc), 1).cuda()
    q = rnd((cu[-1], 6, 64), 8, torch.float16)
    o, lse = fa.forward_paged(q.cuda(), pool[:, 0], pool[:, 1], ints(table), ints(lens), ints(cu), q_len, 300)
    assert fa.fa_check_device_errors(None) == 0
    check(o, lse, q, kc, vc, table, lens, cu)


def test_long_contexts_cut_between_ctas(fa):
    """Contexts that many CTAs share; bounds looser than the lengths; twice the same bits."""
    lens, q_lens = [20000, 3, 9001], [1, 1, 1]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 128, 128, torch.bfloat16, 9)
    q = rnd((3, 16, 128), 10, torch.bfloat16)
    o, lse = run(fa, q, kc, vc, table, lens, cu, max_q=2, max_k=20480)
    check(o, lse, q, kc, vc, table, lens, cu)
    o2, l2 = run(fa, q, kc, vc, table, lens, cu, max_q=2, max_k=20480)
    assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("q_len", [1, 3, 300])
@pytest.mark.parametrize("D", [16, 64, 128])
def test_one_long_sequence(fa, q_len, D):
    """One sequence, one K/V head: the whole GPU shares each unit, in parts that a kernel of its own joins."""
    case(fa, [9000], [q_len], 4, 1, D, 32, "fp16")


@pytest.mark.parametrize("q_len", [1, 200])
def test_loosest_bound(fa, q_len):
    """The largest bound on the cache lengths there is (the kernels then count blocks in 64 bits)."""
    lens, q_lens = [700, 300], [q_len, 1]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 64, 32, torch.float16, 42)
    q = rnd((cu[-1], 8, 64), 43, torch.float16)
    o, lse = run(fa, q, kc, vc, table, lens, cu, max_k=1 << 29)
    check(o, lse, q, kc, vc, table, lens, cu)
    o2, l2 = run(fa, q, kc, vc, table, lens, cu)
    assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("q_len", [1, 20, 200])
def test_garbage_in_the_workspace_does_not_matter(fa, q_len):
    """Every bit pattern a workspace may hold on entry; the same one used again and again."""
    lens, q_lens = [3000, 777], [q_len, q_len]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 64, 32, torch.bfloat16, 40)
    q = rnd((cu[-1], 8, 64), 41, torch.bfloat16)
    need = fa.fa_fwd_paged_workspace_size(2, q_len, 3000, 8, 2, 64)
    first = None
    for fill in (0, 255, 127, None, None):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda") if fill is not None else ws
        o, lse = run(fa, q, kc, vc, table, lens, cu, workspace=ws)
        if first is None:
            check(o, lse, q, kc, vc, table, lens, cu)
            first = (o, lse)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_many_sequences(fa):
    g = torch.Generator().manual_seed(11)
    lens = torch.randint(1, 200, (500,), generator=g).tolist()
    q_lens = [int(x) for x in torch.randint(0, 3, (500,), generator=g)]
    q_lens = [min(a, b) for a, b in zip(q_lens, lens)]
    case(fa, lens, q_lens, 2, 1, 32, 16, "fp16")


@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("H,hk", [(1, 1), (8, 1), (128, 1)])
def test_one_token_under_a_loose_bound(fa, D, H, hk):
    """One sequence, one token, a bound of many: the kernel for chunks takes it."""
    lens, q_lens = [5000], [1]
    kc, vc, table, cu = paged_setup(lens, q_lens, hk, D, 16, torch.bfloat16, 96)
    q = rnd((1, H, D), 97, torch.bfloat16)
    o, lse = run(fa, q, kc, vc, table, lens, cu, max_q=2000, max_k=100000)
    check(o, lse, q, kc, vc, table, lens, cu)


@pytest.mark.parametrize("batch", [250, 650])
@pytest.mark.parametrize("short", [0, 1, 5])
def test_many_sequences_beside_long_ones(fa, batch, short):
    """Many sequences of few (or no) new tokens behind two of many, more of them than a CTA has threads."""
    q_lens = [130] + [short] * (batch - 2) + [90]
    lens = [400] + [20 + i % 50 for i in range(batch - 2)] + [95]
    case(fa, lens, q_lens, 4, 1, 64, 16, "fp16")


def test_offsets_past_32_bits(fa):
    """Pages beyond 2^32 elements of the cache."""
    hk, D, page, pages = 2, 128, 256, 70000  # 4.6e9 elements a cache, one buffer for K and V
    buf = torch.empty(pages, page, hk, D, dtype=torch.bfloat16, device="cuda")
    ids = [69999, 3, 65537, 40000]
    lens, cu = [900, 77], [0, 1, 3]
    table = torch.tensor([ids, [12345, -1, -1, -1]], dtype=torch.int32)
    rows = rnd((5, page, hk, D), 12, torch.bfloat16)
    new = rnd((3, hk, D), 13, torch.bfloat16)
    for i, x in enumerate(ids + [12345]):
        buf[x] = rows[i].cuda()
    fa.paged_append(new.cuda(), new.cuda(), buf, buf, ints(table), ints(lens), ints(cu), 2)
    small = torch.tensor([[0, 1, 2, 3], [4, -1, -1, -1]])
    want = paged.append(rows, new, small, lens, cu)
    for i, x in enumerate(ids + [12345]):
        assert torch.equal(buf[x].cpu(), want[i])
    q = rnd((3, 4, D), 14, torch.bfloat16)
    o, lse = fa.forward_paged(q.cuda(), buf, buf, ints(table), ints(lens), ints(cu), 2, 900)
    assert fa.fa_check_device_errors(None) == 0
    check(o, lse, q, want, want, small, lens, cu)


def test_rows_behind_the_last_sequence_stay(fa):
    lens, q_lens = [100, 60], [3, 2]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 64, 16, torch.float16, 15)
    q = rnd((9, 4, 64), 16, torch.float16)
    q[5:] = float("nan")  # a padded batch: tokens no sequence covers
    o = torch.full((9, 4, 64), 5.0, dtype=torch.float16, device="cuda")
    lse = torch.full((4, 9), 6.0, device="cuda")
    run(fa, q, kc, vc, table, lens, cu, out=o, lse=lse)
    assert bool((o[5:] == 5).all()) and bool((lse[:, 5:] == 6).all())
    check(o[:5], lse[:, :5], q[:5], kc, vc, table, lens, cu)


def test_bad_pages_and_lengths_are_reported(fa):
    lens, q_lens = [100, 60], [1, 1]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 64, 16, torch.float16, 17)
    q = rnd((2, 4, 64), 18, torch.float16)
    kcg, vcg = on_gpu(kc, vc)
    bad = table.clone()
    bad[0, 3] = kc.shape[0]
    for t, n, c, mk in ((bad, lens, cu, 100), (table, [101, 60], cu, 100), (table, [-1, 60], cu, 100), (table, [300, 60], cu, 400),
                        (table, lens, [0, 1, 4], 100), (table, lens, [0, 2, 1], 100)):
        fa.forward_paged(q.cuda(), kcg, vcg, ints(t), ints(n), ints(c), 1, mk)
        assert fa.STATUS[fa.fa_check_device_errors(None)] == "FA_ERR_INVALID_ARG"
    o, lse = run(fa, q, kc, vc, table, lens, cu)
    check(o, lse, q, kc, vc, table, lens, cu)


def test_slice_of_a_wider_table(fa):
    """A block table that is a slice: right, and a length past the slice's row is reported, not followed."""
    lens, q_lens = [48, 33], [1, 1]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 64, 16, torch.float16, 70)
    (_, k, v), (qg, kg, vg) = projection(2, 4, 2, 64, torch.float16, 71)
    kcg, vcg = on_gpu(kc, vc)
    wide = torch.zeros(4, 16, dtype=torch.int32)
    wide[:2, 2:5] = table[:, :3]
    part = wide.cuda()[:2, 2:5]
    o, lse = fa.forward_paged(qg.contiguous(), kcg, vcg, part, ints(lens), ints(cu), 1, 256)
    assert fa.fa_check_device_errors(None) == 0
    check(o, lse, qg.contiguous().cpu(), kc, vc, table, lens, cu)
    for n in ([49, 33], [48, 49]):
        fa.forward_paged(qg.contiguous(), kcg, vcg, part, ints(n), ints(cu), 1, 256)
        assert fa.STATUS[fa.fa_check_device_errors(None)] == "FA_ERR_INVALID_ARG"
    fa.paged_append(kg, vg, kcg, vcg, part, ints([49, 33]), ints(cu), 1)
    assert fa.STATUS[fa.fa_check_device_errors(None)] == "FA_ERR_INVALID_ARG"
    want = kc.clone()
    want.view(-1, 2, 64)[paged.slots(table[1], torch.arange(32, 33), 16)] = k[1:]
    assert torch.equal(kcg.cpu(), want)


def test_a_bad_sequence_leaves_the_others_right(fa):
    lens, q_lens = [100, 60, 500], [1, 1, 1]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 64, 16, torch.float16, 19)
    q = rnd((3, 4, 64), 20, torch.float16)
    kcg, vcg = on_gpu(kc, vc)
    o, lse = fa.forward_paged(q.cuda(), kcg, vcg, ints(table), ints([100, 9999, 500]), ints(cu), 1, 500)
    assert fa.STATUS[fa.fa_check_device_errors(None)] == "FA_ERR_INVALID_ARG"
    check(o[:1], lse[:, :1], q[:1], kc, vc, table[:1], [100], [0, 1])
    check(o[2:], lse[:, 2:], q[2:], kc, vc, table[2:], [500], [0, 1])


@pytest.mark.parametrize("q_len,D", [(1, 128), (1, 64), (300, 128), (300, 64)])
def test_wait_runs_out_and_the_next_call_is_right(fa, q_len, D):
    """With a 1 ns limit the pipeline's waits give up: the call ends, reports it, and the next one is right."""
    lens, q_lens = [3000, 1000], [q_len, q_len]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, D, 32, torch.bfloat16, 21)
    q = rnd((cu[-1], 8, D), 22, torch.bfloat16)
    kcg, vcg = on_gpu(kc, vc)
    assert fa.fa_check_device_errors(None) == 0
    fa.fa_set_wait_limit_ns(1)
    try:
        fa.forward_paged(q.cuda(), kcg, vcg, ints(table), ints(lens), ints(cu), q_len, 3000)
        st = fa.fa_check_device_errors(None)
    finally:
        fa.fa_set_wait_limit_ns(0)
    assert fa.STATUS[st] == "FA_ERR_TIMEOUT"
    o, lse = run(fa, q, kc, vc, table, lens, cu)
    check(o[:1], lse[:, :1], q[:1], kc, vc, table, [lens[0] - q_len + 1], [0, 1])


def test_other_stream_and_captured_graph(fa):
    """A call on a stream of its own; a captured call replayed after the lengths and the cache grew."""
    lens, q_lens = [200, 90], [1, 1]
    kc, vc, table, cu = paged_setup([400, 200], q_lens, 2, 64, 16, torch.bfloat16, 23)
    q = rnd((2, 8, 64), 24, torch.bfloat16)
    kcg, vcg = on_gpu(kc, vc)
    qg, tg, lg, cg = q.cuda(), ints(table), ints(lens), ints(cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, lse = fa.forward_paged(qg, kcg, vcg, tg, lg, cg, 1, 400, stream=side)
    side.synchronize()
    check(o, lse, q, kc, vc, table, lens, cu)
    need = fa.fa_fwd_paged_workspace_size(2, 1, 400, 8, 2, 64)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    graphs = []
    for _ in range(2):  # two captured graphs that share one workspace, replayed in turn
        g, out, l2 = torch.cuda.CUDAGraph(), torch.empty_like(qg), torch.empty(8, 2, device="cuda")
        with torch.cuda.graph(g):
            fa.forward_paged(qg, kcg, vcg, tg, lg, cg, 1, 400, out=out, lse=l2, workspace=ws)
        graphs.append((g, out, l2))
    for step in range(3):
        now = [200 + 60 * step, 90 + 37 * step]
        lg.copy_(ints(now))
        qn = rnd((2, 8, 64), 25 + step, torch.bfloat16)
        qg.copy_(qn)
        g, out, l2 = graphs[step % 2]
        out.zero_()
        g.replay()
        assert fa.fa_check_device_errors(None) == 0
        check(out, l2, qn, kc, vc, table, now, cu)


def test_sequences_that_share_pages(fa):
    """Two sequences with a common prefix in the same pages, and one twice in the batch."""
    lens, q_lens = [100, 80, 100], [3, 1, 2]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 64, 16, torch.float16, 50)
    table[1, :4] = table[0, :4]
    table[2] = table[0]
    q = rnd((cu[-1], 4, 64), 51, torch.float16)
    o, lse = run(fa, q, kc, vc, table, lens, cu)
    check(o, lse, q, kc, vc, table, lens, cu)


@pytest.mark.parametrize("q_len", [1, 150])
def test_two_streams_at_once(fa, q_len):
    """Calls on two streams, back to back and unsynchronised, each with its stream's scratch."""
    lens, q_lens = [5000, 900], [q_len, q_len]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 128, 64, torch.bfloat16, 52)
    kcg, vcg = on_gpu(kc, vc)
    args = (kcg, vcg, ints(table), ints(lens), ints(cu), q_len, 5000)
    qs = [rnd((cu[-1], 8, 128), 53 + i, torch.bfloat16) for i in range(2)]
    qg = [x.cuda() for x in qs]
    want = [fa.forward_paged(x, *args) for x in qg]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        got += [(i, fa.forward_paged(qg[i], *args, stream=streams[i])) for i in range(2)]
    torch.cuda.synchronize()
    assert fa.fa_check_device_errors(None) == 0
    for i, (o, lse) in got:
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
    check(want[0][0], want[0][1], qs[0], kc, vc, table, lens, cu)


@pytest.mark.parametrize("q_len", [1, 40])
def test_threads_that_share_a_stream(fa, q_len):
    """Four threads' calls on one stream, which share its scratch."""
    lens, q_lens = [5000, 900], [q_len, 1]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 64, 64, torch.float16, 72)
    kcg, vcg = on_gpu(kc, vc)
    args = (kcg, vcg, ints(table), ints(lens), ints(cu), q_len, 5000)
    qs = [rnd((cu[-1], 8, 64), 73 + i, torch.float16).cuda() for i in range(4)]
    want = [fa.forward_paged(x, *args) for x in qs]
    got = [[] for _ in qs]

    def work(i):
        for _ in range(100):
            got[i].append(fa.forward_paged(qs[i], *args))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert fa.fa_check_device_errors(None) == 0
    for w, g in zip(want, got):
        assert len(g) == 100 and all(torch.equal(o, w[0]) and torch.equal(lse, w[1]) for o, lse in g)


def test_captured_step_replayed(fa):
    """Append and attention captured as one graph; lengths, positions and rows change between replays."""
    H, hk, D, page = 8, 2, 128, 16
    lens, cu = [300, 60, 1], [0, 1, 2, 3]
    kc, vc, table, _ = paged_setup([n + 40 for n in lens], [1, 1, 1], hk, D, page, torch.bfloat16, 60)
    kcg, vcg = on_gpu(kc, vc)
    x = torch.empty(3, H + 2 * hk, D, dtype=torch.bfloat16, device="cuda")
    tg, lg, cg, inv = ints(table), ints(lens), ints(cu), fa.rope_inv_freq(D)[0]
    steps = fa.rope_steps(inv)

    def step():
        q = fa.paged_append(x[:, H:H + hk], x[:, H + hk:], kcg, vcg, tg, lg, cg, 1, q=x[:, :H], steps=steps)
        return q, *fa.forward_paged(q, kcg, vcg, tg, lg, cg, 1, 340)

    x.copy_(rnd(x.shape, 61, torch.bfloat16))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, o, lse = step()
    for i in range(1, 5):
        now = [n + i for n in lens]
        lg.copy_(ints(now))
        x.copy_(rnd(x.shape, 61 + i, torch.bfloat16))
        g.replay()
        assert fa.fa_check_device_errors(None) == 0
        check(o, lse, q.cpu(), kcg.cpu(), vcg.cpu(), table, now, cu)
        pos = torch.tensor([n - 1 for n in now], dtype=torch.int32, device="cuda")
        qr, kr = fa.rope(x[:, :H], x[:, H:H + hk], pos, steps)
        assert torch.equal(q, qr)
        at = torch.cat([paged.slots(table[b], [now[b] - 1], page) for b in range(3)])
        assert torch.equal(kcg.view(-1, hk, D)[at.cuda()], kr)
        assert torch.equal(vcg.view(-1, hk, D)[at.cuda()], x[:, H + hk:])


def test_prefill_in_chunks_then_decode_matches_the_packed_forward(fa):
    """The operators together: rotate and append a chunk, attend, chunk after chunk and token by token; every
    step's rows agree with the packed causal forward on the whole rotated sequences."""
    H, hk, D, page = 8, 2, 64, 32
    S = [330, 200]
    inv, mag = fa.rope_inv_freq(D, scaling="base", factor=2.0)
    steps = fa.rope_steps(inv)
    x = [rnd((n, H + 2 * hk, D), 30 + i, torch.bfloat16).cuda() for i, n in enumerate(S)]
    full = torch.cat(x)
    pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in S]).cuda()
    qr, kr = fa.rope(full[:, :H], full[:, H:H + hk], pos, steps)
    cu_full = ints([0, S[0], sum(S)])
    o_full, l_full = fa.forward_varlen(qr, kr, full[:, H + hk:].contiguous(), cu_full, max(S), causal=True)
    pages = [-(-n // page) for n in S]
    order = torch.randperm(sum(pages) + 1, generator=torch.Generator().manual_seed(33))
    table = torch.zeros(2, max(pages), dtype=torch.int32)
    table[0, :pages[0]] = order[:pages[0]]
    table[1, :pages[1]] = order[pages[0]:sum(pages)]
    tg = table.cuda()
    kc = torch.full((sum(pages) + 1, page, hk, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, float("nan"))
    done = [0, 0]
    for take in ([150, 1], [100, 120], [1, 0], [70, 70], [1, 1], [1, 1], [7, 7]):
        take = [min(t, n - d) for t, n, d in zip(take, S, done)]
        new = torch.cat([x[b][done[b]:done[b] + take[b]] for b in range(2)])
        done = [d + t for d, t in zip(done, take)]
        cu, lens = ints([0, take[0], sum(take)]), ints(done)
        q = fa.paged_append(new[:, H:H + hk], new[:, H + hk:], kc, vc, tg, lens, cu, max(take), q=new[:, :H],
                            steps=steps)
        o, lse = fa.forward_paged(q, kc, vc, tg, lens, cu, max(take), max(S))
        assert fa.fa_check_device_errors(None) == 0
        at = torch.cat([torch.arange(done[b] - take[b], done[b]) + (0, S[0])[b] for b in range(2)]).cuda()
        assert torch.equal(q, qr[at])
        # Both sides round P and O to 16 bits: twice 2 u W + u |O| of values below 4
        assert float((o.float() - o_full[at].float()).abs().max()) <= 2 * 3 * 2.0 ** -8 * 4
        assert float((lse - l_full[:, at]).abs().max()) <= 2e-5
    assert done == S


def test_wrapper_refuses(fa):
    q = torch.zeros(2, 4, 64, dtype=torch.float16, device="cuda")
    kc = torch.zeros(3, 16, 2, 64, dtype=torch.float16, device="cuda")
    ok = dict(q=q, k_cache=kc, v_cache=kc, block_table=ints([[0], [1]]), kv_lens=ints([3, 4]), cu_seqlens=ints([0, 1, 2]),
              max_seqlen_q=1, max_seqlen_k=16)
    fa.forward_paged(**ok)
    for k, x in (("q", q.float()), ("q", q[:, :3]), ("q", q.transpose(0, 1)), ("k_cache", kc[..., :32]),
                 ("k_cache", kc.bfloat16()), ("block_table", ints([[0]])), ("block_table", ints([[0], [1]]).long()),
                 ("kv_lens", ints([3])), ("cu_seqlens", ints([0, 1])), ("out", q[:1]), ("lse", torch.zeros(2, 4).cuda()),
                 ("out", torch.zeros(2, 4, 64).half())):
        with pytest.raises((ValueError, TypeError)):
            fa.forward_paged(**{**ok, k: x})
    for k, x in (("max_seqlen_k", 1 << 30), ("workspace", torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(fa.FAError):
            fa.forward_paged(**{**ok, k: x})
    assert fa.fa_check_device_errors(None) == 0
