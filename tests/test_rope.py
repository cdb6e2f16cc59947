"""Rotary positions, their gradient and the append to a paged cache on the GPU, against the fp64 oracle.

Tolerance of a rotated element m (a cos t -+ b sin t): the angle's fraction of
a turn is exact up to its rounding to 24 bits (at most pi 2^-25 radians),
sincospif is good to 2 units in the last place, and two products and a sum
round at 2^-24 each, so the fp32 value is off by less than m (|a| + |b|) 2^-21;
the stored one by half a step of its type more (and 2^-25, half of fp16's
subnormal step).
"""
import pytest
import torch

from oracle import paged, rope
from oracle.attention import as_f64

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def fa():
    import exact_attention_18_gb300 as m
    m.load_library()
    return m


def rnd(shape, seed, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def assert_rotated(name, got, x, ref, mag):
    """got (16-bit, GPU) against ref = rotate(x)."""
    g, x = got.detach().cpu().to(torch.float64), as_f64(x)
    u = torch.finfo(got.dtype).eps / 2
    pair = x.abs().amax(-1, keepdim=True) * 2  # |a| + |b| at most
    tol = u * ref.abs() + abs(mag) * pair * 2.0 ** -21 + 2.0 ** -25
    d = (g - ref).abs()
    assert bool((d <= tol).all()), f"{name}: worst error {float((d / tol).max()):.2f} of its bound"


def projection(T, H, hk, D, dtype, seed):
    """q, k, v as slices of one [T, H + 2 hk, D] projection."""
    x = rnd((T, H + 2 * hk, D), seed, dtype)
    g = x.cuda()
    cut = lambda y: (y[:, :H], y[:, H:H + hk], y[:, H + hk:])  # noqa: E731
    return cut(x), cut(g)


CASES = [  # T, H, H_kv, D, rot
    (1, 1, 1, 16, 16), (7, 3, 1, 16, 2), (513, 4, 2, 32, 32), (33, 6, 3, 32, 18), (257, 16, 2, 64, 64),
    (100, 5, 5, 64, 20), (64, 9, 3, 64, 22), (129, 32, 4, 128, 128), (50, 8, 1, 128, 64), (31, 3, 3, 128, 96),
    (17, 40, 8, 128, 126), (3, 200, 1, 128, 128),
]


@pytest.mark.parametrize("T,H,hk,D,rot", CASES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_rope_and_gradient(fa, T, H, hk, D, rot, inter, dtype):
    (q, k, _), (qg, kg, _) = projection(T, H, hk, D, DT[dtype], T + D)
    inv, mag = fa.rope_inv_freq(rot, scaling="parts", factor=4.0, original_len=512.0)
    pos = torch.randint(0, 100000, (T,), generator=torch.Generator().manual_seed(T))
    steps, posg = fa.rope_steps(inv), pos.to(torch.int32).cuda()
    for back, f in ((False, fa.rope), (True, fa.rope_backward)):
        qo, ko = f(qg, kg, posg, steps, interleaved=inter, magnitude=mag)
        for name, got, x in (("q", qo, q), ("k", ko, k)):
            ref = rope.rotate(x, pos, inv, inter, mag, back)
            assert_rotated(f"{name} back={back}", got, x, ref, mag)
            assert torch.equal(got[..., rot:].cpu(), x[..., rot:])  # columns past the rotated part
    torch.cuda.synchronize()
    assert torch.equal(qg.cpu(), q) and torch.equal(kg.cpu(), k)


@pytest.mark.parametrize("rot", [64, 22])
@pytest.mark.parametrize("inter", [False, True])
def test_in_place_gives_the_same_bits(fa, rot, inter):
    _, (q, k, _) = projection(100, 8, 2, 64, torch.bfloat16, 3)
    steps = fa.rope_steps(fa.rope_inv_freq(rot)[0])
    pos = torch.arange(100, dtype=torch.int32, device="cuda")
    qo, ko = fa.rope(q, k, pos, steps, interleaved=inter)
    q1, k1 = fa.rope(q, k, pos, steps, interleaved=inter, q_out=q, k_out=k)
    assert q1.data_ptr() == q.data_ptr() and torch.equal(q, qo) and torch.equal(k, ko)


def test_far_and_negative_positions(fa):
    """Angles stay exact where a 32-bit product of position and frequency has lost whole radians."""
    pos = torch.tensor([0, -1, -100000, 1 << 20, (1 << 31) - 1, -(1 << 31)])
    (q, k, _), (qg, kg, _) = projection(6, 2, 1, 64, torch.float16, 4)
    inv = fa.rope_inv_freq(64)[0]
    qo, ko = fa.rope(qg, kg, pos.to(torch.int32).cuda(), fa.rope_steps(inv))
    # 2^31 positions of a frequency rounded to 53 bits: both sides' angles are off by up to
    # 2^31 2^-53 2 radians more, 2^-21 each
    for got, x in ((qo, q), (ko, k)):
        ref = rope.rotate(x, pos, inv)
        tol = 2.0 ** -11 * ref.abs() + 2 * as_f64(x).abs().amax(-1, keepdim=True) * 2.0 ** -19 + 2.0 ** -25
        assert bool(((got.cpu().double() - ref).abs() <= tol).all())


def test_gradient_against_differences(fa):
    """The loss sum(rope(x) * g) is linear in x: its difference quotient is the gradient, whatever the step."""
    T, H, D = 5, 2, 32
    x, g = rnd((T, H, D), 5, torch.float16), rnd((T, H, D), 6, torch.float16)
    inv, pos = fa.rope_inv_freq(24)[0], torch.arange(T) * 1000
    steps, posg = fa.rope_steps(inv), pos.to(torch.int32).cuda()
    none = torch.zeros(T, 1, D, dtype=torch.float16, device="cuda")
    dx, _ = fa.rope_backward(g.cuda(), none, posg, steps)
    loss = lambda y: float((rope.rotate(y, pos, inv) * as_f64(g)).sum())  # noqa: E731
    base = as_f64(x)
    for t, h, c in ((0, 0, 3), (1, 1, 20), (4, 0, 23), (4, 1, 30)):
        e = torch.zeros_like(base)
        e[t, h, c] = 0.5
        quotient = loss(base + e) - loss(base - e)
        assert abs(quotient - float(dx[t, h, c])) <= 2.0 ** -11 * abs(quotient) + 2.0 ** -18


def test_special_values_stay_in_their_pairs(fa):
    x = torch.ones(2, 1, 16, dtype=torch.bfloat16)
    x[0, 0, 1], x[1, 0, 9], x[1, 0, 15] = float("nan"), float("inf"), float("-inf")
    steps = fa.rope_steps(fa.rope_inv_freq(8)[0])
    y, _ = fa.rope(x.cuda(), x.cuda(), torch.tensor([3, 4], dtype=torch.int32, device="cuda"), steps)
    bad = (~torch.isfinite(y.cpu().float())).nonzero().tolist()
    assert bad == [[0, 0, 1], [0, 0, 5], [1, 0, 9], [1, 0, 15]]


# ----------------------------------------------------------------------- append
def paged_setup(lens, q_lens, hk, D, page, dtype, seed, hnd=False, shared=False, spare=2):
    """Random caches, a shuffled block table whose unused entries are out of range, lengths and cu_seqlens."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    shape = (pages, hk, page, D) if hnd else (pages, page, hk, D)
    if shared:  # K and V interleaved in one pool
        pool = torch.randn(pages, 2, page, hk, D, generator=g).to(dtype)
        kc, vc = pool[:, 0], pool[:, 1]
    else:
        kc, vc = (torch.randn(*shape, generator=g).to(dtype) for _ in range(2))
        if hnd:
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    order = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), max(max(need), 1) + 1), -7, dtype=torch.int32)
    table[:, -1] = 1 << 30
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    cu = [0]
    for n in q_lens:
        cu.append(cu[-1] + n)
    return kc, vc, table, cu


def on_gpu(kc, vc):
    """The caches on the GPU with the same strides."""
    def move(x):
        y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
        return y.copy_(x)
    return move(kc), move(vc)


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


APPENDS = [  # cache lengths with the new tokens, new tokens, H, H_kv, D, page, rot, inter
    ([5], [5], 2, 1, 64, 16, 64, False),
    ([1, 17, 300], [1, 1, 1], 8, 2, 128, 16, 128, False),
    ([40, 0, 33, 129], [40, 0, 20, 1], 6, 3, 32, 32, 20, True),
    ([1000, 513], [700, 500], 4, 4, 64, 64, 64, True),
    ([77, 78, 79], [2, 3, 4], 3, 1, 16, 256, 2, False),
]


@pytest.mark.parametrize("lens,q_lens,H,hk,D,page,rot,inter", APPENDS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("form", ["nhd", "hnd", "pool"])
def test_append(fa, lens, q_lens, H, hk, D, page, rot, inter, dtype, form):
    dt = DT[dtype]
    kc, vc, table, cu = paged_setup(lens, q_lens, hk, D, page, dt, sum(lens), hnd=form == "hnd", shared=form == "pool")
    T = cu[-1] + 3  # three rows no sequence covers
    (q, k, v), (qg, kg, vg) = projection(T, H, hk, D, dt, T)
    kcg, vcg = on_gpu(kc, vc) if form != "pool" else (None, None)
    if form == "pool":
        pool = torch.stack((kc, vc), 1).cuda()
        kcg, vcg = pool[:, 0], pool[:, 1]
    inv, mag = fa.rope_inv_freq(rot, scaling="linear", factor=3.0)
    q_out = torch.full((T, H, D), 7.0, dtype=dt, device="cuda")
    fa.paged_append(kg, vg, kcg, vcg, ints(table), ints(lens), ints(cu), max(q_lens), q=qg, steps=fa.rope_steps(inv),
                    interleaved=inter, magnitude=1.25, q_out=q_out)
    assert fa.fa_check_device_errors(None) == 0
    pos = torch.cat([torch.arange(n - m, n) for n, m in zip(lens, q_lens)])
    n = cu[-1]
    assert_rotated("q", q_out[:n], q[:n], rope.rotate(q[:n], pos, inv, inter, 1.25), 1.25)
    assert bool((q_out[n:] == 7).all())  # rows behind the last sequence
    # V and every slot without a new token are bitwise what they were
    assert torch.equal(vcg.cpu().contiguous(), paged.append(vc.contiguous(), v, table, lens, cu))
    mark = paged.append(torch.zeros_like(kc).contiguous(), torch.ones_like(k), table, lens, cu).bool()
    assert torch.equal(kcg.cpu()[~mark], kc[~mark])
    got = torch.cat([kcg.cpu().reshape(-1, hk, D)[paged.slots(table[b], torch.arange(lens[b] - m, lens[b]), page)]
                     for b, m in enumerate(q_lens)])
    assert_rotated("k", got, k[:n], rope.rotate(k[:n], pos, inv, inter, 1.25), 1.25)


def test_append_positions_and_no_rotation(fa):
    """Positions of their own; without a table K and Q are copied as they are, and Q may be left out."""
    lens, q_lens = [20, 50], [3, 40]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 64, 16, torch.bfloat16, 8)
    (q, k, v), (qg, kg, vg) = projection(43, 4, 2, 64, torch.bfloat16, 9)
    args = (ints(table), ints(lens), ints(cu), 40)
    kcg, vcg = on_gpu(kc, vc)
    qo = fa.paged_append(kg, vg, kcg, vcg, *args, q=qg)
    assert torch.equal(qo.cpu(), q)
    assert torch.equal(kcg.cpu(), paged.append(kc, k, table, lens, cu))
    assert torch.equal(vcg.cpu(), paged.append(vc, v, table, lens, cu))
    kc2, vc2 = on_gpu(kc, vc)
    assert fa.paged_append(kg, vg, kc2, vc2, *args) is None
    assert torch.equal(kc2, kcg) and torch.equal(vc2, vcg)
    inv = fa.rope_inv_freq(64)[0]
    pos = torch.arange(43) * 17 - 100
    qo = fa.paged_append(kg, vg, kc2, vc2, *args, q=qg, steps=fa.rope_steps(inv), positions=ints(pos))
    qr, kr = fa.rope(qg, kg, ints(pos), fa.rope_steps(inv))
    assert torch.equal(qo, qr)
    assert torch.equal(kc2.cpu(), paged.append(kc, kr.cpu(), table, lens, cu))


def test_append_loosest_bound(fa):
    """The largest bound on the new tokens there is: nothing but the tokens themselves sizes the launch."""
    lens, q_lens = [20, 50], [3, 40]
    kc, vc, table, cu = paged_setup(lens, q_lens, 2, 64, 16, torch.bfloat16, 12)
    (_, k, v), (_, kg, vg) = projection(43, 4, 2, 64, torch.bfloat16, 13)
    kcg, vcg = on_gpu(kc, vc)
    fa.paged_append(kg, vg, kcg, vcg, ints(table), ints(lens), ints(cu), (1 << 31) - 1)
    assert fa.fa_check_device_errors(None) == 0
    assert torch.equal(kcg.cpu(), paged.append(kc, k, table, lens, cu))
    assert torch.equal(vcg.cpu(), paged.append(vc, v, table, lens, cu))


def test_append_reports_bad_pages_and_lengths(fa):
    """A bad entry's tokens, or a sequence whose length is below its new tokens, are left out and reported."""
    lens, q_lens = [20, 18, 5], [20, 2, 5]
    kc, vc, table, cu = paged_setup(lens, q_lens, 1, 32, 16, torch.float16, 10)
    (_, k, v), (_, kg, vg) = projection(27, 1, 1, 32, torch.float16, 11)
    bad = table.clone()
    bad[0, 1] = kc.shape[0]           # tokens 16..19 of the first sequence
    kcg, vcg = on_gpu(kc, vc)
    fa.paged_append(kg, vg, kcg, vcg, ints(bad), ints([20, 18, 4]), ints(cu), 20)  # third: 4 < 5 new tokens
    assert fa.STATUS[fa.fa_check_device_errors(None)] == "FA_ERR_INVALID_ARG"
    want = kc.clone()
    flat = want.view(-1, 1, 32)
    flat[paged.slots(table[0], torch.arange(16), 16)] = k[:16]
    flat[paged.slots(table[1], torch.arange(16, 18), 16)] = k[20:22]
    assert torch.equal(kcg.cpu(), want)
    fa.paged_append(kg, vg, kcg, vcg, ints(table), ints(lens), ints(cu), 20)
    assert fa.fa_check_device_errors(None) == 0


def test_wrappers_refuse(fa):
    q = torch.zeros(4, 2, 64, dtype=torch.float16, device="cuda")
    pos, steps = ints([0, 1, 2, 3]), fa.rope_steps(fa.rope_inv_freq(64)[0])
    for bad in ((q.float(), q, pos, steps), (q, q[:2], pos, steps), (q, q, pos.long(), steps),
                (q, q, pos[:3], steps), (q, q, pos, steps.int()), (q.transpose(0, 1), q, pos, steps),
                (q.cpu(), q, pos, steps), (q, q, pos.cpu(), steps)):
        with pytest.raises((ValueError, TypeError)):
            fa.rope(*bad)
    with pytest.raises(fa.FAError):  # more rotated columns than the head has
        fa.rope(q, q, pos, fa.rope_steps(fa.rope_inv_freq(128)[0]))
    kc = torch.zeros(3, 16, 2, 64, dtype=torch.float16, device="cuda")
    ok = dict(k_cache=kc, v_cache=kc.clone(), block_table=ints([[0, 1]]), kv_lens=ints([4]), cu_seqlens=ints([0, 4]),
              max_seqlen=4)
    fa.paged_append(q, q, **ok)
    for k, x in (("k_cache", kc.float()), ("v_cache", kc[:2]), ("block_table", ints([0, 1])),
                 ("block_table", ints([[0, 1], [1, 2]])), ("kv_lens", ints([4, 4])), ("kv_lens", ints([4]).long()),
                 ("cu_seqlens", ints([0, 4]).cpu()), ("v_cache", kc.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            fa.paged_append(q, q, **{**ok, k: x})
    assert fa.fa_check_device_errors(None) == 0
