"""Pins for the rotary and paged-cache oracles, and the host helpers of the rotary entry points (no GPU)."""
import cmath
import ctypes
import math

import pytest
import torch

import exact_attention_18_gb300 as fa
import oracle
from exact_attention_18_gb300 import build as fab
from oracle import paged, rope

F64 = torch.float64


@pytest.fixture(scope="module", autouse=True)
def lib():
    fab.build_library()
    return fa.load_library()


def rnd(shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_complex_multiplication(inter):
    x, pos, f = rnd((3, 2, 8), 0), [0, 5, -7], [1.0, 0.25, 0.01]
    y = rope.rotate(x, pos, torch.tensor(f, dtype=F64), inter, 1.5)
    for t in range(3):
        for h in range(2):
            for i in range(3):
                a, b = (2 * i, 2 * i + 1) if inter else (i, 3 + i)
                z = complex(x[t, h, a], x[t, h, b]) * 1.5 * cmath.exp(1j * pos[t] * f[i])
                assert abs(z - complex(y[t, h, a], y[t, h, b])) < 1e-13
            assert torch.equal(y[t, h, 6:], x[t, h, 6:])


def test_rotation_scores_depend_on_distance_only():
    f, _ = rope.inv_freq(16)
    q, k = rnd((1, 1, 16), 1), rnd((1, 1, 16), 2)
    dots = [float((rope.rotate(q, [p + 9], f) * rope.rotate(k, [p], f)).sum()) for p in (0, 100, 4096)]
    assert max(dots) - min(dots) < 1e-10


def test_rotation_back_is_the_transpose():
    f, _ = rope.inv_freq(12)
    x, g = rnd((4, 2, 16), 3), rnd((4, 2, 16), 4)
    for inter in (False, True):
        lhs = (rope.rotate(x, range(4), f, inter, 1.3) * g).sum()
        rhs = (x * rope.rotate(g, range(4), f, inter, 1.3, back=True)).sum()
        assert abs(float(lhs - rhs)) < 1e-11


def test_paged_oracle_is_causal_attention_when_everything_is_new():
    B, S, H, hk, D, ps = 2, 21, 4, 2, 8, 16
    q, k, v = rnd((B * S, H, D), 5), rnd((B * S, hk, D), 6), rnd((B * S, hk, D), 7)
    table = torch.tensor([[3, 0], [2, 4]])
    cu, lens = [0, S, 2 * S], [S, S]
    empty = torch.full((5, ps, hk, D), float("nan"), dtype=F64)
    kc, vc = paged.append(empty, k, table, lens, cu), paged.append(empty, v, table, lens, cu)
    o, lse, _ = paged.attend(q, kc, vc, table, lens, cu, scale=0.3)
    o2, l2 = oracle.forward_varlen(q, k, v, torch.tensor(cu), True, 0.3)
    assert torch.allclose(o, o2, atol=1e-12) and torch.allclose(lse, l2, atol=1e-12)
    # the last two queries alone, over the same cache
    pick = [S - 2, S - 1, 2 * S - 2, 2 * S - 1]
    o3, l3, _ = paged.attend(q[pick], kc, vc, table, lens, [0, 2, 4], scale=0.3)
    assert torch.allclose(o3, o2[pick], atol=1e-12) and torch.allclose(l3, l2[:, pick], atol=1e-12)


def test_paged_oracle_window_and_empty_rows():
    q, k, v = rnd((3, 1, 4), 8), rnd((16, 1, 4), 9), rnd((16, 1, 4), 10)
    kc, vc = k.view(1, 16, 1, 4), v.view(1, 16, 1, 4)
    o, lse, _ = paged.attend(q, kc, vc, [[0]], [10], [0, 3], window=(0, 0))
    for i in range(3):  # a window of one key: its value
        assert torch.allclose(o[i, 0], v[7 + i, 0], atol=1e-13)
    o, lse, _ = paged.attend(q, kc, vc, [[0]], [1], [0, 3])  # queries at -2, -1, 0 over one key
    assert torch.equal(o[:2], torch.zeros(2, 1, 4, dtype=F64)) and torch.isinf(lse[0, :2]).all()
    assert torch.allclose(o[2, 0], v[0, 0], atol=1e-13)


@pytest.mark.parametrize("rot", [2, 6, 64, 128])
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "parts"])
def test_inverse_frequencies(rot, scaling):
    kw = dict(base=10000.0, factor=8.0, original_len=4096.0)
    f, mag = fa.rope_inv_freq(rot, scaling=scaling, **kw)
    ref, ref_mag = rope.inv_freq(rot, scaling=scaling, **kw)
    # powers and logarithms: a few roundings of 2^-53 each, the exponent at most ln(8e4) large
    assert torch.allclose(f, ref, rtol=1e-14, atol=0) and abs(mag - ref_mag) < 1e-7
    if scaling == "parts" and rot == 128:
        assert f[0] == 1.0 and abs(float(f[-1] / fa.rope_inv_freq(rot)[0][-1]) - 1 / 8) < 1e-14


@pytest.mark.parametrize("base,original_len", [(10000.0, 0.01), (10000.0, 1e15), (1.5, 4096.0)])
def test_ramp_beyond_every_pair(base, original_len):
    """Turns counted pair by pair: all below slow_turns are divided by the factor, all above fast_turns are kept."""
    rot, factor = 64, 8.0
    plain = fa.rope_inv_freq(rot, base)[0]
    turns = original_len * plain / (2 * math.pi)
    assert bool((turns < 1).all()) or bool((turns > 32).all())
    want = plain / factor if turns[0] < 1 else plain
    kw = dict(scaling="parts", factor=factor, original_len=original_len)
    assert torch.allclose(fa.rope_inv_freq(rot, base, **kw)[0], want, rtol=1e-14, atol=0)
    assert torch.allclose(rope.inv_freq(rot, base, **kw)[0], want, rtol=1e-14, atol=0)


def test_phase_steps_are_exact_fractions_of_a_turn():
    f = torch.tensor([2 * math.pi / 8, -2 * math.pi / 8, 0.0, 1.0, 2 * math.pi * 5.25], dtype=F64)
    steps = [int(x) % (1 << 64) for x in fa.rope_steps(f, device="cpu")]
    assert steps[2] == 0
    for got, turns in zip(steps, (1 / 8, 7 / 8, 0, 1 / (2 * math.pi), 0.25)):
        assert abs(got / 2 ** 64 - turns) < 2.0 ** -50
    # at a far position the step's angle agrees with a quotient of big integers
    inv = fa.rope_inv_freq(64)[0]
    two_pi = 6283185307179586476925286766559005768394338798750211642  # 2 pi 10^54
    for s, x in zip(fa.rope_steps(inv, device="cpu"), inv):
        n, d = float(x).as_integer_ratio()
        p = 2 ** 31 - 1
        turns = (p * n * 10 ** 54 * 2 ** 64 // (two_pi // 1 * d)) % 2 ** 64
        diff = (p * int(s) - turns) % 2 ** 64
        # the quotient x / 2 pi is rounded to 53 bits: 2^31 steps of it are off by at most x 2^31 2^-53 turns
        assert min(diff, 2 ** 64 - diff) / 2 ** 64 < 2.0 ** -22


def test_rope_host_helpers_refuse():
    for kw in (dict(rot_dim=3), dict(rot_dim=0), dict(base=0.0), dict(base=float("nan")),
               dict(scaling="linear", factor=0.0), dict(scaling="parts", factor=2.0),
               dict(scaling="parts", factor=2.0, original_len=10.0, fast_turns=1.0, slow_turns=1.0)):
        with pytest.raises(fa.FAError):
            fa.rope_inv_freq(**{"rot_dim": 8, **kw})
    with pytest.raises(ValueError):
        fa.rope_inv_freq(8, scaling="other")
    with pytest.raises(fa.FAError):
        fa.rope_steps(torch.tensor([float("inf")]), device="cpu")
    assert fa.fa_rope_inv_freq(8, 1e4, 9, 1, 1, 2, 1, None, None) == 1


P = 0x10000  # a fake, aligned address: never dereferenced by these calls


def _rope(**kw):
    a = dict(q=P, qs=512, k=P, ks=512, qo=P * 2, qos=256, ko=P * 2, kos=128, pos=P, steps=P, T=5, H=4, hk=2, D=64,
             rot=64, inter=0, mag=1.0, dtype=0)
    a.update(kw)
    args = (a["q"], a["qs"], a["k"], a["ks"], a["qo"], a["qos"], a["ko"], a["kos"], a["pos"], a["steps"], a["T"],
            a["H"], a["hk"], a["D"], a["rot"], a["inter"], a["mag"], a["dtype"], None)
    st = fa.fa_rope(*args)
    assert fa.fa_rope_bwd(*args) == st
    return st


@pytest.mark.parametrize("kw,status", [
    (dict(D=48), 2), (dict(dtype=3), 1), (dict(T=-1), 1), (dict(T=1 << 31), 2), (dict(H=-1), 1),
    (dict(q=0), 1), (dict(qo=P + 8), 3), (dict(qs=252), 3), (dict(qs=248), 1), (dict(kos=64), 1),
    (dict(pos=0), 1), (dict(pos=P + 2), 3), (dict(steps=0), 1), (dict(steps=P + 4), 3),
    (dict(rot=0), 1), (dict(rot=66), 1), (dict(rot=7), 1), (dict(mag=float("inf")), 1),
    (dict(qo=P), 1),
])
def test_rope_refuses(kw, status):
    assert _rope(**kw) == status
    assert fa.fa_last_error_detail() != ""


@pytest.mark.parametrize("kw", [dict(T=0, q=0, pos=0), dict(H=0, hk=0, q=0, k=0)])
def test_rope_empty(kw):
    assert _rope(**kw) == 0


def _cache(**kw):
    a = dict(k=P, v=P, block_table=P, kv_lens=P, table_stride=8, num_pages=10, page_size=16, page_stride=16 * 128,
             row_stride=128, head_stride=64)
    a.update(kw)
    return ctypes.byref(fa.PagedCache(**a))


CACHE_BAD = [
    (dict(k=0), 1), (dict(v=P + 8), 3), (dict(block_table=0), 1), (dict(kv_lens=P + 2), 3),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(num_pages=0), 1), (dict(table_stride=0), 1),
    (dict(table_pages=-1), 1), (dict(table_pages=9), 1),
    (dict(row_stride=0), 1), (dict(row_stride=132), 3), (dict(head_stride=32), 1),
    (dict(row_stride=64, head_stride=64), 1),          # rows of the two heads overlap
    (dict(page_stride=15 * 128), 1),                   # pages overlap
    (dict(page_stride=1 << 40), 2),
]


def _append(cache=None, **kw):
    a = dict(q=P, qs=256, qo=P * 2, qos=256, k=P, ks=128, v=P, vs=128, cu=P, pos=None, steps=P, B=2, ms=4, T=6, H=4,
             hk=2, D=64, rot=64, inter=0, mag=1.0, dtype=0)
    a.update(kw)
    return fa.fa_paged_append(a["q"], a["qs"], a["qo"], a["qos"], a["k"], a["ks"], a["v"], a["vs"],
                              _cache() if cache is None else cache, a["cu"], a["pos"], a["steps"], a["B"], a["ms"],
                              a["T"], a["H"], a["hk"], a["D"], a["rot"], a["inter"], a["mag"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=80), 2), (dict(dtype=5), 1), (dict(B=-1), 1), (dict(ms=-1), 1), (dict(T=-1), 1), (dict(hk=0), 1),
    (dict(q=0), 1), (dict(k=P + 8), 3), (dict(v=0), 1), (dict(ks=120), 1), (dict(vs=129), 3), (dict(cu=0), 1),
    (dict(cu=P + 2), 3), (dict(pos=P + 1), 3), (dict(steps=0), 1), (dict(rot=3), 1), (dict(rot=-2), 1),
    (dict(mag=float("nan")), 1), (dict(qo=P, qos=264), 1), (dict(ms=1 << 31), 2),
])
def test_append_refuses(kw, status):
    assert _append(**kw) == status
    assert fa.fa_last_error_detail() != ""


@pytest.mark.parametrize("kw,status", CACHE_BAD)
def test_append_and_attention_refuse_bad_caches(kw, status):
    assert _append(cache=_cache(**kw)) == status
    assert _attend(cache=_cache(**kw)) == status


def test_append_empty():
    for kw in (dict(B=0), dict(T=0, k=0), dict(ms=0), dict(H=0, hk=0)):
        assert _append(**kw) == 0


def _attend(cache=None, **kw):
    a = dict(q=P, o=P, lse=P, cu=P, B=2, mq=4, mk=100, T=6, H=4, hk=2, D=64, causal=1, wl=-1, wr=-1, scale=0.125,
             dtype=0, ws=P * 16, wsb=1 << 30)
    a.update(kw)
    return fa.fa_fwd_paged(a["q"], a["o"], a["lse"], _cache() if cache is None else cache, a["cu"], a["B"], a["mq"],
                           a["mk"], a["T"], a["H"], a["hk"], a["D"], a["causal"], a["wl"], a["wr"], a["scale"],
                           a["dtype"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), 2), (dict(dtype=2), 1), (dict(scale=float("inf")), 1), (dict(B=-1), 1), (dict(mq=-1), 1),
    (dict(mk=-1), 1), (dict(T=-1), 1), (dict(H=3), 1), (dict(hk=0), 1), (dict(H=258), 2),
    (dict(mk=1 << 30), 2), (dict(mq=1 << 30), 2), (dict(q=0), 1), (dict(o=P + 8), 3), (dict(lse=P + 4), 3),
    (dict(cu=0), 1), (dict(ws=0), 4), (dict(wsb=1000), 4), (dict(ws=P * 16 + 16), 3),
])
def test_paged_attention_refuses(kw, status):
    assert _attend(**kw) == status
    assert fa.fa_last_error_detail() != ""


def test_paged_attention_empty_and_workspace_size():
    for kw in (dict(B=0), dict(T=0, q=0), dict(mq=0), dict(H=0, hk=0)):
        assert _attend(**kw) == 0
    size = fa.fa_fwd_paged_workspace_size
    assert size(0, 1, 1, 1, 1, 64) == 0 and size(1, 1, 1, 3, 2, 64) == 0 and size(1, 1, 1, 1, 1, 48) == 0
    assert size(1, 1, 1, 129, 1, 64) == 0
    # one unit of at most 2 blocks: 2 CTAs, each with room for two partials of 16 rows
    assert size(1, 1, 100, 4, 4, 64) >= 4 * 16 * 65 * 4
    assert size(64, 1, 4096, 8, 1, 64) == size(640, 1, 4096, 8, 1, 64)  # bounded by the GPU, not the batch
