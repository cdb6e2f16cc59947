"""Modified scores on whole sequences (fixed length and packed), forward and backward, on the GPU against the fp64
oracle; bounds in score_bounds.py."""
import math

import pytest
import torch

from oracle import modified
from tests.score_bounds import backward_bounds, forward_bounds

pytestmark = pytest.mark.gpu

DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def fa():
    import exact_attention_18_gb300 as m
    m.load_library()
    return m


def rnd(shape, seed, dtype, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype)


def alibi(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], dtype=torch.float32)


def inside(got, ref, tol, what):
    d = (got.detach().cpu().double() - ref).abs()
    assert bool((d <= tol).all()), f"{what}: worst error {float((d / tol).nan_to_num(nan=math.inf).max()):.2f} of its bound"


def check_sequence(q, k, v, do, o, lse, grads, causal, window, prefix, softcap, slopes, scale):
    """q, o, do [n, H, D], lse [H, n], grads of the same layouts: one sequence, all on the CPU."""
    n, H, D = q.shape
    hk, dt = k.shape[1], q.dtype
    G, u = H // hk, torch.finfo(dt).eps / 2
    at = torch.arange(n)
    seen = modified.visible(n, causal, window, prefix)
    rs = modified.sequence(q, k, v, seen, at, at, scale, softcap, slopes, do if grads is not None else None)
    sums = {}
    for h, r in enumerate(rs):
        kh, vh = k[:, h // G], v[:, h // G]
        tol_o, tol_l, _ = forward_bounds(r, q[:, h], kh, vh, scale, softcap, dt)
        inside(o[:, h], r["o"], tol_o, f"O h={h}")
        inside(lse[h], r["lse"], tol_l, f"L h={h}")
        if grads is None:
            continue
        bq, bk, bv = backward_bounds(r, q[:, h], kh, vh, do[:, h], scale, softcap, dt)
        sub = 2.0 ** -25 if dt == torch.float16 else 0.0
        inside(grads[0][:, h], r["dq"], bq + u * r["dq"].abs() + sub, f"dQ h={h}")
        for name, val, b in (("dK", r["dk"], bk), ("dV", r["dv"], bv)):
            s = sums.setdefault((name, h // G), [torch.zeros_like(val), torch.zeros_like(val)])
            s[0] += val
            s[1] += b
    for (name, g), (val, b) in sums.items():
        got = grads[1 if name == "dK" else 2][:, g]
        inside(got, val, b + u * val.abs() + (2.0 ** -25 if dt == torch.float16 else 0.0), f"{name} head {g}")


def fixed_case(fa, B, H, hk, S, D, dtype, causal=True, window=None, softcap=None, bias=False, prefix=None, gain=1.0,
               scale=None, backward=True, seed=0, slopes=None):
    dt = DT[dtype]
    std = math.sqrt(gain)
    q, k, v, do = (rnd((B, h, S, D), seed + 10 * S + i, dt, s)
                   for i, (h, s) in enumerate(((H, std), (hk, std), (hk, 1.0), (H, 1.0))))
    slopes = alibi(H) if bias and slopes is None else slopes
    pfx = None if prefix is None else torch.tensor([(prefix - 37 * b) for b in range(B)], dtype=torch.int32)
    kw = dict(causal=causal, window=window, softcap=softcap, scale=scale,
              slopes=None if slopes is None else slopes.cuda(), prefix=None if pfx is None else pfx.cuda())
    qg, kg, vg, dog = (x.cuda() for x in (q, k, v, do))
    o, lse = fa.forward(qg, kg, vg, **kw)
    grads = fa.backward(qg, kg, vg, o, dog, lse, **kw) if backward else None
    torch.cuda.synchronize()
    assert fa.fa_check_device_errors(None) == 0, fa.fa_last_error_detail()
    sc = 1 / math.sqrt(D) if scale is None else scale
    tr = lambda x: x.cpu().transpose(0, 1)  # noqa: E731
    for b in range(B):
        check_sequence(tr(q[b]), tr(k[b]), tr(v[b]), tr(do[b]), tr(o[b]), lse[b].cpu(),
                       None if grads is None else [tr(g[b]) for g in grads], causal, window,
                       0 if pfx is None else max(0, min(S, int(pfx[b]))), softcap, slopes, sc)
    return (qg, kg, vg, dog), kw, o, lse, grads


SHAPES = [(1, 2, 1, 1, 64), (2, 3, 1, 63, 32), (1, 2, 2, 65, 16), (1, 4, 2, 200, 128), (1, 3, 3, 513, 64),
          (1, 2, 1, 385, 128)]
MODS = {"cap": dict(softcap=5.0, gain=4.0), "bias": dict(bias=True), "both": dict(softcap=30.0, bias=True, gain=8.0)}


@pytest.mark.parametrize("mods", MODS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_causal(fa, shape, dtype, mods):
    fixed_case(fa, *shape, dtype, **MODS[mods])


@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("mods", MODS)
def test_whole(fa, D, mods):
    """Without a causal mask: distances to both sides."""
    fixed_case(fa, 1, 2, 1, 300, D, "fp16", causal=False, **MODS[mods])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("window", [(0, 0), (17, 0), (130, 65), (-1, 40), (40, -1)])
def test_windows(fa, D, window):
    fixed_case(fa, 1, 2, 1, 333, D, "bf16", causal=False, window=window, softcap=10.0, bias=True, gain=3.0)


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("prefix", [1, 64, 100, 129, 1000, -5])
def test_prefix(fa, D, prefix):
    """Rows before the prefix's end see behind themselves; lengths beyond the sequence count as its end."""
    fixed_case(fa, 2, 2, 1, 260, D, "fp16", prefix=prefix, bias=True, softcap=20.0, gain=2.0)


@pytest.mark.parametrize("D", [64, 128])
def test_prefix_window(fa, D):
    """The window's left side holds within the prefix."""
    fixed_case(fa, 1, 2, 2, 400, D, "bf16", prefix=150, window=(90, 0), bias=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gain,cap", [(0.01, 50.0), (30.0, 50.0), (300.0, 15.0), (1.0, 1e4), (100.0, 0.05)])
def test_reach_of_the_cap(fa, D, gain, cap):
    """Far below the cap, at it, far beyond it (the scores all +-cap), and a cap of no effect."""
    fixed_case(fa, 1, 2, 1, 257, D, "bf16", softcap=cap, gain=gain)


@pytest.mark.parametrize("scale", [0.0, -0.3, 0.7])
def test_scales(fa, scale):
    fixed_case(fa, 1, 2, 1, 150, 64, "fp16", softcap=4.0, bias=True, scale=scale)
    fixed_case(fa, 1, 2, 1, 150, 128, "fp16", softcap=4.0, scale=scale)


def test_slopes_of_any_sign(fa):
    """Negative slopes favour distance, 0 leaves a head alone."""
    fixed_case(fa, 1, 4, 2, 400, 64, "fp16", slopes=torch.tensor([-0.05, 0.0, 3.0, 0.125]))
    fixed_case(fa, 1, 4, 2, 200, 128, "bf16", causal=False, slopes=torch.tensor([-0.05, 0.0, 3.0, 0.125]))


def test_grouped_heads_split_over_ctas(fa):
    """Few K/V heads: the dK/dV pass splits a group, each query head with its own slope."""
    fixed_case(fa, 1, 12, 1, 300, 64, "fp16", softcap=8.0, bias=True, gain=2.0)
    fixed_case(fa, 1, 8, 2, 140, 128, "bf16", softcap=8.0, bias=True, gain=2.0)


PACKS = {"ragged": (17, 300, 1, 0, 130, 257), "one": (1,), "full": (128, 256, 64), "long": (700, 3)}


@pytest.mark.parametrize("D", [16, 64, 128])
@pytest.mark.parametrize("pack", PACKS)
@pytest.mark.parametrize("form", ["cap_prefix", "bias_window", "bias_whole"])
def test_packed(fa, D, pack, form):
    """Documents of a packed batch; what lies behind the last one holds NaN and is left as it was."""
    kw = {"cap_prefix": dict(causal=True, softcap=6.0), "bias_window": dict(causal=True, window=(100, 0)),
          "bias_whole": dict(causal=False)}[form]
    lens = PACKS[pack]
    dt, H, hk, extra = torch.bfloat16 if D == 64 else torch.float16, 4, 2, 70
    T = sum(lens) + extra
    q, k, v, do = (rnd((T, h, D), 7 * T + i, dt, 1.5) for i, h in enumerate((H, hk, hk, H)))
    for x in (q, k, v, do):
        x[sum(lens):] = float("nan")
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    slopes = alibi(H) if "bias" in form else None
    prefix = torch.tensor([n * 2 // 3 for n in lens], dtype=torch.int32) if form == "cap_prefix" else None
    dev = dict(slopes=None if slopes is None else slopes.cuda(), prefix=None if prefix is None else prefix.cuda())
    cug = torch.tensor(cu, dtype=torch.int32, device="cuda")
    qg, kg, vg, dog = (x.cuda() for x in (q, k, v, do))
    out = torch.full_like(qg, 3.0)
    lse_out = torch.full((H, T), 5.0, device="cuda")
    o, lse = fa.forward_varlen(qg, kg, vg, cug, max(lens) + 9, out=out, lse=lse_out, **kw, **dev)
    grads = fa.backward_varlen(qg, kg, vg, o, dog, lse, cug, max(lens) + 9, **kw, **dev)
    torch.cuda.synchronize()
    assert fa.fa_check_device_errors(None) == 0, fa.fa_last_error_detail()
    assert bool((o[cu[-1]:] == 3.0).all()) and bool((lse[:, cu[-1]:] == 5.0).all())
    for b, (a, e) in enumerate(zip(cu[:-1], cu[1:])):
        if a == e:
            continue
        check_sequence(q[a:e], k[a:e], v[a:e], do[a:e], o[a:e].cpu(), lse[:, a:e].cpu(), [g[a:e].cpu() for g in grads],
                       kw["causal"], kw.get("window"), 0 if prefix is None else int(prefix[b]), kw.get("softcap"),
                       slopes, 1 / math.sqrt(D))


def test_packed_window_alone(fa):
    """A window inside the samples of a packed batch, plain scores."""
    lens, D = (90, 201), 64
    q, k, v, do = (rnd((291, 2, D), i, torch.float16) for i in range(4))
    cu = torch.tensor([0, 90, 291], dtype=torch.int32, device="cuda")
    g = [x.cuda() for x in (q, k, v, do)]
    o, lse = fa.forward_varlen(*g[:3], cu, 201, causal=True, window=(33, 0))
    grads = fa.backward_varlen(*g[:3], o, g[3], lse, cu, 201, causal=True, window=(33, 0))
    torch.cuda.synchronize()
    for a, e in ((0, 90), (90, 291)):
        check_sequence(q[a:e], k[a:e], v[a:e], do[a:e], o[a:e].cpu(), lse[:, a:e].cpu(), [x[a:e].cpu() for x in grads],
                       True, (33, 0), 0, None, None, 1 / math.sqrt(D))


@pytest.mark.parametrize("t", [150, 151])
@pytest.mark.parametrize("D", [64, 128])
def test_hidden_keys_have_no_say(fa, D, t):
    """Rows before a changed key keep their bits, forward and backward, whatever the scores behind them."""
    (q, k, v, do), kw, o, lse, grads = fixed_case(fa, 1, 2, 1, 300, D, "fp16", softcap=9.0, bias=True, gain=3.0)
    k2, v2, do2 = k.clone(), v.clone(), do.clone()
    k2[:, :, t:], v2[:, :, t:] = k2[:, :, t:] * 50, -7.0
    o2, lse2 = fa.forward(q, k2, v2, **kw)
    assert torch.equal(o[:, :, :t], o2[:, :, :t]) and torch.equal(lse[:, :, :t], lse2[:, :, :t])
    g2 = fa.backward(q, k2, v2, o2, do, lse2, **kw)
    assert torch.equal(grads[0][:, :, :t], g2[0][:, :, :t])
    do2[:, :, t:] = 0
    g3 = fa.backward(q, k, v, o, do2, lse, **kw)
    assert not bool(g3[1][:, :, t:].any()) and not bool(g3[2][:, :, t:].any())


@pytest.mark.parametrize("D", [64, 128])
def test_nan_reaches_its_row(fa, D):
    q, k, v = (rnd((1, 2, 200, D), i, torch.bfloat16).cuda() for i in range(3))
    q[0, 1, 77, 3] = float("nan")
    o, lse = fa.forward(q, k, v, causal=True, softcap=10.0, slopes=alibi(2).cuda())
    assert bool(o[0, 1, 77].isnan().all()) and bool(lse[0, 1, 77].isnan())
    o[0, 1, 77] = 0
    assert not bool(o.isnan().any()) and int(lse.isnan().sum()) == 1


def test_repeats_and_streams(fa):
    """The same bits again, on another stream, and in a captured graph replayed beside it."""
    (q, k, v, do), kw, o, lse, grads = fixed_case(fa, 1, 4, 2, 700, 64, "fp16", softcap=9.0, bias=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, lse2 = fa.forward(q, k, v, stream=side, **kw)
    g2 = fa.backward(q, k, v, o2, do, lse2, stream=side, **kw)
    side.synchronize()
    for a, b in zip((o, lse, *grads), (o2, lse2, *g2)):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, lse3 = fa.forward(q, k, v, **kw)
        g3 = fa.backward(q, k, v, o3, do, lse3, **kw)
    for _ in range(3):
        for t in (o3, lse3, *g3):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((o, lse, *grads), (o3, lse3, *g3)):
            assert torch.equal(a, b)


def test_plain_scores_are_unchanged(fa):
    """Absent parts run the plain kernels: the same bits as without them."""
    q, k, v = (rnd((1, 2, 300, 64), i, torch.float16).cuda() for i in range(3))
    o, lse = fa.forward(q, k, v, causal=True, window=(50, 0))
    o2, lse2 = torch.empty_like(q), torch.empty_like(lse)
    import ctypes
    s = fa.Scores(0.0, None, None)
    assert fa.fa_fwd_scores(q.data_ptr(), k.data_ptr(), v.data_ptr(), o2.data_ptr(), lse2.data_ptr(), 1, 2, 2, 300, 64,
                            True, 50, 0, ctypes.byref(s), 1 / 8, fa.FA_FP16, torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_tensors_are_checked(fa):
    q, k, v = (rnd((1, 4, 40, 64), i, torch.float16).cuda() for i in range(3))
    for kw in (dict(slopes=torch.ones(3, device="cuda")), dict(slopes=torch.ones(4)),
               dict(slopes=torch.ones(4, device="cuda", dtype=torch.float64)),
               dict(slopes=torch.ones(8, device="cuda")[::2]), dict(prefix=torch.ones(2, device="cuda")),
               dict(prefix=torch.ones(1, dtype=torch.int64, device="cuda")), dict(softcap=0.0), dict(softcap=-1.0),
               dict(softcap=float("nan")), dict(softcap=1.0, out=torch.empty_like(q)[:, :, :20]),
               dict(softcap=1.0, lse=torch.empty(1, 4, 40, dtype=torch.float16, device="cuda"))):
        with pytest.raises(ValueError):
            fa.forward(q, k, v, **kw)
    with pytest.raises(fa.FAError):
        fa.forward(q, k, v, softcap=math.inf)


def test_three_dimensions_and_given_outputs(fa):
    """[B, S, D] tensors are one head; outputs given by the caller are filled."""
    q, k, v, do = (rnd((2, 1, 70, 64), i, torch.float16).cuda() for i in range(4))
    kw = dict(causal=True, softcap=5.0, slopes=torch.tensor([0.25], device="cuda"))
    o, lse = fa.forward(q, k, v, **kw)
    grads = fa.backward(q, k, v, o, do, lse, **kw)
    out, l3 = torch.empty_like(q[:, 0]), torch.empty(2, 70, device="cuda")
    o3, lse3 = fa.forward(*(x[:, 0].contiguous() for x in (q, k, v)), out=out, lse=l3, **kw)
    assert o3.data_ptr() == out.data_ptr() and torch.equal(o3, o[:, 0]) and torch.equal(lse3, lse[:, 0])
    given = [torch.empty_like(out) for _ in range(3)]
    g3 = fa.backward(*(x[:, 0].contiguous() for x in (q, k, v)), o3, do[:, 0].contiguous(), lse3, dq=given[0],
                     dk=given[1], dv=given[2], workspace=torch.empty(1 << 16, dtype=torch.uint8, device="cuda"), **kw)
    for a, b, g in zip(g3, grads, given):
        assert a.data_ptr() == g.data_ptr() and torch.equal(a, b[:, 0])
    with pytest.raises(fa.FAError):
        fa.backward(q, k, v, o, do, lse, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"), **kw)
    with pytest.raises(ValueError):
        fa.backward(q, k, v, o, do.half().expand(2, 1, 70, 64)[:, :, ::2], lse, **kw)
