"""The oracle of modified scores: gradients against differences, limits against the plain oracle, and the bounds of
the GPU tests against planted mistakes; and the refusals of the library's entry points.  No GPU."""
import ctypes
import math

import pytest
import torch

import exact_attention_18_gb300 as fa
import oracle
from exact_attention_18_gb300 import build as fab
from oracle import modified
from tests.score_bounds import backward_bounds, forward_bounds

F64 = torch.float64


def rnd(shape, seed, dtype=F64):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64).to(dtype)


def one(n=11, D=4, softcap=1.5, slope=0.2, causal=True, prefix=4, window=(6, 0), seed=0):
    q, k, v, do = (rnd((n, D), seed + i) for i in range(4))
    at = torch.arange(n)
    args = (modified.visible(n, causal, window, prefix), at, at, 0.7, softcap, slope)
    return q, k, v, do, args


@pytest.mark.parametrize("softcap,slope", [(1.5, 0.2), (None, -0.3), (0.4, None)])
@pytest.mark.parametrize("causal,prefix,window", [(True, 4, (6, 0)), (False, 0, None), (False, 0, (2, 3))])
def test_gradients_against_differences(softcap, slope, causal, prefix, window):
    q, k, v, do, args = one(softcap=softcap, slope=slope, causal=causal, prefix=prefix, window=window)
    r = modified.head(q, k, v, *args, do=do)
    loss = lambda a, b, c: float((modified.head(a, b, c, *args)["o"] * do).sum())  # noqa: E731
    h = 1e-5
    for name, which in (("dq", 0), ("dk", 1), ("dv", 2)):
        x = [q, k, v]
        for seed in range(3):
            d = rnd(q.shape, 50 + seed)
            up, dn = list(x), list(x)
            up[which], dn[which] = x[which] + h * d, x[which] - h * d
            diff = (loss(*up) - loss(*dn)) / (2 * h)
            # central differences: h^2 times a third derivative of order 10, and 2^-52 / h of rounding
            assert abs(diff - float((r[name] * d).sum())) < 1e-7


def test_plain_limits():
    """No cap, no bias: the plain oracle; a huge cap: nearly so."""
    n, D = 30, 8
    q, k, v, do = (rnd((1, 2, n, D), i) for i in range(4))
    seen, at = modified.visible(n, True), torch.arange(n)
    o, lse = oracle.forward(q, k, v, True, 0.3)
    g = oracle.backward(q, k, v, do, True, 0.3)
    for h in range(2):
        r = modified.head(q[0, h], k[0, h], v[0, h], seen, at, at, 0.3, None, None, do[0, h])
        far = modified.head(q[0, h], k[0, h], v[0, h], seen, at, at, 0.3, 1e9, None)
        for a, b in ((r["o"], o[0, h]), (r["lse"], lse[0, h]), (r["dq"], g[0][0, h]), (r["dk"], g[1][0, h]),
                     (r["dv"], g[2][0, h]), (far["o"], o[0, h])):
            assert float((a - b).abs().max()) < 1e-12


def test_visible():
    v = modified.visible(6, True, (2, 0), 3)
    assert v.tolist() == [[j >= i - 2 and (j <= i or j < 3) for j in range(6)] for i in range(6)]
    assert modified.visible(4, False).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_bounds_find_planted_mistakes(dtype):
    """A 16-bit emulation stays inside the bounds; one key too many, a bias or cap a little off, or a missing
    derivative do not."""
    n, D, cap, slope, scale = 120, 32, 6.0, 0.1, 0.3
    q, k, v, do = (rnd((n, D), i).to(dtype) for i in range(4))
    at = torch.arange(n)
    seen = modified.visible(n, True)
    r = modified.head(q, k, v, seen, at, at, scale, cap, slope, do)
    tol_o, tol_l, _ = forward_bounds(r, q, k, v, scale, cap, dtype)
    tq, tk, tv = backward_bounds(r, q, k, v, do, scale, cap, dtype)
    u = torch.finfo(dtype).eps / 2
    kf, qf, vf, df = (x.double() for x in (k, q, v, do))
    w = torch.exp(r["s"] - r["s"].amax(1, keepdim=True))
    o = ((w.to(dtype).double() @ vf) / w.sum(1, keepdim=True)).to(dtype).double()
    assert bool(((o - r["o"]).abs() <= tol_o).all())
    ds = (r["p"] * (r["dp"] - (df * o).sum(1, keepdim=True)) * r["f"]).to(dtype).double()
    for got, ref, tol in ((scale * ds @ kf, r["dq"], tq), (scale * ds.T @ qf, r["dk"], tk),
                          (r["p"].to(dtype).double().T @ df, r["dv"], tv)):
        assert bool(((got.to(dtype).double() - ref).abs() <= tol + u * ref.abs() + 2.0 ** -25).all())
    more = seen | modified.visible(n, False, (-1, 1))
    for wrong in ((more, at, at, scale, cap, slope), (seen, at, at, scale, cap * 1.2, slope),
                  (seen, at, at, scale, cap, slope * 1.1), (seen, at, at + (at > 60), scale, cap, slope * 2),
                  (seen, at, at, scale, None, slope)):
        bad = modified.head(q, k, v, *wrong)
        assert not bool(((bad["o"] - r["o"]).abs() <= tol_o).all())
        assert not bool(((bad["lse"] - r["lse"]).abs() <= tol_l).all())
    flat = r["p"] * r["g"]
    assert not bool(((scale * flat @ kf - r["dq"]).abs() <= tq).all())
    assert not bool(((scale * flat.T @ qf - r["dk"]).abs() <= tk).all())


# ----------------------------------------------------------------------- refusals
P = 0x10000  # a fake aligned address: never dereferenced by these calls


@pytest.fixture(scope="module")
def lib():
    fab.build_library()
    return fa.load_library()


def fwd(scores, D=64, scale=0.125, B=1, H=4, hk=2, S=8, q=P, packed=False):
    s = None if scores is None else ctypes.byref(scores)
    if packed:
        return fa.fa_fwd_scores_varlen(q, P, P, P, P, P, 2, S, 2 * S, H, hk, D, True, -1, -1, s, scale, fa.FA_BF16, None)
    return fa.fa_fwd_scores(q, P, P, P, P, B, H, hk, S, D, True, -1, -1, s, scale, fa.FA_BF16, None)


def bwd(scores, D=64, scale=0.125, ws=P, ws_bytes=1 << 30, packed=False):
    s = None if scores is None else ctypes.byref(scores)
    if packed:
        return fa.fa_bwd_scores_varlen(*[P] * 9, P, 2, 8, 16, 4, 2, D, True, -1, -1, s, scale, fa.FA_BF16, ws, ws_bytes, None)
    return fa.fa_bwd_scores(*[P] * 9, 1, 4, 2, 8, D, True, -1, -1, s, scale, fa.FA_BF16, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("packed", [False, True])
def test_refusals(lib, call, packed):
    invalid, unsupported, alignment = 1, 2, 3
    assert call(fa.Scores(-1.0, None, None), packed=packed) == invalid
    assert call(fa.Scores(math.nan, None, None), packed=packed) == invalid
    assert call(fa.Scores(math.inf, None, None), packed=packed) == invalid
    assert call(fa.Scores(1e-12, None, None), packed=packed) == unsupported
    assert call(fa.Scores(1e12, None, None), packed=packed) == unsupported
    assert call(fa.Scores(1e-9, None, None), scale=3e38, packed=packed) == unsupported
    assert call(fa.Scores(0.0, P + 2, None), packed=packed) == alignment
    assert call(fa.Scores(0.0, None, P + 1), packed=packed) == alignment
    assert call(fa.Scores(5.0, P, None), D=48, packed=packed) == unsupported
    assert call(fa.Scores(5.0, P, None), scale=math.inf, packed=packed) == invalid


def test_workspace_and_pointers(lib):
    s = fa.Scores(5.0, P, P)
    assert bwd(s, ws=None) == 4 and bwd(s, ws_bytes=16) == 4
    assert fwd(s, q=None) == 1 and fwd(s, q=P + 8) == 3
    assert fwd(s, H=4, hk=3) == 1


def cache_of(page_size=16):
    return fa.PagedCache(P, P, P, P, 4, 4, 64, page_size, page_size * 128, 128, 64)


def paged_call(scores=None, tree=True, positions=P, rows=P, stride=2, words=2, max_q=40, total=80, D=64, ws=None):
    c, s = cache_of(), None if scores is None else ctypes.byref(scores)
    if tree:
        return fa.fa_fwd_paged_tree(P, P, P, ctypes.byref(c), P, positions, rows, stride, words, 2, max_q, 64, total, 4,
                                    2, D, -1, s, 0.125, fa.FA_BF16, ws, 0, None)
    return fa.fa_fwd_paged_scores(P, P, P, ctypes.byref(c), P, 2, max_q, 64, total, 4, 2, D, True, -1, -1, s, 0.125,
                                  fa.FA_BF16, ws, 0, None)


def test_paged_refusals(lib):
    """Bad trees and scores are refused before the workspace is looked at (4: it is missing)."""
    assert paged_call() == 4 and paged_call(fa.Scores(3.0, P, None), tree=False) == 4
    assert paged_call(words=1) == 1 and paged_call(stride=1) == 1 and paged_call(words=0, stride=0) == 1
    assert paged_call(words=1, max_q=32) == 4 and paged_call(words=1, max_q=400, total=30) == 4
    assert paged_call(positions=None) == 1 and paged_call(rows=None) == 1
    assert paged_call(positions=P + 2) == 3 and paged_call(rows=P + 1) == 3
    assert paged_call(stride=1 << 31) == 2 and paged_call(D=96) == 2
    for tree in (True, False):
        assert paged_call(fa.Scores(0.0, None, P), tree=tree) == 2
        assert paged_call(fa.Scores(-3.0, None, None), tree=tree) == 1
        assert paged_call(fa.Scores(0.0, P + 1, None), tree=tree) == 3


def keep_call(cache=None, path=P, lens=P, stride=4, cols=4, batch=2, max_q=8, hk=2, D=64, dtype=None, cu=P):
    c = cache_of() if cache is None else cache
    return fa.fa_paged_keep(ctypes.byref(c), cu, path, stride, cols, lens, batch, max_q, hk, D,
                            fa.FA_BF16 if dtype is None else dtype, None)


def test_keep_refusals(lib):
    assert keep_call(path=None) == 1 and keep_call(lens=None) == 1 and keep_call(cu=None) == 1
    assert keep_call(path=P + 1) == 3 and keep_call(lens=P + 2) == 3
    assert keep_call(stride=3) == 1 and keep_call(cols=-1) == 1 and keep_call(batch=-1) == 1 and keep_call(max_q=-1) == 1
    assert keep_call(cache_of(page_size=24)) == 2 and keep_call(D=40) == 2 and keep_call(dtype=7) == 1
    assert keep_call(batch=1 << 31) == 2 and keep_call(cols=1 << 31, stride=1 << 31) == 2 and keep_call(hk=1 << 20) == 2
    assert keep_call(batch=0) == 0 and keep_call(cols=0, path=None) == 0 and keep_call(max_q=0) == 0 and keep_call(hk=0) == 0


def test_empty_calls(lib):
    s = fa.Scores(5.0, P, P)
    assert fwd(s, S=0) == 0 and fwd(s, B=0) == 0
    assert fwd(fa.Scores(-1.0, None, None), S=0) == 1  # (arguments are looked at first)
