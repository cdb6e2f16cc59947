"""The error of capped scores that fa.h states: the tanh polynomial replayed in fp32 on the CPU, and single scores on
the GPU."""
import math
import os
import re

import numpy as np
import pytest
import torch

from tests.test_rope import ints
from tests.test_scores import rnd

F = np.float32
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "exact_attention_18_gb300", "csrc")
SCALES = [32 ** -0.5, 64 ** -0.5, 128 ** -0.5, 16 ** -0.5, 1.0, 0.037, 1e-3, 7.0, 1e4, -0.125]
CAPS = [50.0, 30.0, 20.0, 15.0, 5.0, 1.0, 0.01, 1e-4, 1e-10, 1000.0, 1e5, 1e10]


def fma(a, b, c):
    """fp32 a * b + c with one rounding: the product is exact in 64 bits, and the sum's rounding there is 2^-53."""
    return (a.astype(np.float64) * np.float64(b) + np.asarray(c, np.float64)).astype(F)


def coefficients():
    text = open(os.path.join(CSRC, "fa_api.cu")).read()
    values = re.search(r"kC\[fa::kTanhTerms\] = \{([^}]*)\}", text).group(1)
    return [float(x) for x in values.split(",")], float(re.search(r"constexpr double kMax = ([\d.]+);", text).group(1))


def folded(scale, cap):
    """The coefficients of x^(2k + 1) and the |x| up to which the polynomial is used (below 0: none)."""
    c, reach = coefficients()
    scale, cap = float(F(scale)), float(F(cap))
    into, poly, none = scale / cap, [], False
    for k, ck in enumerate(c):
        f = into ** (2 * k + 1) if abs(math.log10(abs(into))) * (2 * k + 1) < 300 else math.inf * (abs(into) > 1)
        size = abs(ck * f)
        none |= not size <= 1e37
        poly.append(F(ck * f) if size <= 1e37 else F(math.inf))
        if k > 0 and size < 1e-37:
            poly[-1] = F(0)
            reach = min(reach, (2.4e-7 / (2 * abs(ck))) ** (1 / (2 * k)))
    return poly, -1.0 if none else float(F(min(reach / abs(into), 1e18)))


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("scale", SCALES)
def test_polynomial(scale, cap):
    """tanh(scale x / cap) as the kernels' multiply-adds form it, up to where the polynomial is used: 2^-20 of itself."""
    poly, small = folded(scale, cap)
    if small < 0:
        pytest.skip("every score takes the exact form")
    g = np.random.default_rng(1)
    x = np.concatenate([np.linspace(small / 1e4, small, 40001), small * g.random(40000)]).astype(F)
    x = x[x <= F(small)]
    w = (x * x).astype(F)
    t = np.full_like(x, poly[-1])
    for c in poly[-2::-1]:
        t = fma(t, w, c)
    t = (t * x).astype(F)
    ref = np.tanh(np.float64(F(scale)) / np.float64(F(cap)) * x.astype(np.float64))
    assert float(np.abs(t / ref - 1).max()) < 2.0 ** -20


def test_reach_of_the_polynomial():
    """Usual calls: 1.25 of the cap, or 0.49 where the last coefficient, 5.8e-4 (scale / cap)^13, is below 1e-37: from
    cap / scale = 400 or so on (10^(33.8 / 13) = 396)."""
    for scale, cap, reach in ((32 ** -0.5, 20, 1.25), (64 ** -0.5, 30, 1.25), (128 ** -0.5, 15, 1.25),
                              (128 ** -0.5, 50, 0.49), (64 ** -0.5, 50, 0.49), (128 ** -0.5, 30, 1.25)):
        assert math.isclose(folded(scale, cap)[1] * scale / cap, reach, rel_tol=0.01), (scale, cap)


@pytest.fixture(scope="module")
def fa():
    import exact_attention_18_gb300 as m
    m.load_library()
    return m


# One key: L is its score.  m is the score rounded upwards (2^-23), L = (m + log2 l) ln 2 with l = 2^(score - m) takes
# three roundings more (2^-24 each) and an exponential and a logarithm of about 1 (2^-21 together).
OWN, FLAT = 2.0 ** -23 + 3 * 2.0 ** -24, 2.0 ** -21


def single(D, dtype):
    """q, k of one element each: their product is exact."""
    n = 4096
    a, b = torch.linspace(-8, 8, n).to(dtype), torch.linspace(0.5, 9.5, n).flip(0).to(dtype)
    q, k = torch.zeros(n, D, dtype=dtype), torch.zeros(n, D, dtype=dtype)
    at = torch.arange(n) % D
    q[torch.arange(n), at], k[torch.arange(n), at] = a, b
    return q, k, a.double() * b.double()


def check_single(lse, x, scale, cap, extra=0.0):
    v = float(F(scale)) / float(F(cap)) * x
    s = float(F(cap)) * torch.tanh(v)
    small = folded(scale, cap)[1]
    own = torch.where(x.abs() <= small, 2.0 ** -20 * s.abs(), torch.full_like(s, 2.0 ** -21 * cap))
    tol = own + OWN * s.abs() + FLAT + extra
    d = (lse.cpu().double() - s).abs()
    assert bool((d <= tol).all()), float((d / tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [16, 32, 64, 128])
@pytest.mark.parametrize("scale,cap", [(None, 50.0), (None, 5.0), (1.0, 20.0), (1.0, 50.0), (3.0, 30.0), (1e-3, 1e-2),
                                       (-0.7, 15.0)])
def test_single_scores(fa, scale, cap, D, dtype):
    """Whole sequences of one token, fixed and packed, and one key in a cache."""
    q, k, x = single(D, dtype)
    n, sc = len(q), D ** -0.5 if scale is None else scale
    kw = dict(softcap=cap, scale=sc)
    v = rnd((n, D), 1, dtype)
    g = [t.cuda() for t in (q, k, v)]
    o, lse = fa.forward(*(t[:, None, None] for t in g), causal=True, **kw)
    check_single(lse.view(-1), x, sc, cap)
    assert torch.equal(o.cpu()[:, 0, 0], v)
    o, lse = fa.forward_varlen(*(t[:, None] for t in g), ints(range(n + 1)), 1, **kw)
    check_single(lse[0], x, sc, cap)
    pages = [t[:, None, None].expand(n, 16, 1, D).contiguous() for t in g[1:]]
    o, lse = fa.forward_paged(g[0][:, None], *pages, torch.arange(n, dtype=torch.int32, device="cuda")[:, None],
                              ints([1] * n), ints(range(n + 1)), 1, 1, **kw)
    check_single(lse[0], x, sc, cap)
    assert fa.fa_check_device_errors(None) == 0
