"""What follows a packed backward on its stream comes after all of its kernels, also where no CTA of its passes has
work: no sample has a token, or none has offsets that the call allows.  The kernel that sums dO . O runs over all tokens
of the batch all the same and writes the workspace; here it takes longer than starting the work behind it."""
import pytest
import torch

from tests.test_rope import ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import exact_attention_18_gb300 as m
    m.load_library()
    return m


@pytest.mark.parametrize("mods", [{}, dict(softcap=9.0)], ids=["plain", "capped"])
@pytest.mark.parametrize("cu,bad", [([0, 0, 0], False), ([0, 70000, 90000], True)], ids=["empty", "contradicting"])
def test_work_behind_a_backward_without_rows(fa, cu, bad, mods):
    T, H, D, bound = 100000, 32, 128, 500
    x = torch.zeros(T, H, D, dtype=torch.float16, device="cuda")
    do = torch.ones_like(x)
    lse = torch.zeros(H, T, device="cuda")
    size = fa.fa_bwd_varlen_workspace_size(2, bound, T, H, H, D)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    offs = ints(cu)
    for _ in range(5):
        fa.backward_varlen(x, x, x, do, do, lse, offs, bound, workspace=ws, **mods)
        ws.fill_(0xA5)
        do.fill_(1.0)
        torch.cuda.synchronize()
        assert bool((ws == 0xA5).all())
    status = fa.STATUS[fa.fa_check_device_errors(None)]
    assert status == ("FA_ERR_INVALID_ARG" if bad else "FA_OK")


def test_gradients_beside_empty_samples(fa):
    """Samples without a token, and ones shorter than the bound by many tiles, beside others: their gradients alone."""
    H, D = 2, 64
    g = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn(700, H, D, generator=g).half().cuda() for _ in range(4))
    for kw in ({}, dict(softcap=9.0)):
        o, lse = fa.forward_varlen(q, k, v, ints([0, 0, 650, 650, 700]), 650, causal=True, **kw)
        many = fa.backward_varlen(q, k, v, o, do, lse, ints([0, 0, 650, 650, 700]), 650, causal=True, **kw)
        for a, b in ((0, 650), (650, 700)):
            part = [x[a:b].contiguous() for x in (q, k, v, o, do)]
            alone = fa.backward_varlen(*part, lse[:, a:b].contiguous(), ints([0, b - a]), b - a, causal=True, **kw)
            for m, s in zip(many, alone):
                assert torch.equal(m[a:b], s)
    assert fa.fa_check_device_errors(None) == 0
