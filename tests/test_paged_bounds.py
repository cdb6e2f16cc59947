"""Bounds and workspace sizes of attention over a paged cache (no GPU)."""
import random

import pytest

import exact_attention_18_gb300 as fa
from exact_attention_18_gb300 import build as fab
from tests.test_oracle_paged import _attend, _cache


@pytest.fixture(scope="module", autouse=True)
def lib():
    fab.build_library()
    return fa.load_library()


def test_workspace_of_the_largest_bounds():
    """Bounds that the interface allows have a workspace, of the size that the GPU gives, not the bounds."""
    size = fa.fa_fwd_paged_workspace_size
    big = size(64, 1 << 29, 131072, 32, 8, 64)
    assert 0 < big == size(64, 2000, 131072, 32, 8, 64)
    assert size(1 << 20, 1 << 29, 1 << 29, 128, 1, 128) > 0
    assert size(64, (1 << 29) + 1, 100, 32, 8, 64) == 0 and size(64, 100, (1 << 29) + 1, 32, 8, 64) == 0


def test_workspace_never_shrinks_with_looser_bounds():
    """A call plans with the tightest bounds it knows; the workspace was sized for the caller's."""
    rng, size = random.Random(5), fa.fa_fwd_paged_workspace_size
    for _ in range(20000):
        hk = rng.choice([1, 2, 3, 8])
        H, D = hk * rng.choice([1, 2, 3, 4, 5, 8, 16, 40, 64, 65, 128]), rng.choice([16, 32, 64, 128])
        batch = rng.choice([1, 2, 3, 17, 64, 300, 5000])
        mq, mk = int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(0, 20))
        lq, lk = mq + int(mq * rng.expovariate(1)), mk + int(mk * rng.expovariate(1))
        assert 0 < size(batch, mq, mk, H, hk, D) <= size(batch, lq, lk, H, hk, D), (batch, mq, mk, lq, lk, H, hk, D)
        assert size(batch, mq, mk, H, hk, D) <= size(batch, 1 << 29, 1 << 29, H, hk, D)


def test_refusal_is_by_what_the_call_can_hold():
    """Loose bounds alone refuse nothing (a workspace too small is found after the plan: status 4); a batch of more
    tiles than the library counts is refused whatever its workspace."""
    wide = _cache(table_stride=1 << 20, num_pages=1 << 20)
    assert _attend(B=64, mq=1 << 29, mk=1 << 29, T=64, wsb=0) == 4
    assert _attend(cache=wide, B=64, mq=1 << 29, mk=1 << 29, T=4096, wsb=0) == 4
    assert _attend(cache=wide, B=1 << 30, mq=1 << 29, mk=1 << 29, T=1 << 29, wsb=0) == 2
    assert _attend(cache=wide, B=1 << 24, mq=1, mk=1 << 29, T=1 << 24, wsb=0) == 2
