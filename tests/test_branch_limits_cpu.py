"""Sizes at the edge of what one launch holds, and of nothing, in the operators that continue one prompt several
times (no GPU: no call here gets as far as a launch)."""

import pytest

from gated_delta_rule_82_amd import kda
from tests.test_attn_abi_cpu import call
from tests.test_branch_abi_cpu import FORK, SHARED

SHAPE, WORKSPACE = 2, 6


@pytest.fixture(scope="module")
def lib():
    return kda.load()


@pytest.mark.parametrize("B,Tq,H,HK,D,fits", [(1, 2 ** 24, 8, 1, 128, False), (1, 2 ** 24 - 1, 8, 1, 128, True), (4, 2 ** 22, 8, 1, 128, False),
                                              (1, 2 ** 25, 8, 1, 64, False), (1, 2 ** 25 - 64, 8, 1, 64, True), (1, 2 ** 24, 8, 1, 64, True)])
def test_rows_that_one_join_takes(lib, B, Tq, H, HK, D, fits):
    """The join of the parts is a second launch, of B Tq H D / 4 threads: below 2^32 of them, checked before the
    first launch."""
    size = dict(B=B, Tq=Tq, H=H, HK=HK, D=D, n_groups=0, max_pages=4, page=32)
    assert (lib.kda_attn_shared_workspace(B, Tq, H, HK, D, 0, 4 * 32) > 0) == fits
    assert call(lib.kda_attn_shared, SHARED, **size, ws_bytes=0) == (WORKSPACE if fits else SHAPE)


def test_a_fork_without_entries(lib):
    """Tables without pages, and no children: nothing to write, nothing to drop, no launch."""
    for K_in in (0, 1, 5):
        assert call(lib.kda_cache_fork, FORK, K_in=K_in, K_out=0, max_pages=0) == 0
