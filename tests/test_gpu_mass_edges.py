"""Masses at the edges of what the calls allow, against the definition in 64 bits: blocks that rows do not fill."""
import pytest
import torch

from .eviction_common import Cache, check_mass, lse_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,group", [(150, 5), (130, 9), (300, 1), (100, 37), (7, 100), (3, 127), (385, 3)])
@pytest.mark.parametrize("d", [64, 128])
def test_blocks_of_rows_that_end_inside_a_warp(n, group, d):
    """Many blocks: some lanes have a row and others none, in every block or in the last."""
    c = Cache([n, n + 300, n + 1000], 2, d, 16, seed=n + d)
    pool = c.pool()
    q = c.randn(3, n, 2 * group, d)
    lse = lse_of(c, q, 0.08, True)
    old = c.mass()
    got = pool.prefill_mass(q, lse, old, decay=0.5, scale=0.08, out=torch.zeros_like(old))
    assert pool.check_errors() == 0
    check_mass(c, q, lse, 0.08, True, 0.5, old, got)
