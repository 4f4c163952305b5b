"""Selection and move at the edges of what the calls allow."""
import pytest
import torch

from .eviction_common import check_selection
from .test_gpu_evict import draw_masses, select_pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["uniform", "few values"])
@pytest.mark.parametrize("lens", [[33000, 40001], [131072, 20000, 65551], [393216]])
def test_clusters_whose_lanes_write_unequally_many(lens, kind):
    """A row's CTAs meet at its end while the lanes of a warp come from loops of different length, and from none."""
    pool = select_pool(lens, 2)
    mass = draw_masses(kind, len(lens), 2, max(lens), seed=len(lens))
    mass[:, 0, : max(lens) // 2] = -1.0      # warps that choose nothing at all
    for few in (1, 33, 1000, 16385):
        keep = [min(L - 1, few + 3) for L in lens]
        check_selection(mass, lens, keep, 2, 1, pool.select_tokens(mass, keep, sink=2, recent=1))
    assert pool.check_errors() == 0
