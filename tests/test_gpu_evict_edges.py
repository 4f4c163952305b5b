"""Selection and move at the edges of what the calls allow."""
import pytest
import torch

from cross_model_shared_gb300 import _native as N

from .eviction_common import Cache, check_selection
from .test_gpu_evict import draw_masses, drawn_index, select_pool, spare_table

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


@pytest.mark.parametrize("where", ["in place", "out"])
@pytest.mark.parametrize("aside", [False, True])
def test_a_token_that_is_not_copied_has_no_mass(where, aside):
    """Its slot still holds what was there before: a mass beside it would have the next selection keep that."""
    c = Cache([5000, 100], 2, 128, 16, seed=5, spare=330)
    keep = [4500, 40]
    index, new = drawn_index(c, keep, c.lens), spare_table(c, keep, c.lens)
    k0, v0 = c.k.clone(), c.v.clone()
    for bad in (-1, c.num, 2 ** 31 - 1, -2 ** 31):
        for which in ("source", "new"):
            c.k.copy_(k0), c.v.copy_(v0)
            pool = c.pool()
            table, to = c.table.cuda(), new.clone()
            lost = torch.zeros(2, 2, 4500, dtype=torch.bool, device="cuda")
            if which == "source":
                table[0, 2], table[0, 300], table[1, 1] = bad, bad, bad
                pool.block_table.copy_(table)
                for b, pages in ((0, (2, 300)), (1, (1,))):
                    for pg in pages:
                        lost[b, :, : keep[b]] |= index[b, :, : keep[b]] // 16 == pg
            else:
                to[0, 0], to[0, 281], to[1, 1] = bad, bad, bad
                lost[0, :, :16], lost[0, :, 281 * 16: 4500], lost[1, :, 16:32] = True, True, True
            old = torch.rand(2, 2, 5000, generator=c.g).cuda() + 0.5
            mass, out = old.clone(), torch.full_like(old, 7.0)
            pool.evict_tokens(index, keep, to, mass=mass, out=out if where == "out" else None,
                              source=(table, c.lens) if aside else None)
            assert pool.check_errors() == N.SHKV_ERRF_PAGE_OOB
            got = mass if where == "in place" else out
            for b, n in enumerate(keep):
                want = old[b].gather(1, index[b, :, :n].long()).masked_fill(lost[b, :, :n], 0.0)
                assert lost[b].any() and torch.equal(got[b, :, :n], want)
                assert not got[b, :, n: c.lens[b]].any()


def test_a_replay_that_moves_nobody_flags_requests_that_have_grown():
    c = Cache([300, 77], 2, 128, 16, seed=3)
    pool = c.pool(lens=[30, 0])
    index = torch.zeros(2, 2, 40, dtype=torch.int32, device="cuda")
    new = torch.full((2, 3), -1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.evict_tokens(index, [40, 40], new)
    g.replay()
    torch.cuda.synchronize()
    assert pool.check_errors() == 0
    table = pool.block_table.clone()
    for lens in ([200, 0], [30, 1], [29, 0]):
        pool.set_seq_lens(lens)
        g.replay()
        torch.cuda.synchronize()
        assert pool.check_errors() == N.SHKV_ERRF_SEQ_LEN, lens
        assert torch.equal(pool.block_table, table) and pool.seq_lens.tolist() == lens


def test_a_batch_of_empty_requests():
    pool = Cache([0, 0, 0], 2, 64, 16).pool()
    mass = torch.zeros(3, 2, 0, device="cuda")
    index = pool.select_tokens(mass, [4, 4, 4], sink=1, recent=2)
    assert index.shape == (3, 2, 1) and (index == -1).all()
    index = torch.full((3, 2, 5), 9, dtype=torch.int32, device="cuda")
    pool.select_tokens(mass, [4, 0, 4], out=index)
    assert (index == -1).all()
    pool.evict_tokens(index, [4, 0, 4], torch.zeros(3, 1, dtype=torch.int32, device="cuda"), mass=mass)
    assert pool.host_seq_lens().tolist() == [0, 0, 0] and pool.check_errors() == 0
