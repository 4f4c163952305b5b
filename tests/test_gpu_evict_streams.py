"""Eviction's calls on several streams and in CUDA graphs."""
import pytest
import torch

from cross_model_shared_gb300 import _native as N

from .eviction_common import Cache, check_mass, check_selection, evicted, lse_of

pytestmark = pytest.mark.gpu

SOME_50_MS = 100_000_000


def test_inputs_may_be_dropped_on_a_side_stream():
    c = Cache([900, 300], 2, 128, 16, seed=1, spare=60)
    pool = c.pool()
    scale = 128 ** -0.5
    q0 = c.randn(2, 2, 8, 128)
    lse0 = lse_of(c, q0, scale, False)
    old = c.mass()
    keep = [400, 100]
    want_index = None
    for named in (False, True):
        pool.set_seq_lens(c.lens)
        pool.block_table.copy_(c.table)
        side = torch.cuda.Stream()
        q, lse, mass = q0.clone(), lse0.clone(), old.clone()
        new = torch.tensor(c.free[:25] + c.free[25:32] + [-1] * 18, dtype=torch.int32).view(2, 25).cuda()
        out = torch.zeros_like(old)
        torch.cuda.synchronize()
        kw = dict(stream=side) if named else {}
        with torch.cuda.stream(side):
            torch.cuda._sleep(SOME_50_MS)
        with (torch.cuda.stream(torch.cuda.default_stream()) if named else torch.cuda.stream(side)):
            pool.decode_mass(q.view(2, 16, 128), lse.view(2, 16), 2, mass, out=out, **kw)
            pool.prefill_mass(q, lse, mass, **kw)
            index = pool.select_tokens(out, keep, sink=4, recent=16, **kw)
            pool.evict_tokens(index, keep, new, mass=mass, **kw)
        del q, lse, mass, new
        others = [torch.full_like(t, 7.0) for t in (q0, lse0, old) for _ in range(3)]
        others += [torch.full((2, 25), 7, dtype=torch.int32, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert pool.check_errors() == 0 and all((t == 7).all() for t in others)
        check_mass(c, q0, lse0, scale, False, 1.0, old, out)
        check_selection(out, c.lens, keep, 4, 16, index)
        assert pool.seq_lens.tolist() == keep
        if want_index is None:
            want_index = index.clone()
        assert torch.equal(index, want_index)


def test_a_captured_session_replays():
    """Two graphs, each with the four calls on buffers of its own, replayed in turn and at once."""
    c = Cache([700, 260], 2, 128, 16, seed=2, spare=120)
    scale = 128 ** -0.5
    keep = [300, 100]
    pools = [c.pool() for _ in range(2)]
    table, lens = c.table.cuda(), list(c.lens)
    graphs, sets = [], []
    for i, pool in enumerate(pools):
        q = c.randn(2, 4, 8, 128)
        lse = lse_of(c, q, scale, True)
        mass, out, moved = c.mass(), c.mass(), c.mass()
        new = torch.full((2, 19), -1, dtype=torch.int32)
        new[0] = torch.tensor(c.free[40 * i: 40 * i + 19])
        new[1, :7] = torch.tensor(c.free[40 * i + 19: 40 * i + 26])
        new = new.cuda()
        index = torch.zeros(2, 2, 300, dtype=torch.int32, device="cuda")

        def calls():
            pool.prefill_mass(q, lse, mass, decay=0.5, out=out)
            pool.select_tokens(out, keep, sink=1, recent=8, out=index)
            pool.evict_tokens(index, keep, new, mass=out, out=moved, source=(table, lens))
            pool.set_seq_lens(lens) if not torch.cuda.is_current_stream_capturing() else None

        calls()                             # kernels loaded
        pool.block_table.copy_(table)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            calls()
        graphs.append(g)
        sets.append((pool, q, lse, mass, out, moved, new, index))
    for at_once in (False, True):
        for pool, q, lse, mass, out, moved, new, index in sets:
            pool.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
            pool.block_table.copy_(table)
            q.copy_(c.randn(2, 4, 8, 128))
            lse.copy_(lse_of(c, q, scale, True))
            mass.copy_(c.mass())
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                if at_once:
                    torch.cuda._sleep(1_000_000)
                g.replay()
            if not at_once:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        for pool, q, lse, mass, out, moved, new, index in sets:
            assert pool.check_errors() == 0
            check_mass(c, q, lse, scale, True, 0.5, mass, out)
            check_selection(out, lens, keep, 1, 8, index)
            k, v = evicted(c, index, keep, new, lens=lens, table=table)
            assert torch.equal(c.k, k) and torch.equal(c.v, v)
            assert pool.seq_lens.tolist() == keep
            for b, n in enumerate(keep):
                assert torch.equal(moved[b, :, :n], out[b].gather(1, index[b, :, :n].long()))


def test_a_replay_with_other_lengths_is_flagged():
    c = Cache([300, 77], 2, 128, 16, seed=3)
    pool = c.pool()
    q = c.randn(2, 8, 128)
    lse = lse_of(c, q.view(2, 1, 8, 128), 0.05, False).view(2, 8)
    mass = c.mass()
    pool.decode_mass(q, lse, 1, mass, scale=0.05)
    pool.select_tokens(mass, [100, 50])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.decode_mass(q, lse, 1, mass, scale=0.05)
        index = pool.select_tokens(mass, [100, 50])
    g.replay()
    torch.cuda.synchronize()
    assert pool.check_errors() == 0
    check_selection(mass, c.lens, [100, 50], 0, 0, index)
    pool.set_seq_lens([299, 77])
    g.replay()
    torch.cuda.synchronize()
    assert pool.check_errors() == N.SHKV_ERRF_SEQ_LEN
