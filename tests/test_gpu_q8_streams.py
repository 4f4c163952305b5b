"""The 8-bit cache's calls on several streams: whose memory may be given back when."""
import pytest
import torch

from cross_model_shared_gb300 import _native as N

from .q8_common import Cache, check_decode, dequantise, quantise

pytestmark = pytest.mark.gpu


def test_inputs_of_another_stream_may_be_dropped_where_the_current_one_is_a_side_stream():
    """A call waits on the side stream that is current while its inputs are freed and their memory is asked for
    again elsewhere."""
    c = Cache([700, 90], 2, 128, 16, seed=46)
    pool = c.pool(lens=[690, 90])
    run = torch.cuda.Stream()
    q0 = c.q(2, 16)
    kv0 = torch.randn(2, 10, 2, 128, generator=c.g).to(torch.bfloat16).cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(run):                                     # kernels loaded, workspace made
        pool.append_kv(kv0[0], kv0[1], [10, 0], start=[690, 90])
        pool.decode_attention(q0, 2, return_lse=True)
    torch.full_like(q0, 7.0)
    pool.set_seq_lens([690, 90])
    q, k, v = q0.clone(), kv0[0].clone(), kv0[1].clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(run):
        torch.cuda._sleep(100_000_000)                               # some 50 ms
        pool.append_kv(k, v, [10, 0])
        out, lse = pool.decode_attention(q, 2, scale=0.05, return_lse=True)
    del q, k, v
    others = [torch.full_like(t, 7.0) for t in (q0, kv0[0], kv0[1]) for _ in range(3)]
    torch.cuda.synchronize()
    assert pool.check_errors() == 0
    del others
    got_k, got_v = pool.read_kv([690, 0], [10, 0])
    for got, src in ((got_k, kv0[0]), (got_v, kv0[1])):
        codes, sc = quantise(src.double().cpu().numpy())
        assert torch.equal(got.double().cpu(), dequantise(torch.from_numpy(codes), torch.from_numpy(sc)))
    check_decode(c, q0, 2, 0.05, out, lse)


def test_a_pool_may_be_dropped_while_a_call_on_a_side_stream_waits():
    """Its pages, scales, table and lengths are read and written to the end, though their memory is asked for again."""
    c = Cache([700, 90], 2, 128, 16, seed=47)
    q = c.q(2, 16)
    kv = torch.randn(2, 10, 2, 128, generator=c.g).to(torch.bfloat16).cuda()
    side = torch.cuda.Stream()
    warm = c.pool()
    with torch.cuda.stream(side):
        warm.decode_attention(q, 2, return_lse=True)
    torch.cuda.synchronize()
    for _ in range(2):
        pages = [t.clone() for t in (c.k, c.v, c.sc)]
        pool = c.pool.__func__(type("Own", (), dict(vars(c), k=pages[0], v=pages[1], sc=pages[2]))(), lens=[690, 90])
        del pages
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
            pool.append_kv(kv[0], kv[1], [10, 0])
            out, lse = pool.decode_attention(q, 2, scale=0.05, return_lse=True)
        del pool
        others = [torch.full_like(t, 7) for t in (c.k, c.v, c.sc) for _ in range(3)]
        others += [torch.full((2, c.table.shape[1]), 7, dtype=torch.int32, device="cuda") for _ in range(4)]
        others += [torch.full((n,), 7, dtype=torch.int32, device="cuda") for n in (1, 1, 2, 2)]
        torch.cuda.synchronize()
        k8, v8, sc = c.k.clone(), c.v.clone(), c.sc.clone()
        check_pool = c.pool(lens=[690, 90])
        check_pool.append_kv(kv[0], kv[1], [10, 0])
        check_decode(c, q, 2, 0.05, out, lse)
        assert all((t == 7).all() for t in others)                   # and nothing was written behind its back
        for t, was in ((c.k, k8), (c.v, v8), (c.sc, sc)):
            t.copy_(was)


def test_error_bits_of_another_stream_are_not_lost():
    """A side stream's calls set one bit while the current stream's checks read and clear another."""
    c = Cache([100, 100], 1, 64, 16, seed=48)
    pool = c.pool()
    q = c.q(2, 2)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        pool.decode_attention(q, 1)
    torch.cuda.synchronize()
    assert pool.check_errors() == 0
    good = pool.block_table.clone()
    lens = pool.seq_lens.clone()
    for spin in range(20):
        pool.block_table[1, 2] = -5                                  # PAGE_OOB on the current stream
        pool.decode_attention(q, 1)
        torch.cuda.synchronize()
        pool.block_table.copy_(good)
        pool.seq_lens.sub_(1)                                        # SEQ_LEN on the side stream
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(5_000 * spin)
            pool.decode_attention(q, 1)
        got = [pool.check_errors() for _ in range(3)]
        torch.cuda.synchronize()
        pool.seq_lens.copy_(lens)
        got.append(pool.check_errors())
        assert got[0] & N.SHKV_ERRF_PAGE_OOB and not any(g & N.SHKV_ERRF_PAGE_OOB for g in got[1:])
        assert any(g & N.SHKV_ERRF_SEQ_LEN for g in got)
        assert pool.check_errors() == 0


def test_calls_that_wait_are_refused_while_their_stream_is_captured():
    """... before they change anything: the lengths stay, and the capture goes on."""
    c = Cache([300, 77], 2, 128, 16, seed=49)
    pool = c.pool()
    q = c.q(2, 8)
    pool.decode_attention(q, 1, scale=0.05)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for f in (lambda: pool.set_seq_lens([5, 6]), pool.check_errors):
            with pytest.raises(N.ShkvError) as e:
                f()
            assert e.value.status == N.SHKV_ERR_INVALID_ARG
        out, lse = pool.decode_attention(q, 1, scale=0.05, return_lse=True)
    assert pool.host_seq_lens().tolist() == [300, 77]
    g.replay()
    torch.cuda.synchronize()
    assert pool.check_errors() == 0
    check_decode(c, q, 1, 0.05, out, lse)
