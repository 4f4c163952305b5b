"""The 8-bit cache's calls on several streams: whose memory may be given back when."""
import pytest
import torch

from .q8_common import Cache, check_decode, dequantise, quantise

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("current", ["side", "default"])
def test_inputs_of_another_stream_may_be_dropped_where_the_calls_is_the_current_one(current):
    """A call on the current stream, a side stream or the default one, waits on it while its inputs, made on the
    other one, are freed and their memory is asked for again there."""
    c = Cache([700, 90], 2, 128, 16, seed=46)
    pool = c.pool(lens=[690, 90])
    side, main = torch.cuda.Stream(), torch.cuda.default_stream()
    run, make = (side, main) if current == "side" else (main, side)
    q0 = c.q(2, 16)
    kv0 = torch.randn(2, 10, 2, 128, generator=c.g).to(torch.bfloat16).cuda()
    torch.cuda.synchronize()
    with torch.cuda.stream(run):                                     # kernels loaded, workspace made
        pool.append_kv(kv0[0], kv0[1], [10, 0], start=[690, 90])
        pool.decode_attention(q0, 2, return_lse=True)
    torch.full_like(q0, 7.0)
    pool.set_seq_lens([690, 90])
    with torch.cuda.stream(make):
        q, k, v = q0.clone(), kv0[0].clone(), kv0[1].clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(run):
        torch.cuda._sleep(100_000_000)                               # some 50 ms
        pool.append_kv(k, v, [10, 0])
        out, lse = pool.decode_attention(q, 2, scale=0.05, return_lse=True)
    del q, k, v
    with torch.cuda.stream(make):
        others = [torch.full_like(t, 7.0) for t in (q0, kv0[0], kv0[1]) for _ in range(3)]
    torch.cuda.synchronize()
    assert pool.check_errors() == 0
    del others
    got_k, got_v = pool.read_kv([690, 0], [10, 0])
    for got, src in ((got_k, kv0[0]), (got_v, kv0[1])):
        codes, sc = quantise(src.double().cpu().numpy())
        assert torch.equal(got.double().cpu(), dequantise(torch.from_numpy(codes), torch.from_numpy(sc)))
    check_decode(c, q0, 2, 0.05, out, lse)
