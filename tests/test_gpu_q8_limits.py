"""The 8-bit cache at the ends of what its documentation allows: the largest batch, in-place outputs, aliased pages."""
import numpy as np
import pytest
import torch

from .q8_common import Cache, attend, check, check_chunk, check_decode, dequantise, quantise

pytestmark = pytest.mark.gpu


def test_the_largest_batch():
    """1024 requests, a third of them without new tokens, some empty, through every operator."""
    B, hkv, hq, d, page = 1024, 2, 6, 64, 16
    g = torch.Generator().manual_seed(1)
    start = torch.randint(0, 40, (B,), generator=g).tolist()
    new = [n if n < 30 else 0 for n in torch.randint(0, 45, (B,), generator=g).tolist()]
    new[0], new[1], start[2], new[2] = 200, 90, 0, 0
    lens = [s + n for s, n in zip(start, new)]
    c = Cache(lens, hkv, d, page, seed=2)
    pool = c.pool(lens=start)
    T = sum(new)
    k, v = (torch.randn(T, hkv, d, generator=g).to(torch.bfloat16).cuda() for _ in "kv")
    pool.append_kv(k, v, new)
    assert pool.host_seq_lens().tolist() == lens == pool.seq_lens.tolist()
    got = pool.read_kv(start, new)
    for x, src in zip(got, (k, v)):
        codes, s = quantise(src.double().cpu().numpy())
        assert torch.equal(x.double().cpu(), dequantise(torch.from_numpy(codes), torch.from_numpy(s)))
    q = c.q(B, 2 * hq)
    out, lse = pool.decode_attention(q, 2, scale=0.05, return_lse=True)
    q2 = c.q(T, hq)
    out2, lse2 = pool.chunk_attention(q2, new, scale=0.05, return_lse=True)
    assert pool.check_errors() == 0
    check_decode(c, q, 2, 0.05, out, lse, requests=[*range(0, 12), *range(500, 510), *range(1014, 1024)])
    keep = [n if b < 12 or 500 <= b < 510 or b >= 1014 else 0 for b, n in enumerate(new)]
    rows = torch.tensor([bool(m) for m, n in zip(keep, new) for _ in range(n)], device="cuda")
    check_chunk(c, q2[rows], keep, 0.05, out2[rows], lse2[rows])


@pytest.mark.parametrize("new", [[4, 200], [64, 3]])
def test_outputs_over_the_queries(new):
    """`out` may be the queries' own memory: every row is read before its output is written."""
    c = Cache([9000, 3000], 2, 128, 16, seed=3)
    pool = c.pool()
    q = c.q(sum(new), 8)
    want, wl = pool.chunk_attention(q, new, scale=0.02, return_lse=True)
    x = q.clone()
    out, lse = pool.chunk_attention(x, new, scale=0.02, return_lse=True, out=x)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    q = c.q(2, 16)
    want = pool.decode_attention(q, 2, scale=0.02)
    x = q.clone()
    assert torch.equal(pool.decode_attention(x, 2, scale=0.02, out=x), want)
    assert pool.check_errors() == 0


def test_requests_that_share_their_pages():
    """A common prefix on the same pages, then pages of their own; one request maps a page twice."""
    c = Cache([320, 320, 320], 2, 128, 32, seed=4)
    c.table[1, :6] = c.table[0, :6]
    c.table[2, :6] = c.table[0, :6]
    c.table[2, 7] = c.table[2, 1]
    pool = c.pool()
    q = c.q(3, 16)
    out, lse = pool.decode_attention(q, 2, scale=0.02, return_lse=True)
    check_decode(c, q, 2, 0.02, out, lse)
    new = [100, 2, 70]
    q = c.q(sum(new), 8)
    out, lse = pool.chunk_attention(q, new, scale=0.02, return_lse=True)
    assert pool.check_errors() == 0
    check_chunk(c, q, new, 0.02, out, lse)


@pytest.mark.parametrize("head_dim,page", [(64, 32), (128, 16)])
def test_every_length_around_a_stage(head_dim, page):
    lens = [*range(1, 4), *range(15, 18), *range(31, 34), *range(126, 131), *range(254, 259), 383, 384, 385]
    c = Cache(lens, 1, head_dim, page, seed=5)
    pool = c.pool()
    q = c.q(len(lens), 9)
    out, lse = pool.decode_attention(q, 3, scale=0.05, return_lse=True)
    check_decode(c, q, 3, 0.05, out, lse)
    for new in ([1] * len(lens), lens, [min(n, 65) for n in lens], [max(1, n - 1) for n in lens]):
        q = c.q(sum(new), 3)
        out, lse = pool.chunk_attention(q, new, scale=0.05, return_lse=True)
        check_chunk(c, q, new, 0.05, out, lse)
    assert pool.check_errors() == 0


def test_values_at_the_top_of_bf16():
    """A row whose largest magnitude is 1.9375 * 2^127 or more rounds to 2^128 there, which bf16 reads back as an
    infinity; below that, and in the other elements, the format's rule holds as everywhere."""
    c = Cache([4], 1, 64, 16, seed=6)
    pool = c.pool(lens=[0])
    x = torch.zeros(4, 1, 64)
    x[0, 0, :3] = torch.tensor([1.9375, -1.0, 0.5]) * 2.0 ** 127
    x[1, 0, :3] = torch.tensor([1.9296875, -1.9296875, 0.5]) * 2.0 ** 127
    x[2, 0, :2] = torch.tensor([-1.9921875, 2.0 ** -8]) * 2.0 ** 127
    x[3, 0, 0] = 1.75 * 2.0 ** 127
    x = x.to(torch.bfloat16).cuda()
    pool.append_kv(x, x, [4])
    k, _ = pool.read_kv([0], [4])
    k = k[:, 0, :3].double().cpu() * 2.0 ** -127
    inf = float("inf")
    assert k.tolist() == [[inf, -1.0, 0.5], [1.875, -1.875, 0.5], [-inf, 2.0 ** -8, 0.0], [1.75, 0.0, 0.0]]
    assert pool.check_errors() == 0
