"""Masses at the edges of what the calls allow, against the definition in 64 bits."""
import pytest
import torch

from cross_model_shared_gb300 import SharedKVPool
from cross_model_shared_gb300 import _native as N

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


class Window:
    """Tokens [t0, t1) of a long cache as a request of their own, for check_mass."""

    def __init__(self, k, t0, t1):
        self.lens, self.hkv, self.k = [t1 - t0], 1, k.view(-1, k.shape[-1])[t0:t1]

    def rows(self, b):
        return self.k.double()[None]


def test_requests_whose_rows_times_tokens_pass_32_bits():
    """34 million tokens of one KV head: 64 stacked rows of a decode, and two new tokens of 128 heads."""
    d, P, L = 64, 32, 34_000_001
    pages = -(-L // P)
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.empty(pages, 1, P, d, dtype=torch.bfloat16, device="cuda")
    for i in range(0, pages, 1 << 17):
        k[i: i + (1 << 17)] = torch.randn(k[i: i + (1 << 17)].shape, generator=g, device="cuda", dtype=torch.bfloat16)
    pool = SharedKVPool(pages, P, 1, d, max_batch=1, max_pages_per_seq=pages, k_pages=k, v_pages=k, initial_seq_lens=[L])
    pool.block_table.copy_(torch.arange(pages, dtype=torch.int32)[None])
    windows = [(0, 300_000), (L // 3, L // 3 + 1000), (33_554_432 - 400_000, L)]
    windows += [(t, t + 1000) for t in (L - (1 << 25) - 500, L - (1 << 24) - 500, L // 2)]
    for n, hq, causal in ((8, 8, False), (1, 64, False), (2, 128, True), (1, 128, True)):
        q = torch.randn(1, n, hq, d, generator=g, device="cuda").to(torch.bfloat16)
        lse = torch.full((1, n, hq), 3.0, device="cuda")
        if causal:
            got = pool.prefill_mass(q, lse, None, scale=0.1)
        else:
            got = pool.decode_mass(q.view(1, n * hq, d), lse.view(1, -1), n, None, scale=0.1)
        assert pool.check_errors() == 0
        for t0, t1 in windows:
            check_mass(Window(k, t0, t1), q, lse, 0.1, causal and t1 == L, 1.0, None, got[:, :, t0:t1])


@pytest.mark.parametrize("n,group", [(1, 5), (2, 16), (7, 4), (40, 5), (64, 3), (300, 3), (150, 9)])
@pytest.mark.parametrize("what", ["nan", "inf", "inf key", "nan key"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_that_attend_nothing_add_nothing_whatever_they_hold(n, group, what, d):
    """An lse of -inf takes a row out, also where its scores are no number or infinite: an inactive decoder's queries
    may hold anything, and a key may be infinite."""
    c = Cache([n + 500, n + 77], 2, d, 16, seed=n + group)
    q = c.randn(2, n, 2 * group, d)
    q[..., 0] = -q[..., 0].abs() - 1         # an infinite key below is -inf to the rows that attend
    pool = c.pool()
    scale = 0.05
    lse = lse_of(c, q, scale, True)
    dead = torch.rand(2, n, 2 * group, generator=c.g).cuda() < 0.3
    dead[0, 0], dead[0, 0, 1] = True, False
    dead[1, :, group:] = True                # a KV head that nobody attends
    lse[dead] = -float("inf")
    if what in ("nan", "inf"):
        q[dead] = float(what)
    else:
        q[..., 0] = torch.where(dead, q[..., 0].abs(), q[..., 0])
        for b, t in ((0, 5), (0, n + 499), (1, 30)):
            row = c.k[int(c.table[b, t // 16]), :, t % 16]
            row[:] = 0
            row[:, 0] = float("inf")
            if what == "nan key":            # of a head whose rows are all out
                c.k[int(c.table[1, 1]), 1, 3] = float("nan")
    old = c.mass()
    for form in ("decode", "prefill"):
        if form == "decode":
            if n * group > 64:
                continue
            got = pool.decode_mass(q.view(2, -1, d), lse.view(2, -1), n, old, scale=scale, out=torch.zeros_like(old))
        else:
            got = pool.prefill_mass(q, lse, old, scale=scale, out=torch.zeros_like(old))
        assert pool.check_errors() == 0 and not torch.isnan(got).any()
        check_mass(c, q, lse, scale, form == "prefill", 1.0, old, got)
        assert torch.equal(got[1, 1, : c.lens[1]], old[1, 1, : c.lens[1]])


@pytest.mark.parametrize("n,group", [(2, 8), (60, 4), (300, 3)])
def test_a_row_of_an_infinite_sum_weighs_its_infinite_key_as_no_number(n, group):
    """An lse of +inf is that of a row with an infinite score: exp(inf - inf) there, 0 elsewhere."""
    c = Cache([n + 100], 1, 128, 16, seed=n)
    c.k[int(c.table[0, 0]), 0, 7] = 0
    c.k[int(c.table[0, 0]), 0, 7, 0] = float("inf")
    q = c.randn(1, n, group, 128)
    q[..., 0] = q[..., 0].abs() + 1
    pool = c.pool()
    lse = torch.full((1, n, group), float("inf"), device="cuda")
    lse[0, 0, 0] = -float("inf")
    nan = torch.isnan(pool.prefill_mass(q, lse, None, scale=0.05))
    assert nan[0, 0, 7] and int(nan.sum()) == 1


@pytest.mark.parametrize("lens", [[300, 0, 20], [0, 0, 0], [0, 300, 0]])
def test_a_replay_after_empty_requests_have_grown_is_flagged(lens):
    c = Cache([300, 300, 300], 2, 128, 16, seed=4)
    pool = c.pool(lens=lens)
    q, lse = c.randn(3, 8, 128), torch.full((3, 8), 4.0, device="cuda")
    mass = torch.zeros(3, 2, 300, device="cuda")
    pool.decode_mass(q, lse, 1, mass)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pool.decode_mass(q, lse, 1, mass)
    g.replay()
    torch.cuda.synchronize()
    assert pool.check_errors() == 0
    for b in range(3):
        pool.set_seq_lens([L + (1 if L < 300 else -1) * (i == b) for i, L in enumerate(lens)])
        g.replay()
        torch.cuda.synchronize()
        assert pool.check_errors() == N.SHKV_ERRF_SEQ_LEN, b


def test_a_batch_of_empty_requests():
    pool = Cache([0, 0, 0], 2, 64, 16).pool()
    q, lse = torch.zeros(3, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, 8, device="cuda")
    got = pool.decode_mass(q, lse, 2, None)
    assert got.shape == (3, 2, 0)
    assert pool.decode_mass(q, lse, 2, got) is got
    out = torch.full((3, 2, 5), 7.0, device="cuda")
    pool.decode_mass(q, lse, 2, got, out=out)
    assert (out == 7).all() and pool.check_errors() == 0


@pytest.mark.parametrize("T", [1, 5, 8])
@pytest.mark.parametrize("d", [64, 128])
def test_one_new_token_out_of_a_fused_projection(T, d):
    """q, k and v heads of a token side by side: the token stride is no multiple of its query heads'."""
    c = Cache([100, 450, 33], 8, d, 16, seed=T)
    pool = c.pool()
    qkv = c.randn(3, T, 48, d)
    q = qkv[:, -1:, :32]
    lse = lse_of(c, q, 0.07, True)
    fused = torch.zeros(3, T, 48, device="cuda")
    fused[:, -1:, :32] = lse
    got = pool.prefill_mass(q, fused[:, -1:, :32], None, scale=0.07)
    assert pool.check_errors() == 0
    check_mass(c, q, lse, 0.07, True, 1.0, None, got)
    assert torch.equal(pool.prefill_mass(q.contiguous(), lse, None, scale=0.07), got)
    one = pool.prefill_mass(q[:1], lse[:1], None, scale=0.07)
    check_mass(c, q[:1], lse[:1], 0.07, True, 1.0, None, one, requests=[0])
