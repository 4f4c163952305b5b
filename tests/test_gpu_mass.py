"""Masses of a decode step and of a causal chunk against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from cross_model_shared_gb300 import _native as N

from .eviction_common import Cache, check_mass, lse_of

pytestmark = pytest.mark.gpu


def decode_case(c, n_models, hq, scale=None):
    scale = c.d ** -0.5 if scale is None else scale
    q = c.randn(len(c.lens), n_models, hq, c.d)
    lse = lse_of(c, q, scale, False)
    return q, lse, scale


def run_decode(pool, q, lse, mass, **kw):
    B, n, hq, d = q.shape
    return pool.decode_mass(q.view(B, n * hq, d), lse.view(B, n * hq), n, mass, **kw)


# lengths around a page's, a tile's and a pair of tiles' ends, empty requests among them
LENS = [[1], [256], [0, 15, 16, 17, 0], [127, 128, 129, 255], [256, 257, 31, 33, 600], [1, 3000, 0, 511, 513, 1024]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("d,page", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("n_models,hq,hkv", [(1, 1, 1), (2, 8, 2), (1, 14, 2), (3, 15, 3)])
def test_decode(lens, d, page, n_models, hq, hkv):
    c = Cache(lens, hkv, d, page, seed=len(lens) + d + hq)
    pool = c.pool()
    q, lse, scale = decode_case(c, n_models, hq)
    old = c.mass(extra=5)
    mass = old.clone()
    got = run_decode(pool, q, lse, mass)
    assert pool.check_errors() == 0 and got is mass
    check_mass(c, q, lse, scale, False, 1.0, old, mass)
    for b, L in enumerate(lens):
        assert torch.equal(mass[b, :, L:], old[b, :, L:])


@pytest.mark.parametrize("n_models,group", [(1, 8), (2, 4), (8, 1), (3, 5), (4, 4), (1, 17), (5, 5), (8, 4), (1, 33), (8, 5),
                                            (7, 7), (8, 8), (64, 1), (1, 64)])
@pytest.mark.parametrize("d", [64, 128])
def test_stacked_rows(n_models, group, d):
    c = Cache([700, 130, 2049], 2, d, 16, seed=n_models + group)
    pool = c.pool()
    q, lse, scale = decode_case(c, n_models, 2 * group)
    got = run_decode(pool, q, lse, None)
    assert pool.check_errors() == 0 and got.shape == (3, 2, 2049)
    check_mass(c, q, lse, scale, False, 1.0, None, got)
    for b, L in enumerate(c.lens):          # every row's weights add up to one
        assert torch.allclose(got[b, :, :L].double().sum(1), torch.full((2,), float(n_models * group), device="cuda",
                                                                        dtype=torch.float64), rtol=1e-4)
        assert not got[b, :, L:].any()


@pytest.mark.parametrize("decay", [0.0, 0.5, 1.0, -1.0, 0.97])
@pytest.mark.parametrize("where", ["in place", "out", "sums alone"])
def test_decay_and_destination(decay, where):
    c = Cache([300, 77, 0], 2, 128, 16, seed=3)
    pool = c.pool()
    q, lse, scale = decode_case(c, 2, 4)
    old = c.mass(extra=3)
    if decay == 0.0:
        old[:, :, ::3] = float("nan")       # not read
    mass = old.clone()
    out = {"in place": mass, "out": c.mass(extra=9), "sums alone": c.mass()}[where]
    before = out.clone()
    got = run_decode(pool, q, lse, None if where == "sums alone" else mass, decay=decay,
                     out=None if where == "in place" else out)
    assert got is out and pool.check_errors() == 0
    check_mass(c, q, lse, scale, False, decay, None if where == "sums alone" else old, out)
    for b, L in enumerate(c.lens):
        assert torch.equal(out[b, :, L:].nan_to_num(), before[b, :, L:].nan_to_num())
    if where == "out":
        assert torch.equal(mass.nan_to_num(), old.nan_to_num())


def test_masses_of_any_stride():
    c = Cache([300, 77, 129], 2, 64, 16, seed=4)
    pool = c.pool()
    q, lse, scale = decode_case(c, 1, 6)
    old = torch.rand(2, 4, 311, generator=c.g).cuda()[:, :, 1:].transpose(0, 1)      # heads outside, odd rows, a request more
    into = torch.full((3, 5, 2, 301), 7.0, device="cuda")[:, 2]
    got = run_decode(pool, q, lse, old, out=into)
    assert got is into
    check_mass(c, q, lse, scale, False, 1.0, old, into)
    one = torch.rand(1, 1, 300, generator=c.g).cuda().expand(3, 2, 300)              # the same masses for all
    check_mass(c, q, lse, scale, False, 1.0, one, run_decode(pool, q, lse, one, out=torch.zeros(3, 2, 300, device="cuda")))


def test_rows_that_attend_nothing_and_values_out_of_range():
    """An lse of -inf adds nothing; what lies behind a request's end, NaN or infinite, reaches nobody; weights
    of 2^-126 and less, and of rows whose lse is far above, vanish."""
    c = Cache([200, 40], 2, 128, 16, seed=5)
    for b, L in enumerate(c.lens):
        last = int(c.table[b, (L - 1) // 16])
        c.k[last, :, L % 16:] = float("nan")
    c.k[int(c.free[0])] = float("inf")
    pool = c.pool()
    q, lse, scale = decode_case(c, 3, 8)
    lse[0, 1] = -np.inf
    lse[1, 0, 3] = np.inf
    lse[1, 2] += 200.0
    got = run_decode(pool, q, lse, None)
    assert torch.isfinite(got[0, :, :200]).all() and torch.isfinite(got[1, :, :40]).all()
    lse_ref = lse.clone()
    check_mass(c, q, lse_ref, scale, False, 1.0, None, got)


def test_nan_and_infinities_reach_their_own_tokens_and_rows():
    c = Cache([300], 2, 128, 16, seed=6)
    at = (int(c.table[0, 150 // 16]), 1, 150 % 16)
    c.k[at] = float("nan")
    pool = c.pool()
    q = c.randn(1, 2, 8, 128)
    lse = torch.full((1, 2, 8), 3.0, device="cuda")
    got = run_decode(pool, q, lse, None)
    nan = torch.isnan(got)
    assert nan[0, 1, 150] and int(nan.sum()) == 1
    q[0, 1, 2] = float("nan")               # a row of head 0
    nan = torch.isnan(run_decode(pool, q, lse, None))
    assert nan[0, 0].all() and int(nan.sum()) == 301
    lse[0, 0, 5] = float("nan")             # and one of head 1
    assert torch.isnan(run_decode(pool, q, lse, None)).all()


@pytest.mark.parametrize("n,group", [(1, 3), (1, 17), (7, 1), (40, 5), (100, 5), (300, 3), (300, 9)])
@pytest.mark.parametrize("d", [64, 128])
def test_infinite_keys_meet_the_rows_that_there_are(n, group, d):
    """A key whose product with every row is -inf gets 0: the zeros that fill up a block of rows would give NaN."""
    c = Cache([700, 333], 1, d, 16, seed=n + group)
    for b, t in ((0, 5), (0, 399), (1, 30)):
        row = c.k[int(c.table[b, t // 16]), 0, t % 16]
        row.zero_()
        row[0] = float("inf")
    pool = c.pool()
    q = c.randn(2, n, group, d)
    q[..., 0] = -q[..., 0].abs() - 1
    lse = torch.zeros(2, n, group, device="cuda")
    for f in (lambda: run_decode(pool, q, lse, None, scale=0.01), lambda: pool.prefill_mass(q, lse, None, scale=0.01)):
        if n * group > 64 and "run_decode" in f.__code__.co_names:
            continue
        got = f()
        assert pool.check_errors() == 0 and not torch.isnan(got).any()
        assert got[0, 0, 5] == 0 and got[0, 0, 399] == 0 and got[1, 0, 30] == 0 and int((got[0, 0, :400] == 0).sum()) == 2


@pytest.mark.parametrize("lens,n,hq,hkv", [([900, 2000], 700, 10, 2), ([256, 300], 256, 4, 1), ([3000], 64, 8, 2)])
def test_prefill_in_place(lens, n, hq, hkv):
    """Also where an item's blocks are shared out and joined by the second kernel."""
    c = Cache(lens, hkv, 128, 16, seed=n)
    pool = c.pool()
    q = c.randn(len(lens), n, hq, 128)
    lse = lse_of(c, q, 0.05, True)
    old = c.mass(extra=7)
    mass = old.clone()
    for decay in (1.0, 0.5):
        before = mass.clone()
        assert pool.prefill_mass(q, lse, mass, decay=decay, scale=0.05) is mass
        check_mass(c, q, lse, 0.05, True, decay, before, mass)
    for b, L in enumerate(lens):
        assert torch.equal(mass[b, :, L:], old[b, :, L:])


def test_scale_and_large_scores():
    """Scores of some thousand, negative scales, a scale of zero."""
    c = Cache([500, 129], 1, 64, 32, seed=7, big=40.0)
    pool = c.pool()
    for scale in (1.0, -0.25, 0.0, 3.5):
        q, lse, _ = decode_case(c, 2, 5, scale)
        got = run_decode(pool, q, lse, None, scale=scale)
        check_mass(c, q, lse, scale, False, 1.0, None, got)


def test_pages_outside_the_pool():
    c = Cache([300, 100], 2, 128, 16, seed=8)
    pool = c.pool()
    q, lse, scale = decode_case(c, 2, 4)
    old = c.mass()
    good = run_decode(pool, q, lse, old, out=torch.zeros_like(old))
    for bad in (-1, c.num, 2 ** 31 - 1, -2 ** 31):
        pool.block_table[0, 3] = bad
        got = run_decode(pool, q, lse, old, out=torch.zeros_like(old))
        assert pool.check_errors() == N.SHKV_ERRF_PAGE_OOB
        assert torch.equal(got[0, :, 48:64], old[0, :, 48:64])
        assert torch.equal(got[0, :, :48], good[0, :, :48]) and torch.equal(got[0, :, 64:], good[0, :, 64:])
        assert torch.equal(got[1], good[1])
        got = pool.prefill_mass(q, lse, old, out=torch.zeros_like(old))
        assert pool.check_errors() == N.SHKV_ERRF_PAGE_OOB
        assert torch.equal(got[0, :, 48:64], old[0, :, 48:64])
    pool.block_table.copy_(c.table)
    pool.seq_lens[1] += 1
    run_decode(pool, q, lse, old, out=torch.zeros_like(old))
    assert pool.check_errors() == N.SHKV_ERRF_SEQ_LEN


PREFILL = [
    # lens, n, hq, hkv, d, page
    ([1], 1, 1, 1, 64, 16),
    ([5, 40, 300], 5, 8, 2, 128, 16),
    ([128, 129, 127], 127, 4, 2, 128, 32),
    ([256, 300, 1000], 256, 2, 1, 128, 16),
    ([257, 258, 700], 257, 3, 3, 64, 32),
    ([513, 900], 400, 10, 2, 128, 16),
    ([300, 2000], 100, 14, 2, 64, 16),
    ([140, 141], 33, 128, 1, 128, 16),
    ([77, 1200], 65, 127, 1, 64, 32),
    ([600], 600, 66, 2, 128, 32),
    ([4000, 3000], 32, 32, 8, 128, 16),
    ([2500], 2500, 5, 1, 128, 16),
    ([900, 1100, 1300, 901], 16, 8, 8, 64, 16),
]


@pytest.mark.parametrize("lens,n,hq,hkv,d,page", PREFILL)
@pytest.mark.parametrize("decay", [0.0, 0.9])
def test_prefill(lens, n, hq, hkv, d, page, decay):
    c = Cache(lens, hkv, d, page, seed=n + hq)
    for b, L in enumerate(lens):            # slots behind the end
        if L % page:
            c.k[int(c.table[b, L // page]), :, L % page:] = float("nan")
    pool = c.pool()
    q = c.randn(len(lens), n, hq, d)
    scale = d ** -0.5
    lse = lse_of(c, q, scale, True)
    old = c.mass(extra=1)
    out = torch.full_like(old, 3.0)
    got = pool.prefill_mass(q, lse, old, decay=decay, out=out)
    assert got is out and pool.check_errors() == 0
    check_mass(c, q, lse, scale, True, decay, old, got)
    for b, L in enumerate(lens):
        assert (got[b, :, L:] == 3.0).all()


@pytest.mark.parametrize("window", [1, 7, 64, 100])
def test_a_window_of_the_last_tokens(window):
    c = Cache([100, 450, 1500], 4, 128, 16, seed=window)
    pool = c.pool()
    q = c.randn(3, 100, 12, 128)
    scale = 0.07
    lse = lse_of(c, q, scale, True)
    got = pool.prefill_mass(q[:, -window:], lse[:, -window:], None, scale=scale)
    check_mass(c, q[:, -window:], lse[:, -window:], scale, True, 1.0, None, got)
    wide = torch.zeros(3, 100, 3, 12, 128, dtype=torch.bfloat16, device="cuda")       # tokens of a fused projection
    wide[:, :, 1] = q
    same = pool.prefill_mass(wide[:, -window:, 1], lse[:, -window:], None, scale=scale)
    assert torch.equal(same, got)


def test_new_tokens_weigh_nothing_behind_themselves():
    """NaN and infinities in keys that a row does not see stay out of its sums, and a NaN query stays among the
    tokens that it sees; queries of another request, and those before a window, reach nobody."""
    c = Cache([150, 260], 1, 128, 16, seed=9)
    n, hq = 40, 6
    pool = c.pool()
    q = c.randn(2, n + 8, hq, 128)
    lse = lse_of(c, q[:, 8:], c.d ** -0.5, True)
    full = torch.full((2, n + 8, hq), float("nan"), device="cuda")
    full[:, 8:] = lse
    q[:, :8] = float("nan")
    got = pool.prefill_mass(q[:, 8:], full[:, 8:], None)
    check_mass(c, q[:, 8:], lse, c.d ** -0.5, True, 1.0, None, got)
    q[0, 8 + 10] = float("inf")             # token 120 of request 0 sees tokens 0 .. 120
    nan = torch.isnan(pool.prefill_mass(q[:, 8:], full[:, 8:], None))
    assert nan[0, 0, :121].all() and int(nan.sum()) == 121


def test_every_row_adds_up_to_one():
    """A prompt with its attention's own log-sum-exps: the masses of a head add up to its rows."""
    c = Cache([700, 1000], 2, 128, 16, seed=10)
    pool = c.pool()
    q = c.randn(2, 600, 8, 128)
    _, lse = pool.prefill_attention(q, return_lse=True)
    got = pool.prefill_mass(q, lse, None)
    assert torch.allclose(got.double().sum(2), torch.full((2, 2), 2400.0, device="cuda", dtype=torch.float64), rtol=1e-3)
    check_mass(c, q, lse, c.d ** -0.5, True, 1.0, None, got)


def test_the_same_call_gives_the_same_bits():
    c = Cache([3000, 1700, 5], 2, 128, 16, seed=11)
    pool = c.pool()
    q, lse, _ = decode_case(c, 5, 8)
    ref = run_decode(pool, q, lse, None)
    qp = c.randn(3, 5, 64, 128)
    lp = lse_of(c, qp, 0.05, True)
    refp = pool.prefill_mass(qp, lp, None, scale=0.05)
    for _ in range(5):
        assert torch.equal(run_decode(pool, q, lse, None), ref)
        assert torch.equal(pool.prefill_mass(qp, lp, None, scale=0.05), refp)


def test_many_requests_and_a_long_one():
    """The largest batch of short requests; one whose masses lie past 2^31 bytes; lengths past 131072."""
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 200, (1024,), generator=g).tolist()
    c = Cache(lens, 1, 64, 16, seed=12)
    pool = c.pool()
    q, lse, scale = decode_case(c, 1, 3)
    got = run_decode(pool, q, lse, None)
    assert pool.check_errors() == 0
    check_mass(c, q, lse, scale, False, 1.0, None, got, requests=range(0, 1024, 31))
    c = Cache([200003, 40], 1, 128, 32, seed=13)
    pool = c.pool()
    q, lse, scale = decode_case(c, 2, 4)
    wide = torch.zeros(2 * 600_000_000, device="cuda").view(2, 1, -1)
    got = run_decode(pool, q, lse, wide)
    check_mass(c, q, lse, scale, False, 1.0, None, got[:, :, :200003])
    del wide, got
    qp = c.randn(2, 20, 4, 128)
    lp = lse_of(c, qp, scale, True)
    check_mass(c, qp, lp, scale, True, 1.0, None, pool.prefill_mass(qp, lp, None))
    assert pool.check_errors() == 0


def test_refusals():
    c = Cache([100, 60], 2, 128, 16)
    pool = c.pool()
    q, lse, _ = decode_case(c, 2, 8)
    for kw in (dict(scale=float("nan")), dict(scale=float("inf")), dict(decay=float("nan")), dict(decay=float("inf"))):
        with pytest.raises(N.ShkvError) as e:
            run_decode(pool, q, lse, c.mass(), **kw)
        assert e.value.status == N.SHKV_ERR_INVALID_ARG
    with pytest.raises(N.ShkvError) as e:    # more than 64 stacked rows
        run_decode(pool, *(t for t in decode_case(c, 5, 26)[:2]), c.mass())
    assert e.value.status == N.SHKV_ERR_UNSUPPORTED
    with pytest.raises(N.ShkvError) as e:    # query heads that KV heads do not divide
        run_decode(pool, c.randn(2, 1, 3, 128), torch.zeros(2, 1, 3, device="cuda"), c.mass())
    assert e.value.status == N.SHKV_ERR_UNSUPPORTED
    with pytest.raises(N.ShkvError) as e:    # a request shorter than the chunk
        pool.prefill_mass(c.randn(2, 61, 8, 128), torch.zeros(2, 61, 8, device="cuda"), c.mass())
    assert e.value.status == N.SHKV_ERR_INVALID_ARG
    with pytest.raises(N.ShkvError) as e:    # more than 128 heads a KV head
        pool.prefill_mass(c.randn(2, 1, 258, 128), torch.zeros(2, 1, 258, device="cuda"), c.mass())
    assert e.value.status == N.SHKV_ERR_UNSUPPORTED
    m = c.mass()
    for out in (m[:1].expand(2, 2, 100), m[:, :1].expand(2, 2, 100), m.view(-1)[:250].as_strided((2, 2, 100), (50, 100, 1))):
        with pytest.raises(N.ShkvError) as e:                # rows that overlap
            run_decode(pool, q, lse, None, out=out)
        assert e.value.status == N.SHKV_ERR_INVALID_ARG
    with pytest.raises(N.ShkvError) as e:                    # the same memory in another layout
        run_decode(pool, q, lse, m, out=m.view(2, 2, 100).transpose(0, 1))
    assert e.value.status == N.SHKV_ERR_INVALID_ARG
    for mass in (c.mass().double(), c.mass()[:, :, :99], c.mass()[:1], c.mass()[:, :1], c.mass().cpu(),
                 c.mass().repeat(1, 1, 2)[:, :, ::2], c.mass()[0]):
        with pytest.raises((N.ShkvError, ValueError)):
            run_decode(pool, q, lse, mass)
    with pytest.raises(ValueError):
        pool.decode_mass(q.view(2, 16, 128), lse.view(2, 16), 3, m)
    with pytest.raises(ValueError):
        pool.decode_mass(q.view(2, 16, 128), lse.view(2, 16).double(), 2, m)
    with pytest.raises(ValueError):
        pool.decode_mass(q.view(2, 16, 128).half(), lse.view(2, 16), 2, m)
    with pytest.raises(ValueError):
        pool.prefill_mass(q.transpose(2, 3).contiguous().transpose(2, 3), lse, m)
    with pytest.raises(N.ShkvError):         # tokens that share elements, or are not 16 bytes apart
        pool.prefill_mass(c.randn(2, 1, 8, 128).expand(2, 20, 8, 128), torch.zeros(2, 20, 8, device="cuda"), m)
    with pytest.raises(N.ShkvError):
        wide = torch.zeros(2, 20, 8 * 128 + 4, dtype=torch.bfloat16, device="cuda")
        pool.prefill_mass(wide[:, :, : 8 * 128].unflatten(2, (8, 128)), torch.zeros(2, 20, 8, device="cuda"), m)
    assert pool.check_errors() == 0
