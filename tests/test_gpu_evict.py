"""Which tokens stay, and their move into new pages, against the definitions; the
operators together, as a session uses them."""
import numpy as np
import pytest
import torch

from cross_model_shared_gb300 import DecoderTails, PrefixPages
from cross_model_shared_gb300 import _native as N

from .eviction_common import Cache, check_mass, check_selection, evicted, lse_of, scores
from .gpu_common import compare

pytestmark = pytest.mark.gpu


def select_pool(lens, hkv):
    """A pool whose requests only have lengths: a selection reads no page."""
    c = Cache([0] * len(lens), hkv, 64, 16)
    c.table = torch.full((len(lens), max(1, -(-max(lens) // 16))), -1, dtype=torch.int32)
    return c.pool(lens=lens)


def draw_masses(kind, B, hkv, T, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.rand(B, hkv, T, generator=g)
    if kind == "octaves":
        return torch.exp(6.0 * torch.randn(B, hkv, T, generator=g)).cuda()
    if kind == "few values":                 # many ties, also at the border
        return (x * 5).floor().cuda()
    if kind == "zeros":                      # of both signs
        return torch.where(x < 0.5, torch.tensor(0.0), torch.tensor(-0.0)).cuda()
    if kind == "anything":                   # every bit pattern: NaN of both signs, infinities, subnormals
        return torch.randint(-2 ** 31, 2 ** 31, (B, hkv, T), generator=g).int().view(torch.float32).cuda()
    if kind == "specials":
        pool = torch.tensor([float("nan"), -float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-45, -1e-45, 1.0, -1.0])
        return pool[(x * len(pool)).long()].cuda()
    if kind == "close":                      # they differ in the last bits alone
        return (torch.ones(B, hkv, T).view(torch.int32) + (x * 40).int()).view(torch.float32).cuda()
    return x.cuda()


@pytest.mark.parametrize("kind", ["uniform", "octaves", "few values", "zeros", "anything", "specials", "close"])
@pytest.mark.parametrize("lens,hkv", [([1, 2, 0, 3, 31, 32, 33], 1), ([1000, 1023, 1024, 1025, 2049, 500], 2),
                                      ([5000, 130, 4097], 3), ([20000], 2)])
def test_selection(kind, lens, hkv):
    pool = select_pool(lens, hkv)
    mass = draw_masses(kind, len(lens), hkv, max(lens) + 3, seed=len(kind) + len(lens))
    for sink, recent in ((0, 0), (1, 0), (0, 7), (4, 32)):
        for f in (0.0, 0.1, 0.5, 0.99, 1.0):
            keep = [max(int(f * L), sink + recent) for L in lens]
            index = pool.select_tokens(mass, keep, sink=sink, recent=recent)
            assert index.shape[2] == max(1, max(min(k, L) for k, L in zip(keep, lens)))
            check_selection(mass, lens, keep, sink, recent, index)
    assert pool.check_errors() == 0


@pytest.mark.parametrize("lens", [[131584, 70001], [400000], [65536, 65537, 16384, 16385, 262145]])
@pytest.mark.parametrize("kind", ["octaves", "few values", "zeros"])
def test_selection_of_long_requests(lens, kind):
    pool = select_pool(lens, 1)
    mass = draw_masses(kind, len(lens), 1, max(lens), seed=5)
    for keep in ([L // 8 for L in lens], [L - 1 for L in lens]):
        check_selection(mass, lens, keep, 16, 1024, pool.select_tokens(mass, keep, sink=16, recent=1024))
    assert pool.check_errors() == 0


@pytest.mark.parametrize("lens,hkv", [
    ([49152], 1), ([49153, 17], 1), ([393216], 1), ([393217, 1], 1),        # keys that just fit, and that do not
    ([50000, 98305, 1, 60000] * 6, 8),                                      # more rows than SMs, in clusters all the same
    ([12000, 30, 4097, 9000] * 6, 8), ([15000, 16000] * 12, 8),             # 512 threads: two or three rows an SM
    ([5000, 4097, 1] * 2, 8), ([16384, 300], 8), ([16385, 300], 8)])        # few rows, short and just long enough
@pytest.mark.parametrize("kind", ["octaves", "few values", "-inf"])
def test_selection_in_every_launch_shape(lens, hkv, kind):
    pool = select_pool(lens, hkv)
    mass = draw_masses("few values" if kind == "-inf" else kind, len(lens), hkv, max(lens), seed=7)
    if kind == "-inf":                       # below every number, and equal to nothing behind the row's end
        mass[mass < 4] = -float("inf")
    for f, sink, recent in ((0.3, 5, 33), (0.9, 0, 0)):
        keep = [max(int(f * L), min(L, sink + recent)) for L in lens]
        check_selection(mass, lens, keep, sink, recent, pool.select_tokens(mass, keep, sink=sink, recent=recent))
    assert pool.check_errors() == 0


def test_selection_of_many_rows_and_every_keep():
    lens = np.random.default_rng(1).integers(0, 90, 1024).tolist()
    pool = select_pool(lens, 2)
    mass = draw_masses("octaves", 1024, 2, 90, seed=1)
    keep = [L // 3 + 6 for L in lens]
    check_selection(mass, lens, keep, 2, 4, pool.select_tokens(mass, keep, sink=2, recent=4))
    pool = select_pool([67], 2)
    mass = draw_masses("few values", 1, 2, 67, seed=2)
    for keep in range(0, 70):
        check_selection(mass, [67], [keep], 0, 0, pool.select_tokens(mass, [keep]))
    for keep in range(5, 70):
        check_selection(mass, [67], [keep], 3, 2, pool.select_tokens(mass, [keep], sink=3, recent=2))


def test_selection_into_a_wider_tensor_and_from_any_stride():
    lens = [300, 41]
    pool = select_pool(lens, 2)
    mass = draw_masses("octaves", 2, 2, 601, seed=3).transpose(0, 1)[:, :, 1:]
    out = torch.full((2, 2, 333), 5, dtype=torch.int32, device="cuda")
    got = pool.select_tokens(mass, [100, 100], sink=1, recent=3, out=out)
    assert got is out
    check_selection(mass, lens, [100, 100], 1, 3, out)
    assert (out[0, :, 100:] == -1).all() and (out[1, :, 41:] == -1).all()


def test_selection_refusals():
    pool = select_pool([300, 41], 2)
    mass = draw_masses("uniform", 2, 2, 300, seed=3)
    for keep, sink, recent in (([5, 5], 3, 3), ([-1, 5], 0, 0), ([100, 100], -1, 0), ([100, 100], 0, -1),
                               ([100, 100], 2 ** 31 - 1, 2 ** 31 - 1)):
        with pytest.raises((N.ShkvError, ValueError)):
            pool.select_tokens(mass, keep, sink=sink, recent=recent)
    assert pool.select_tokens(mass, [300, 50], sink=30, recent=30).shape == (2, 2, 300)    # nobody is over the budget
    for m in (mass[:, :, :299], mass.double(), mass.cpu(), mass[:, :1], mass[:1], mass[0]):
        with pytest.raises((N.ShkvError, ValueError)):
            pool.select_tokens(m, [100, 20])
    for out in (torch.zeros(2, 2, 99, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, 100, device="cuda"),
                torch.zeros(2, 1, 100, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, 100, dtype=torch.int32)):
        with pytest.raises((N.ShkvError, ValueError)):
            pool.select_tokens(mass, [100, 20], out=out)
    with pytest.raises(ValueError):
        pool.select_tokens(mass, [100, 20, 30])
    assert pool.select_tokens(mass, []).shape[0] == 0
    assert pool.check_errors() == 0


def spare_table(c, keep, lens, at=0, width=0):
    """New pages for the moved requests, from the cache's spare ones."""
    need = [-(-k // c.page) if k < L else 0 for k, L in zip(keep, lens)]
    t = torch.full((len(keep), max(need + [1]) + width), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        t[b, :n] = torch.tensor(c.free[at: at + n], dtype=torch.int32)
        at += n
    return t.cuda()


def drawn_index(c, keep, lens, seed=0):
    g = torch.Generator().manual_seed(seed)
    index = torch.full((len(keep), c.hkv, max(max(min(k, L) for k, L in zip(keep, lens)), 1)), -1, dtype=torch.int32)
    for b, (k, L) in enumerate(zip(keep, lens)):
        for h in range(c.hkv):
            n = min(k, L)
            index[b, h, :n] = torch.sort(torch.randperm(L, generator=g)[:n]).values.int()
    return index.cuda()


@pytest.mark.parametrize("d,page", [(64, 16), (64, 32), (128, 16), (128, 32)])
@pytest.mark.parametrize("lens,keep,hkv", [
    ([1], [0], 1), ([40], [39], 2), ([100, 0, 33, 64, 17], [50, 0, 33, 70, 1], 3), ([16, 32, 48], [15, 16, 17], 1),
    ([3000, 1500, 700], [1000, 1499, 0], 2), ([5000], [4999], 8)])
@pytest.mark.parametrize("where", ["none", "in place", "out"])
def test_eviction(d, page, lens, keep, hkv, where):
    c = Cache(lens, hkv, d, page, seed=sum(lens) + d, spare=sum(-(-k // page) for k in keep) + 2)
    pool = c.pool()
    index, new = drawn_index(c, keep, lens), spare_table(c, keep, lens, width=1)
    want_k, want_v = evicted(c, index, keep, new)
    old = c.mass(extra=3)
    mass, out = old.clone(), torch.full_like(old, 7.0)
    pool.evict_tokens(index, keep, new, mass=None if where == "none" else mass, out=out if where == "out" else None)
    assert pool.check_errors() == 0
    assert torch.equal(c.k, want_k) and torch.equal(c.v, want_v)
    for b, (L, k) in enumerate(zip(lens, keep)):
        n = min(L, k)
        assert pool.host_seq_lens()[b] == n and int(pool.seq_lens[b]) == n
        row = torch.full((pool.max_pages_per_seq,), -1, dtype=torch.int32)
        if k < L:
            row[: -(-k // page)] = new[b, : -(-k // page)].cpu()
        else:
            row[: c.table.shape[1]] = c.table[b]
        assert torch.equal(pool.block_table[b].cpu(), row)
        got, rest = (mass, old) if where == "in place" else (out, torch.full_like(old, 7.0))
        if where != "none" and k < L:
            assert torch.equal(got[b, :, :k], old[b].gather(1, index[b, :, :k].long()))
            assert not got[b, :, k:L].any() and torch.equal(got[b, :, L:], rest[b, :, L:])
        elif where != "none":
            assert torch.equal(got[b], rest[b])
    if where != "in place":
        assert torch.equal(mass, old)
    if where != "out":
        assert (out == 7.0).all()


def test_eviction_of_long_requests_with_their_masses():
    lens, keep = [140000, 9000], [70001, 4500]
    c = Cache(lens, 1, 64, 32, seed=2, spare=2400)
    pool = c.pool()
    mass = c.mass()
    index = pool.select_tokens(mass, keep, sink=5, recent=500)
    check_selection(mass, lens, keep, 5, 500, index)
    new = spare_table(c, keep, lens)
    want_k, want_v = evicted(c, index, keep, new)
    want_mass = [mass[b].gather(1, index[b, :, :n].long()) for b, n in enumerate(keep)]
    pool.evict_tokens(index, keep, new, mass=mass)
    assert pool.check_errors() == 0 and torch.equal(c.k, want_k) and torch.equal(c.v, want_v)
    for b, n in enumerate(keep):
        assert torch.equal(mass[b, :, :n], want_mass[b]) and not mass[b, :, n: lens[b]].any()


def test_an_index_in_no_order_into_other_masses():
    """Any positions may be named, also one more than once; masses then go elsewhere."""
    c = Cache([200, 90], 2, 128, 16, seed=3, spare=20)
    pool = c.pool()
    index = torch.randint(0, 90, (2, 2, 60), generator=c.g, dtype=torch.int32).cuda()
    new = spare_table(c, [60, 60], c.lens)
    want_k, want_v = evicted(c, index, [60, 60], new)
    old = c.mass()
    out = torch.zeros_like(old)
    pool.evict_tokens(index, [60, 60], new, mass=old, out=out)
    assert pool.check_errors() == 0 and torch.equal(c.k, want_k) and torch.equal(c.v, want_v)
    for b in range(2):
        assert torch.equal(out[b, :, :60], old[b].gather(1, index[b].long()))


@pytest.mark.parametrize("source", ["a copy", "the pool's own", "part of a wider one"])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32)])
@pytest.mark.parametrize("masses", [False, True])
def test_a_named_source(source, d, page, masses):
    """The table that the call reads may be the one that it writes."""
    lens, keep = [700, 33, 0, 512, 90], [300, 40, 3, 511, 0]
    c = Cache(lens, 3, d, page, seed=31, spare=70)
    pool = c.pool()
    if source == "the pool's own":
        table = pool.block_table[:5]
    else:
        table = torch.full((5, c.table.shape[1] + 7), -1, dtype=torch.int32, device="cuda")
        table[:, : c.table.shape[1]] = c.table.cuda()
        table = table if source == "part of a wider one" else table[:, : c.table.shape[1]].contiguous()
    index, new = drawn_index(c, keep, lens, seed=5), spare_table(c, keep, lens, width=2)
    want_k, want_v = evicted(c, index, keep, new)
    old = c.mass(extra=2)
    mass = old.clone()
    pool.evict_tokens(index, keep, new, mass=mass if masses else None, source=(table, lens))
    assert pool.check_errors() == 0
    assert torch.equal(c.k, want_k) and torch.equal(c.v, want_v)
    assert pool.seq_lens.tolist() == pool.host_seq_lens().tolist() == [300, 33, 0, 511, 0]
    for b, (L, n) in enumerate(zip(lens, keep)):
        row = c.table[b].clone()
        if n < L:
            row[:] = -1
            w = min(new.shape[1], len(row))
            row[:w] = new[b, :w].cpu()
        assert torch.equal(pool.block_table[b].cpu(), row)
        if masses and n < L:
            assert torch.equal(mass[b, :, :n], old[b].gather(1, index[b, :, :n].long()))
            assert not mass[b, :, n:L].any() and torch.equal(mass[b, :, L:], old[b, :, L:])
        else:
            assert torch.equal(mass[b], old[b])


def test_from_a_table_and_lengths_put_aside():
    """A shared prompt's pages, read for two requests at once, stay intact; a call may be repeated."""
    c = Cache([300], 2, 128, 16, seed=4, spare=30)
    pool = c.pool(lens=[0, 0, 5], max_batch=3)
    table = c.table.repeat(2, 1).cuda()
    keep = [100, 40]
    index = drawn_index(c, keep, [300, 300], seed=9)
    new = spare_table(c, keep, [300, 300])
    want = evicted(c, index, keep, new, lens=[300, 300], table=table)
    for _ in range(2):
        pool.evict_tokens(index, keep, new, source=(table, [300, 300]))
        assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])
        assert pool.host_seq_lens().tolist() == [100, 40, 5] and pool.seq_lens.tolist() == [100, 40, 5]
    before = pool.block_table.clone()
    pool.evict_tokens(index, keep, new, source=(table, [100, 30]))   # nobody is over the budget
    assert torch.equal(pool.block_table, before) and pool.host_seq_lens().tolist() == [100, 40, 5]
    assert pool.check_errors() == 0


def test_bad_indexes_and_pages():
    c = Cache([100, 100], 2, 128, 16, seed=5, spare=20)
    keep = [40, 40]
    good, new = drawn_index(c, keep, c.lens), spare_table(c, keep, c.lens)
    k0, v0 = c.k.clone(), c.v.clone()

    def run(index=good, table=new, bt=None):
        c.k.copy_(k0), c.v.copy_(v0)
        pool = c.pool()
        if bt is not None:
            pool.block_table[bt[0], bt[1]] = bt[2]
        mass = torch.ones(2, 2, 100, device="cuda")
        pool.evict_tokens(index, keep, table, mass=mass)
        return pool.check_errors(), mass

    want_k, want_v = evicted(c, good, keep, new)
    for bad in (-1, 100, 2 ** 31 - 1, -2 ** 31):
        index = good.clone()
        index[1, 0, 7] = bad
        flags, mass = run(index)
        assert flags == N.SHKV_ERRF_INDEX
        k, v = want_k.clone(), want_v.clone()
        to = (int(new[1, 0]), 0, 7)
        k[to], v[to] = k0[to], v0[to]
        assert torch.equal(c.k, k) and torch.equal(c.v, v)
        assert mass[1, 0, 7] == 0 and int(mass[:, :, :40].sum()) == 159
    for bad in (-1, c.num, 2 ** 31 - 1, -2 ** 31):
        table = new.clone()
        table[0, 1] = bad
        flags, _ = run(table=table)
        assert flags == N.SHKV_ERRF_PAGE_OOB
        k, v = want_k.clone(), want_v.clone()
        to = int(new[0, 1])
        k[to], v[to] = k0[to], v0[to]
        assert torch.equal(c.k, k) and torch.equal(c.v, v)
        flags, _ = run(bt=(0, 2, bad))
        assert flags == (N.SHKV_ERRF_PAGE_OOB if bool(((good[0] // 16) == 2).any()) else 0)
        k, v = want_k.clone(), want_v.clone()
        for h in range(2):
            for j in ((good[0, h] // 16) == 2).nonzero()[:, 0].tolist():
                to = (int(new[0, j // 16]), h, j % 16)
                k[to], v[to] = k0[to], v0[to]
        assert torch.equal(c.k, k) and torch.equal(c.v, v)
    c.k.copy_(k0), c.v.copy_(v0)
    pool = c.pool()
    pool.seq_lens[0] = 99
    pool.evict_tokens(good, keep, new)
    assert pool.check_errors() == N.SHKV_ERRF_SEQ_LEN


def test_eviction_refusals():
    c = Cache([100, 100], 2, 128, 16, seed=6, spare=30)
    pool = c.pool()
    keep = [40, 40]
    index, new = drawn_index(c, keep, c.lens), spare_table(c, keep, c.lens)
    mass = c.mass()
    before = c.k.clone()
    bad = [
        lambda: pool.evict_tokens(index, [41, 40], new),                              # past the index
        lambda: pool.evict_tokens(index, keep, new[:, :2].contiguous()),              # past the new table
        lambda: pool.evict_tokens(index, [-1, 40], new),
        lambda: pool.evict_tokens(index, [40, 40, 40], new),
        lambda: pool.evict_tokens(index, keep, pool.block_table),
        lambda: pool.evict_tokens(index[:1].contiguous(), keep[:1], pool.block_table[1:]),   # a part of the pool's own
        lambda: pool.evict_tokens(index, keep, new, out=mass),
        lambda: pool.evict_tokens(index, keep, new, mass=mass[:, :, :99]),
        lambda: pool.evict_tokens(index, keep, new, mass=mass, out=mass[:1].expand(2, 2, 100)),
        lambda: pool.evict_tokens(index.long(), keep, new),
        lambda: pool.evict_tokens(index[:1], keep, new),
        lambda: pool.evict_tokens(index[:, :1], keep, new),
        lambda: pool.evict_tokens(index.cpu(), keep, new),
        lambda: pool.evict_tokens(index, keep, new.long()),
        lambda: pool.evict_tokens(index, keep, new.cpu()),
        lambda: pool.evict_tokens(index, keep, new, source=(pool.block_table, [100])),
        lambda: pool.evict_tokens(index, keep, new, source=(new, [100, 100])),        # longer than its table
        lambda: pool.evict_tokens(index, keep, new, source=(new.cpu(), [40, 48])),
    ]
    for f in bad:
        with pytest.raises((N.ShkvError, ValueError)):
            f()
    assert pool.host_seq_lens().tolist() == [100, 100] and torch.equal(c.k, before) and pool.check_errors() == 0
    big = Cache([2000], 1, 64, 16, seed=7, spare=130)                                 # kept tokens past the pool's capacity
    small = big.pool(lens=[0])
    small.close()
    table = big.table.cuda()
    pool = type(small)(big.num, 16, 1, 64, max_batch=1, max_pages_per_seq=4, k_pages=big.k, v_pages=big.v)
    with pytest.raises(N.ShkvError) as e:
        pool.evict_tokens(drawn_index(big, [65], [2000]), [65], spare_table(big, [65], [2000]), source=(table, [2000]))
    assert e.value.status == N.SHKV_ERR_CAPACITY
    pool.evict_tokens(torch.zeros(0, 1, 1, dtype=torch.int32, device="cuda"), [], table[:0])
    assert pool.check_errors() == 0


@pytest.mark.parametrize("d,page,hkv,group", [(128, 16, 2, 4), (128, 32, 4, 2)])
def test_a_session_within_a_budget_of_pages(d, page, hkv, group):
    """Prompt, attention, votes, eviction, decode steps that vote again, with tails, and a second eviction; pages from
    the page manager.  Attention over what is left is that of the chosen rows."""
    B, T, n_models, hq = 3, 200, 2, hkv * group
    lens = [T, T + 37, T + 300]
    c = Cache([0] * B, hkv, d, page, seed=20, spare=200, extra=60)
    g = c.g
    pages = PrefixPages(c.num, page)
    pool = c.pool(max_batch=B)
    scale = d ** -0.5
    kv = [[torch.randn(L, hkv, d, generator=g).to(torch.bfloat16).cuda() for L in lens] for _ in range(2)]
    held = []
    for b, L in enumerate(lens):
        got = pages.alloc_transfer(-(-(L + 40) // page))
        held.append(list(got))
        pool.block_table[b, : len(got)] = torch.from_numpy(got).cuda()
    # prompts: T new tokens behind prefixes of different length, which are written slot by slot
    for b, L in enumerate(lens):
        for t in range(L - T):
            for pg, x in ((c.k, kv[0]), (c.v, kv[1])):
                pg[held[b][t // page], :, t % page] = x[b][t]
    pool.set_seq_lens([L - T for L in lens])
    pool.append_kv(*(torch.stack([x[b][-T:] for b in range(B)]) for x in kv))
    c.lens, c.table = list(lens), pool.block_table.cpu()
    q = c.randn(B, T, hq, d)
    _, lse = pool.prefill_attention(q, return_lse=True)
    mass = torch.zeros(B, hkv, 600, device="cuda")
    pool.prefill_mass(q[:, -32:], lse[:, -32:], mass)
    check_mass(c, q[:, -32:], lse[:, -32:], scale, True, 1.0, torch.zeros_like(mass), mass)
    rows = [[[x[b].transpose(0, 1).double() for x in kv] for b in range(B)]][0]      # fp64 [hkv, L, d] of each request
    tails = DecoderTails(pool, B, n_models, 2)
    for step, keep in enumerate(([90, 90, 120], [60, 300, 61])):
        index = pool.select_tokens(mass, keep, sink=4, recent=16)
        check_selection(mass, lens, keep, 4, 16, index)
        new = torch.full((B, 40), -1, dtype=torch.int32)
        old = []
        for b, (k, L) in enumerate(zip(keep, lens)):
            if k < L:                       # pages for the kept tokens and for some to come
                got = pages.alloc_transfer(-(-(k + 40) // page))
                old += held[b]
                held[b] = list(got)
                new[b, : len(got)] = torch.from_numpy(got)
                rows[b] = [torch.stack([x[h][index[b, h, :k].long()] for h in range(hkv)]) for x in rows[b]]
                lens[b] = k
        pool.evict_tokens(index, keep, new.cuda(), mass=mass)
        pages.release(old)
        assert pool.host_seq_lens().tolist() == lens
        for _ in range(3):                  # decode steps
            kn, vn = (c.randn(B, 1, hkv, d) for _ in range(2))
            pool.append_kv(kn, vn)
            for b in range(B):
                rows[b] = [torch.cat([r, x[b].transpose(0, 1).double()], 1) for r, x in zip(rows[b], (kn, vn))]
                lens[b] += 1
            qd = c.randn(B, n_models * hq, d)
            out, lse = pool.decode_attention(qd, n_models, return_lse=True)
            want = torch.zeros(B, n_models, hq, d, dtype=torch.float64, device="cuda")
            for b in range(B):
                s, _ = scores(qd[b].view(n_models, hq, d), rows[b][0], scale, False)
                o = torch.softmax(s, -1) @ rows[b][1]
                want[b] = o.view(hkv, n_models, group, d).transpose(0, 1).reshape(n_models, hq, d)
            compare(out.view(-1, d), want.view(-1, d).cpu().numpy(), what=f"after eviction {step}")
            before = mass.clone()
            pool.decode_mass(qd, lse, n_models, mass, decay=0.9)
            c.lens, c.table = list(lens), pool.block_table.cpu()
            check_mass(c, qd.view(B, n_models, hq, d), lse.view(B, n_models, hq), scale, False, 0.9, before, mass)
        # a step with per-decoder tails: weights of the shared tokens under the whole softmax
        tpages = torch.from_numpy(pages.alloc_transfer(B * n_models * 2).reshape(B, n_models, 2)).cuda()
        tails.block_table.copy_(tpages)
        tails.set_lens(np.zeros((B, n_models), np.int32))
        tails.append(*(c.randn(B, n_models, 5, hkv, d) for _ in range(2)))
        _, tl = tails.decode_attention(qd, return_lse=True)
        assert (tl > lse).all()
        got = pool.decode_mass(qd, tl, n_models, None)
        check_mass(c, qd.view(B, n_models, hq, d), tl.view(B, n_models, hq), scale, False, 1.0, None, got)
        pages.release(tpages.cpu().numpy().reshape(-1))
    assert pool.check_errors() == 0


@pytest.mark.parametrize("aside", [False, True])
def test_a_decode_with_tails_right_behind_an_eviction(aside):
    """Its unit kernel reads the block table that the eviction has just written."""
    c = Cache([3000, 2500], 2, 128, 16, seed=21, spare=400)
    pool = c.pool()
    q = c.randn(2, 16, 128)
    tails = DecoderTails(pool, 2, 2, 1)
    tails.block_table.copy_(torch.tensor(c.free[-4:], dtype=torch.int32).view(2, 2, 1))
    tails.set_lens(np.full((2, 2), 7, np.int32))
    keep = [1500, 1100]
    index, new = drawn_index(c, keep, c.lens), spare_table(c, keep, c.lens)
    old = pool.block_table.clone()
    want = None
    for i in range(10):
        pool.block_table.copy_(old)
        pool.set_seq_lens(c.lens)
        tails.decode_attention(q)
        pool.evict_tokens(index, keep, new, source=(old, c.lens) if aside else None)
        got = tails.decode_attention(q)
        torch.cuda.synchronize()
        if want is None:
            want = tails.decode_attention(q)
        assert torch.equal(got, want), i
    assert pool.check_errors() == 0
