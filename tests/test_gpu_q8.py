"""The 8-bit KV cache's operators on the GPU against their definitions in 64 bits."""
import numpy as np
import pytest
import torch

from cross_model_shared_gb300 import QuantizedKVPool
from cross_model_shared_gb300 import _native as N

from .q8_common import TABLE, Cache, attend, check, check_chunk, check_decode, dequantise, quantise

pytestmark = pytest.mark.gpu


def no_errors(pool):
    assert pool.check_errors() == 0


# ---------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------
def special_rows(rows):
    """Rows [n, d] whose first ones hold what a rounding or a scale can get wrong."""
    rows = rows.clone()
    n, d = rows.shape
    big = torch.finfo(torch.bfloat16).max
    special = [
        torch.zeros(d),
        torch.full((d,), big),
        torch.full((d,), -2.0 ** -133),                                    # the smallest subnormal
        torch.where(torch.arange(d) % 2 == 0, 1.75, -2.0 ** -9),            # 448 exactly, and subnormal codes
        torch.full((d,), 1.7578125),                                        # one step above 1.75
        torch.tensor([1.75] + [(2 * i + 1) * 1.75 / 1024 for i in range(d - 1)]),   # ties between codes
        torch.tensor([float("inf")] + [1.0] * (d - 1)),
        torch.tensor([1.0] * (d - 1) + [float("nan")]),
        torch.tensor([-0.0, 3.0] * (d // 2)),
        torch.linspace(-2.0 ** -118, 2.0 ** -118, d),
    ]
    for i, r in enumerate(special[:n]):
        rows[i] = r
    return rows.to(torch.bfloat16)


@pytest.mark.parametrize("hkv,d,page", [(1, 64, 16), (2, 128, 16), (3, 64, 32), (8, 128, 32)])
@pytest.mark.parametrize("strided", [False, True])
def test_append_writes_the_nearest_codes_and_nothing_else(hkv, d, page, strided):
    start, new = [0, 5, 31, 0, 17], [19, 0, 1, 40, 33]
    lens = [s + n for s, n in zip(start, new)]
    c = Cache(lens, hkv, d, page, seed=hkv * 100 + d)
    pool = c.pool(lens=start)
    T = sum(new)
    g = torch.Generator().manual_seed(7)
    x = [torch.randn(T * hkv, d, generator=g) * torch.exp2(torch.randn(T * hkv, 1, generator=g) * 4) for _ in "kv"]
    k, v = (special_rows(r).view(T, hkv, d).cuda() for r in x)
    if strided:
        both = torch.cat([k, v, k], 1)
        k, v = both[:, :hkv], both[:, hkv: 2 * hkv]
    before = [t.clone() for t in (c.k, c.v, c.sc)]
    pool.append_kv(k, v, new, start=start if strided else None)
    no_errors(pool)
    assert pool.host_seq_lens().tolist() == lens and pool.seq_lens.tolist() == lens
    want = [t.clone() for t in before]
    at = 0
    for b, n in enumerate(new):
        for i in range(n):
            page_id, slot = int(c.table[b, (start[b] + i) // page]), (start[b] + i) % page
            for j, t in enumerate((k, v)):
                codes, s = quantise(t[at + i].double().cpu().numpy())
                want[j][page_id, :, slot] = torch.from_numpy(codes).cuda()
                want[2][page_id, :, j, slot] = torch.from_numpy(s).cuda()
        at += n
    for got, ref in zip((c.k, c.v, c.sc), want):
        assert torch.equal(got, ref)


@pytest.mark.parametrize("hkv,d,page", [(1, 64, 16), (2, 128, 16), (3, 64, 32), (8, 128, 32)])
def test_read_returns_the_rows_exactly(hkv, d, page):
    lens = [0, 1, 77, 130]
    c = Cache(lens, hkv, d, page, seed=3, scale_lo=0, scale_hi=246)
    c.k[0, 0, 0, 0], c.sc[0, 0, 0, 0] = 0x7F, 255
    pool = c.pool()
    start, n = [0, 0, 33, 0], [0, 1, 44, 130]
    T = sum(n)
    buf = torch.full((2, T + 3, hkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = pool.read_kv(start, n, k_out=buf[0, :T], v_out=buf[1, :T])
    no_errors(pool)
    assert (buf[:, T:] == 7).all()
    want = [torch.cat([c.rows(b)[j][start[b]: start[b] + n[b]] for b in range(len(lens))]) for j in (0, 1)]
    for got, ref in zip((k, v), want):
        same = torch.equal(got.double().nan_to_num(1e30), ref.to(torch.bfloat16).double().nan_to_num(1e30))
        assert same


def test_requantising_what_was_read_gives_the_same_values():
    c = Cache([50], 2, 128, 16, seed=4)
    pool = c.pool()
    x = torch.randn(50, 2, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    pool.append_kv(x, -x, [50], start=[0])
    k, v = pool.read_kv([0], [50])
    pool.append_kv(k, v, [50], start=[0])
    k2, v2 = pool.read_kv([0], [50])
    assert torch.equal(k, k2) and torch.equal(v, v2)
    assert torch.equal(v, -k)
    x = x.double().abs()
    assert ((k.double().abs() - x).abs() <= x * 2.0 ** -4 + x.amax(-1, keepdim=True) * 2.0 ** -18).all()


def test_start_drops_rejected_tokens():
    c = Cache([64, 40], 2, 64, 16, seed=5)
    pool = c.pool(lens=[20, 30])
    x = torch.randn(9, 2, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    pool.append_kv(x, x, [5, 4])
    assert pool.host_seq_lens().tolist() == [25, 34]
    pool.append_kv(x[:2], x[:2], [2, 0], start=[22, 31])
    assert pool.host_seq_lens().tolist() == [24, 31] == pool.seq_lens.tolist()
    pool.append_kv(x[:0], x[:0], [0, 0], start=[10, 0])
    assert pool.host_seq_lens().tolist() == [10, 0] == pool.seq_lens.tolist()
    pool.append_kv(x[:0], x[:0], [0, 0])
    no_errors(pool)
    assert pool.host_seq_lens().tolist() == [10, 0]


def test_pages_outside_the_pool_are_skipped_and_flagged():
    c = Cache([48, 32], 2, 128, 16, seed=6)
    pool = c.pool(lens=[0, 0])
    pool.block_table[0, 1] = c.num
    pool.block_table[1, 0] = -1
    before = [t.clone() for t in (c.k, c.v, c.sc)]
    x = torch.randn(80, 2, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    pool.append_kv(x, x, [48, 32])
    assert pool.check_errors() == N.SHKV_ERRF_PAGE_OOB
    mapped = {int(c.table[0, 0]), int(c.table[0, 2]), int(c.table[1, 1])}
    for got, ref in zip((c.k, c.v, c.sc), before):
        same = [i for i in range(c.num) if torch.equal(got[i], ref[i])]
        assert set(range(c.num)) - set(same) == mapped
    k, v = pool.read_kv([0, 0], [48, 32])
    assert pool.check_errors() == N.SHKV_ERRF_PAGE_OOB
    zero = [*range(16, 32), *range(48, 64)]
    assert not k[zero].any() and not v[zero].any() and k[64:].any()


# ---------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------
DECODES = [
    # lens, N, hq, hkv, d, page
    ([256], 2, 8, 2, 64, 16),
    ([1], 1, 1, 1, 64, 16),
    ([1, 0, 17, 128], 1, 4, 4, 128, 32),
    ([127, 128, 129, 255, 257], 2, 8, 2, 128, 16),
    ([1000, 3, 0, 2047], 3, 10, 2, 128, 16),
    ([700, 1, 1300], 8, 14, 2, 64, 32),
    ([511, 640], 8, 40, 8, 128, 32),
    ([900, 33], 8, 8, 1, 128, 16),
    ([333, 4097], 4, 16, 1, 64, 16),
    ([5000], 1, 3, 3, 128, 32),
    ([20011], 8, 16, 8, 128, 16),
    ([3] * 70, 1, 2, 1, 128, 16),
    ([0, 0], 1, 2, 1, 128, 16),
]


@pytest.mark.parametrize("lens,N_,hq,hkv,d,page", DECODES)
def test_decode(lens, N_, hq, hkv, d, page):
    c = Cache(lens, hkv, d, page, seed=len(lens) + hq)
    pool = c.pool()
    q = c.q(len(lens), N_ * hq)
    scale = 1 / np.sqrt(d) / 8
    out, lse = pool.decode_attention(q, N_, scale=scale, return_lse=True)
    no_errors(pool)
    check_decode(c, q, N_, scale, out, lse)
    # the workspace is ready for the next call, and the result does not depend on it
    again = pool.decode_attention(q, N_, scale=scale)
    check_decode(c, q, N_, scale, again, lse)
    no_errors(pool)


@pytest.mark.parametrize("scale", [0.0, -0.02, 3e-4, 0.5])
def test_decode_scales(scale):
    c = Cache([300, 45], 2, 128, 16, seed=8)
    pool = c.pool()
    q = c.q(2, 16)
    out, lse = pool.decode_attention(q, 2, scale=scale, return_lse=True)
    check_decode(c, q, 2, scale, out, lse)


def test_decode_of_uneven_magnitudes():
    """Scales over the whole range of a row's exponent: a first token with a dominating score and a small value,
    values whose magnitudes differ by 2^40, and a row of queries far smaller than its neighbours."""
    c = Cache([700, 700], 2, 128, 16, seed=9, scale_lo=100, scale_hi=140)
    c.sc[:, :, 0] = 119
    for b in range(2):
        first = int(c.table[b, 0])
        c.sc[first, :, 0, 0], c.sc[first, :, 1, 0] = 126, 104
    c.sc[int(c.table[1, 40]), :, 1, :] = 240
    pool = c.pool()
    q = c.q(2, 8)
    q[:, 3] *= 2.0 ** -12
    q[:, 5] *= 2.0 ** 6
    out, lse = pool.decode_attention(q, 1, scale=0.02, return_lse=True)
    no_errors(pool)
    check_decode(c, q, 1, 0.02, out, lse)


def poison(c, lens):
    """NaN codes and scales in every slot that no request's tokens use."""
    used = torch.zeros(c.num, c.page, dtype=torch.bool)
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        used[c.table[b, pos // c.page].long(), pos % c.page] = True
    free = (~used).to(c.device)
    for t in (c.k, c.v):
        t.transpose(1, 2)[free] = 0x7F
    c.sc.permute(0, 3, 1, 2)[free] = 255


@pytest.mark.parametrize("d,page", [(64, 16), (128, 16), (128, 32)])
def test_what_lies_behind_the_last_token_has_no_effect(d, page):
    lens = [1, 15, 140, 261, 1000]
    c = Cache(lens, 2, d, page, seed=10)
    poison(c, lens)
    pool = c.pool()
    q = c.q(len(lens), 16)
    out, lse = pool.decode_attention(q, 2, scale=0.01, return_lse=True)
    no_errors(pool)
    check_decode(c, q, 2, 0.01, out, lse)
    new = [1, 9, 0, 200, 3]
    qc = c.q(sum(new), 8)
    out, lse = pool.chunk_attention(qc, new, scale=0.01, return_lse=True)
    no_errors(pool)
    check_chunk(c, qc, new, 0.01, out, lse)


@pytest.mark.parametrize("n", [60, 5])
def test_nan_rows_of_the_cache_reach_the_rows_that_attend_them(n):
    c = Cache([100, 100, 100], 1, 128, 16, seed=11)
    at = 98 if n == 5 else 55
    for b, j in ((0, 0), (1, 1)):                            # a NaN key of request 0, a NaN value of request 1
        page, slot = int(c.table[b, at // 16]), at % 16
        (c.k, c.v)[j][page, 0, slot], c.sc[page, 0, j, slot] = 0x7F, 255
    pool = c.pool()
    q = c.q(3, 4)
    out = pool.decode_attention(q, 1, scale=0.01)
    assert torch.isnan(out[:2]).all() and torch.isfinite(out[2]).all()
    out = pool.chunk_attention(c.q(3 * n, 4), [n] * 3, scale=0.01).view(3, n, 4, 128)
    sees = at - (100 - n)
    assert torch.isfinite(out[:2, :sees]).all() and torch.isnan(out[:2, sees:]).all() and torch.isfinite(out[2]).all()
    no_errors(pool)


def test_decode_skips_pages_outside_the_pool():
    c = Cache([300, 64], 2, 128, 16, seed=12)
    pool = c.pool()
    q = c.q(2, 8)
    pool.block_table[0, 4] = -7
    pool.block_table[0, 9] = c.num + 3
    out, lse = pool.decode_attention(q, 1, scale=0.01, return_lse=True)
    assert pool.check_errors() == N.SHKV_ERRF_PAGE_OOB
    keep = torch.tensor([t for t in range(300) if t // 16 not in (4, 9)], device="cuda")
    k, v = c.rows(0)
    for h in range(2):
        o, e, to, te = attend(q[0, 4 * h: 4 * h + 4], k[keep][:, h], v[keep][:, h], 0.01)
        check(out[0, 4 * h: 4 * h + 4], o, to, "out")
        check(lse[0, 4 * h: 4 * h + 4], e, te, "lse")
    check_decode(c, q, 1, 0.01, out, lse, requests=[1])


def test_offsets_past_32_bits():
    """Pages whose byte offsets exceed 2^31 and 2^32."""
    num, hkv, page, d = 9 * 2 ** 18, 1, 16, 128
    c = Cache([1], hkv, d, page, seed=13)
    c.num, c.lens = num, [100, 40]
    c.k = torch.zeros(num, hkv, page, d, dtype=torch.uint8, device="cuda")
    c.v, c.sc = torch.zeros_like(c.k), torch.zeros(num, hkv, 2, page, dtype=torch.uint8, device="cuda")
    ids = [num - 1, 2 ** 20 + 5, 0, 2 ** 21 + 1, num - 2, 7, 2 ** 20 - 1]
    c.table = torch.full((2, 7), -1, dtype=torch.int32)
    c.table[0] = torch.tensor(ids, dtype=torch.int32)
    c.table[1, :3] = torch.tensor([num - 3, 2 ** 21, 2 ** 20 + 9], dtype=torch.int32)
    pool = c.pool(lens=[0, 0])
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(140, hkv, d, generator=g).to(torch.bfloat16).cuda() for _ in "kv")
    pool.append_kv(k, v, [100, 40])
    no_errors(pool)
    kr, vr = pool.read_kv([0, 0], [100, 40])
    for got, src in ((kr, k), (vr, v)):
        codes, s = quantise(src.double().cpu().numpy())
        assert torch.equal(got.double().cpu(), dequantise(torch.from_numpy(codes), torch.from_numpy(s)))
    q = c.q(2, 4)
    out, lse = pool.decode_attention(q, 1, scale=0.05, return_lse=True)
    no_errors(pool)
    check_decode(c, q, 1, 0.05, out, lse)
    qc = c.q(57, 4)
    out, lse = pool.chunk_attention(qc, [37, 20], scale=0.05, return_lse=True)
    check_chunk(c, qc, [37, 20], 0.05, out, lse)


# ---------------------------------------------------------------------------
# chunk
# ---------------------------------------------------------------------------
CHUNKS = [
    # lens (with the new tokens), new, hq, hkv, d, page
    ([1], [1], 1, 1, 64, 16),
    ([256, 300], [256, 1], 8, 2, 128, 16),
    ([5, 0, 129, 1000], [5, 0, 1, 37], 4, 4, 128, 32),
    ([700, 64, 2000], [300, 64, 129], 14, 2, 64, 16),
    ([333, 900], [333, 8], 40, 8, 128, 32),
    ([1500], [1200], 5, 1, 128, 16),
    ([130, 131, 132], [128, 129, 2], 128, 1, 64, 32),
    ([4000, 10, 3000], [3, 2, 7], 32, 8, 128, 16),
    ([9000], [64], 8, 1, 128, 16),
    ([2100, 77, 2050], [30, 70, 513], 3, 3, 64, 16),
]


@pytest.mark.parametrize("lens,new,hq,hkv,d,page", CHUNKS)
def test_chunk(lens, new, hq, hkv, d, page):
    c = Cache(lens, hkv, d, page, seed=len(lens) * 7 + hq)
    pool = c.pool()
    q = c.q(sum(new), hq)
    scale = 1 / np.sqrt(d) / 8
    out, lse = pool.chunk_attention(q, new, scale=scale, return_lse=True)
    no_errors(pool)
    check_chunk(c, q, new, scale, out, lse)
    out = pool.chunk_attention(q, new, scale=scale)
    no_errors(pool)
    check_chunk(c, q, new, scale, out, lse)


@pytest.mark.parametrize("scale", [0.0, -0.02, 0.3])
def test_chunk_scales(scale):
    c = Cache([400, 45], 2, 128, 16, seed=15)
    pool = c.pool()
    q = c.q(245, 8)
    out, lse = pool.chunk_attention(q, [200, 45], scale=scale, return_lse=True)
    check_chunk(c, q, [200, 45], scale, out, lse)


@pytest.mark.parametrize("new", [[150, 260], [3, 5]])
def test_chunk_of_uneven_magnitudes(new):
    c = Cache([700, 600], 2, 128, 16, seed=16, scale_lo=100, scale_hi=140)
    c.sc[:, :, 0] = 119
    for b in range(2):
        first = int(c.table[b, 0])
        c.sc[first, :, 0, 0], c.sc[first, :, 1, 0] = 126, 104
    c.sc[int(c.table[1, 30]), :, 1, :] = 240
    pool = c.pool()
    q = c.q(sum(new), 8)
    q[::3, 3] *= 2.0 ** -12
    q[1::3, 5] *= 2.0 ** 6
    out, lse = pool.chunk_attention(q, new, scale=0.02, return_lse=True)
    no_errors(pool)
    check_chunk(c, q, new, 0.02, out, lse)


@pytest.mark.parametrize("new", [150, 5])
def test_a_later_tokens_magnitude_has_no_effect_on_earlier_rows(new):
    c = Cache([300], 2, 128, 16, seed=26)
    for t, j, byte in ((299, 1, 240), (298, 0, 200), (297, 1, 170)):
        c.sc[int(c.table[0, t // 16]), :, j, t % 16] = byte
    pool = c.pool()
    q = c.q(new, 8)
    out, lse = pool.chunk_attention(q, [new], scale=0.01, return_lse=True)
    no_errors(pool)
    k, v = c.rows(0)
    n = new - 3                                              # the rows that see none of the three
    limit = (torch.arange(n, device="cuda") + 300 - new + 1).repeat_interleave(4)
    for h in range(2):
        s = slice(4 * h, 4 * h + 4)
        o, e, to, te = attend(q[:n, s].reshape(4 * n, -1), k[:297, h], v[:297, h], 0.01, limit)
        check(out[:n, s].reshape(4 * n, -1), o, to, "out")
        check(lse[:n, s].reshape(-1), e, te, "lse")


def test_chunk_reads_strided_queries_and_writes_no_row_behind_the_last():
    c = Cache([200, 90], 2, 128, 16, seed=17)
    pool = c.pool()
    new = [33, 90]
    wide = c.q(123, 12)
    q = wide[:, 2: 10]
    buf = torch.full((126, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = pool.chunk_attention(q, new, scale=0.01, return_lse=True, out=buf[:123])
    no_errors(pool)
    assert (buf[123:] == 7).all()
    check_chunk(c, q, new, 0.01, out, lse)


def test_chunk_skips_pages_outside_the_pool():
    c = Cache([300, 64], 2, 128, 16, seed=18)
    pool = c.pool()
    pool.block_table[0, 4] = -7
    for new in ([40, 64], [2, 3]):
        q = c.q(sum(new), 8)
        out, lse = pool.chunk_attention(q, new, scale=0.01, return_lse=True)
        assert pool.check_errors() == N.SHKV_ERRF_PAGE_OOB
        keep = torch.tensor([t for t in range(300) if t // 16 != 4], device="cuda")
        k, v = c.rows(0)
        n = new[0]
        limit = (torch.arange(n, device="cuda") + 300 - n + 1 - 16).repeat_interleave(4)
        for h in range(2):
            s = slice(4 * h, 4 * h + 4)
            o, e, to, te = attend(q[:n, s].reshape(4 * n, -1), k[keep][:, h], v[keep][:, h], 0.01, limit)
            check(out[:n, s].reshape(4 * n, -1), o, to, "out")
            check(lse[:n, s].reshape(-1), e, te, "lse")


def test_chunk_of_one_token_equals_a_decode():
    c = Cache([300, 77, 1], 2, 128, 16, seed=19)
    pool = c.pool()
    q = c.q(3, 8)
    a, la = pool.decode_attention(q, 1, scale=0.01, return_lse=True)
    b, lb = pool.chunk_attention(q, [1, 1, 1], scale=0.01, return_lse=True)
    check_decode(c, q, 1, 0.01, a, la)
    check_decode(c, q, 1, 0.01, b, lb)


# ---------------------------------------------------------------------------
# together, and how they are called
# ---------------------------------------------------------------------------
def test_a_session_from_prompt_to_answer():
    """Prompts are appended and attended, drafts are verified and partly
    rejected, a step is decoded by two decoders, and the cache is read back."""
    hkv, hq, d, page, scale = 2, 8, 128, 16, 0.05
    c = Cache([400, 150, 64], hkv, d, page, seed=20)
    pool = c.pool(lens=[0, 0, 0])
    g = torch.Generator().manual_seed(3)
    have = [[], [], []]

    def step(new, start=None):
        T = sum(new)
        k, v = (torch.randn(T, hkv, d, generator=g).to(torch.bfloat16).cuda() for _ in "kv")
        pool.append_kv(k, v, new, start=start)
        at = 0
        for b, n in enumerate(new):
            have[b] = have[b][: len(have[b]) if start is None else start[b]]
            have[b] += [(k[at + i], v[at + i]) for i in range(n)]
            at += n
        c.lens = [len(x) for x in have]
        q = c.q(T, hq)
        out, lse = pool.chunk_attention(q, new, scale=scale, return_lse=True)
        check_chunk(c, q, new, scale, out, lse)

    step([200, 100, 0])
    step([4, 4, 30])
    step([4, 2, 1], start=[202, 100, 30])
    q = c.q(3, 2 * hq)
    out, lse = pool.decode_attention(q, 2, scale=scale, return_lse=True)
    check_decode(c, q, 2, scale, out, lse)
    k, v = pool.read_kv([0, 0, 0], c.lens)
    no_errors(pool)
    for j, got in enumerate((k, v)):
        rows = torch.stack([x[j] for b in range(3) for x in have[b]])
        codes, s = quantise(rows.double().cpu().numpy())
        assert torch.equal(got.double().cpu(), dequantise(torch.from_numpy(codes), torch.from_numpy(s)))


def test_captured_calls_replay_with_new_inputs_and_share_no_workspace():
    c = Cache([900, 333], 2, 128, 16, seed=21)
    pool = c.pool()
    new = [3, 200]
    qd, qc = c.q(2, 16), c.q(203, 8)
    pool.decode_attention(qd, 2, scale=0.01)
    pool.chunk_attention(qc, new, scale=0.01)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append((pool.decode_attention(qd, 2, scale=0.01, return_lse=True),
                         pool.chunk_attention(qc, new, scale=0.01, return_lse=True)))
        graphs.append(g)
    qd.copy_(c.q(2, 16))
    qc.copy_(c.q(203, 8))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    eager = pool.decode_attention(qd, 2, scale=0.01)
    torch.cuda.synchronize()
    for (a, la), (b, lb) in outs:
        check_decode(c, qd, 2, 0.01, a, la)
        check_chunk(c, qc, new, 0.01, b, lb)
        assert torch.equal(a, eager)
    no_errors(pool)


def test_calls_on_two_streams_at_once():
    c = Cache([3000, 2500, 10], 2, 128, 16, seed=22)
    pool = c.pool()
    q = c.q(3, 16)
    qc = c.q(300, 8)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for s in streams:
            got.append(pool.decode_attention(q, 2, scale=0.01, return_lse=True, stream=s))
            with torch.cuda.stream(s):
                got.append(pool.chunk_attention(qc, [200, 100, 0], scale=0.01, return_lse=True))
    torch.cuda.synchronize()
    for out, lse in got[::2]:
        check_decode(c, q, 2, 0.01, out, lse)
    for out, lse in got[1::2]:
        check_chunk(c, qc, [200, 100, 0], 0.01, out, lse)
    no_errors(pool)


def test_results_do_not_change_from_call_to_call():
    c = Cache([5000, 4000, 333], 2, 128, 16, seed=23)
    pool = c.pool()
    q, qc = c.q(3, 16), c.q(404, 8)
    a, b = pool.decode_attention(q, 2, scale=0.01), pool.chunk_attention(qc, [4, 300, 100], scale=0.01)
    for _ in range(10):
        assert torch.equal(a, pool.decode_attention(q, 2, scale=0.01))
        assert torch.equal(b, pool.chunk_attention(qc, [4, 300, 100], scale=0.01))


def test_a_length_that_differs_on_the_device_is_flagged():
    c = Cache([100], 1, 64, 16, seed=24)
    pool = c.pool()
    pool.seq_lens.fill_(99)
    pool.decode_attention(c.q(1, 2), 1, scale=0.01)
    assert pool.check_errors() == N.SHKV_ERRF_SEQ_LEN
    pool.chunk_attention(c.q(2, 2), [2], scale=0.01)
    assert pool.check_errors() == N.SHKV_ERRF_SEQ_LEN


def test_refusals():
    c = Cache([40, 10], 2, 64, 16, seed=25)
    pool = c.pool()
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = c.q(2, 4)
    cap = pool.max_pages_per_seq * 16

    def refused(status, f, *a, **k):
        with pytest.raises(N.ShkvError) as e:
            f(*a, **k)
        assert e.value.status == status

    def wrong(f, *a, **k):
        with pytest.raises(ValueError):
            f(*a, **k)

    refused(N.SHKV_ERR_INVALID_ARG, pool.append_kv, x, x, [4, 0], start=[41, 0])        # a gap
    refused(N.SHKV_ERR_CAPACITY, pool.append_kv, *[torch.zeros(cap, 2, 64, dtype=torch.bfloat16, device="cuda")] * 2,
            [cap, 0])
    refused(N.SHKV_ERR_INVALID_ARG, pool.append_kv, x, x, [2, 2, 0])                    # more requests than the pool's
    wrong(pool.append_kv, x, x, [2, 1])
    wrong(pool.append_kv, x, x[:3], [2, 2])
    wrong(pool.append_kv, x.float(), x.float(), [2, 2])
    wrong(pool.append_kv, x.cpu(), x.cpu(), [2, 2])
    wrong(pool.append_kv, x, x, [5, -1])
    wrong(pool.append_kv, x, x, [2, 2], start=[0])
    wrong(pool.append_kv, x.transpose(1, 2).contiguous().transpose(1, 2), x, [2, 2])    # a token's rows are not contiguous
    refused(N.SHKV_ERR_INVALID_ARG, pool.read_kv, [0, 5], [40, 6])
    wrong(pool.read_kv, [0, 0], [4, 4], k_out=x[:, :1])
    refused(N.SHKV_ERR_UNSUPPORTED, pool.decode_attention, c.q(2, 132), 1)               # 66 rows per KV head
    refused(N.SHKV_ERR_UNSUPPORTED, pool.decode_attention, c.q(2, 3), 1)                 # 3 heads on 2 KV heads
    refused(N.SHKV_ERR_INVALID_ARG, pool.decode_attention, c.q(3, 4), 1)
    refused(N.SHKV_ERR_INVALID_ARG, pool.decode_attention, q, 1, scale=float("inf"))
    refused(N.SHKV_ERR_INVALID_ARG, pool.decode_attention, q, 1, workspace=torch.zeros(128, dtype=torch.uint8,
                                                                                      device="cuda"))
    wrong(pool.decode_attention, q, 3)
    wrong(pool.decode_attention, q.float(), 1)
    wrong(pool.decode_attention, q, 1, out=q[:1])
    wrong(pool.decode_attention, q, 1, lse=torch.zeros(2, 4, dtype=torch.float64, device="cuda"))
    refused(N.SHKV_ERR_INVALID_ARG, pool.chunk_attention, c.q(51, 4), [40, 11])          # more new tokens than cached
    refused(N.SHKV_ERR_UNSUPPORTED, pool.chunk_attention, c.q(2, 258), [1, 1])           # 129 heads a KV head
    wrong(pool.chunk_attention, c.q(3, 4), [1, 1])
    wrong(pool.chunk_attention, c.q(2, 4)[:, :, :32], [1, 1])
    no_errors(pool)
    assert pool.host_seq_lens().tolist() == [40, 10]
    for bad in (dict(page_size=8), dict(head_dim=96), dict(max_batch=1025)):
        a = dict(num_pages=4, page_size=16, num_kv_heads=1, head_dim=64, max_batch=1, max_pages_per_seq=4)
        refused(N.SHKV_ERR_UNSUPPORTED, QuantizedKVPool, **{**a, **bad})
    wrong(QuantizedKVPool, 4, 16, 1, 64, 1, 4, k_pages=torch.zeros(4, 1, 16, 64, device="cuda"))
    refused(N.SHKV_ERR_CAPACITY, QuantizedKVPool, 4, 16, 1, 64, 1, 4, initial_seq_lens=[65])


def test_table_of_codes_matches_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), TABLE, equal_nan=True)


# ---------------------------------------------------------------------------
# splits, joins and mixed batches
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("N_,hq,hkv,d,page", [(1, 16, 2, 128, 16), (3, 16, 2, 64, 32), (5, 16, 2, 128, 32), (8, 16, 2, 128, 16)])
def test_decode_of_long_split_requests(N_, hq, hkv, d, page):
    """Work ranges that open and close inside units, for every number of rows a kernel is built for (16 to 64)."""
    c = Cache([20011, 0, 7, 9001, 13120], hkv, d, page, seed=40 + N_)
    pool = c.pool()
    q = c.q(5, N_ * hq)
    out, lse = pool.decode_attention(q, N_, return_lse=True)
    no_errors(pool)
    check_decode(c, q, N_, d ** -0.5, out, lse)
    again, lse2 = pool.decode_attention(q, N_, return_lse=True)      # the join's counters are back at zero
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("small", [24, 3])
def test_chunk_of_few_tokens_beside_many(small):
    """Requests of a few new tokens beside large ones: many (a launch of their own) and few (none)."""
    lens, new = [700] * small + [900, 0, 5], [3] * small + [40, 0, 5]
    c = Cache(lens, 8, 128, 16, seed=44)
    pool = c.pool()
    q = c.q(sum(new), 32)
    out, lse = pool.chunk_attention(q, new, scale=0.05, return_lse=True)
    no_errors(pool)
    check_chunk(c, q, new, 0.05, out, lse)


@pytest.mark.parametrize("n", [70, 6])
def test_queries_that_are_no_numbers_stay_in_their_rows(n):
    """An infinity or a NaN in a query row makes that row NaN and no other; a row of zeros weighs all keys alike."""
    c = Cache([300], 1, 128, 16, seed=45)
    pool = c.pool()
    q = c.q(n, 2)
    q[1, 0, 5], q[2, 1, 127], q[3] = float("inf"), float("nan"), 0
    out, lse = pool.chunk_attention(q, [n], scale=0.05, return_lse=True)
    no_errors(pool)
    bad = torch.zeros(n, 2, dtype=torch.bool, device="cuda")
    bad[1, 0] = bad[2, 1] = True
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    q[1, 0], q[2, 1] = 0, 0
    k, v = c.rows(0)
    limit = (torch.arange(n, device="cuda") + 301 - n).repeat_interleave(2)
    o, e, to, te = attend(q.reshape(2 * n, -1), k[:, 0], v[:, 0], 0.05, limit)
    ok = ~bad.reshape(-1)
    check(out.reshape(2 * n, -1)[ok], o[ok], to[ok], "out")
    check(lse.reshape(-1)[ok], e[ok], te[ok], "lse")

def test_inputs_of_another_stream_may_be_dropped():
    """A call waits on its stream while its inputs are freed and their memory is asked for again elsewhere."""
    c = Cache([700, 90], 2, 128, 16, seed=46)
    pool = c.pool(lens=[690, 90])
    q0 = c.q(2, 16)
    kv0 = torch.randn(2, 10, 2, 128, generator=c.g).to(torch.bfloat16).cuda()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    pool.append_kv(kv0[0], kv0[1], [10, 0], start=[690, 90], stream=s)       # kernels loaded, workspace made
    pool.decode_attention(q0, 2, return_lse=True, stream=s)
    torch.full_like(q0, 7.0)
    pool.set_seq_lens([690, 90])
    q, k, v = q0.clone(), kv0[0].clone(), kv0[1].clone()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)                               # some 50 ms
    pool.append_kv(k, v, [10, 0], stream=s)
    out, lse = pool.decode_attention(q, 2, scale=0.05, return_lse=True, stream=s)
    del q, k, v
    others = [torch.full_like(t, 7.0) for t in (q0, kv0[0], kv0[1]) for _ in range(3)]
    torch.cuda.synchronize()
    no_errors(pool)
    del others
    got_k, got_v = pool.read_kv([690, 0], [10, 0])
    for got, src in ((got_k, kv0[0]), (got_v, kv0[1])):
        codes, sc = quantise(src.double().cpu().numpy())
        assert torch.equal(got.double().cpu(), dequantise(torch.from_numpy(codes), torch.from_numpy(sc)))
    check_decode(c, q0, 2, 0.05, out, lse)
