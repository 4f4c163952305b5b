"""Weights and values of very different magnitudes in the 8-bit cache's attentions, against 64 bits."""
import numpy as np
import pytest
import torch

from cross_model_shared_gb300 import _native as N

from .q8_common import attend, check, check_chunk, check_decode
from .q8_marked import SCALE, marked, queries, share

pytestmark = pytest.mark.gpu


def chunk_some(c, new, hq, requests, heads):
    """Chunk attention of the whole batch, checked at some requests and KV heads."""
    pool = c.pool()
    q = queries(c, sum(new), hq)
    out, lse = pool.chunk_attention(q, new, scale=SCALE, return_lse=True)
    assert pool.check_errors() == 0
    g = hq // c.hkv
    for b in requests:
        n, at = new[b], sum(new[:b])
        k, v = c.rows(b)
        limit = (torch.arange(n, device="cuda") + c.lens[b] - n + 1).repeat_interleave(g)
        for h in heads:
            s = slice(h * g, h * g + g)
            o, e, to, te = attend(q[at: at + n, s].reshape(n * g, -1), k[:, h], v[:, h], SCALE, limit)
            check(out[at: at + n, s].reshape(n * g, -1), o, to, f"out of request {b}, head {h}")
            check(lse[at: at + n, s].reshape(-1), e, te, f"lse of request {b}, head {h}")


@pytest.mark.parametrize("below", [8, 10, 12, 14])
@pytest.mark.parametrize("L", [16384, 65536])
def test_chunk_keeps_tokens_far_below_a_key_of_small_value(L, below):
    """A first key 2^32 above the others, with a value 2^-below of theirs: the others are a part of the sum."""
    c = marked([L], {(0, 0): (32.0, 127 - below, 0x78)}, 1, 128, 16, seed=50 + below)
    chunk_some(c, [128], 8, [0], [0])


@pytest.mark.parametrize("L,below", [(16384, 8), (16384, 10), (16384, 12), (16384, 14), (65536, 8), (65536, 12)])
def test_whole_units_keep_them_too(L, below):
    """As above with more units than work ranges: most are not split."""
    c = share(marked([L], {(0, 0): (32.0, 127 - below, 0x78)}, 8, 128, 32, seed=60), 40)
    chunk_some(c, [64] * 40, 32, [0, 23, 39], [0, 5])


@pytest.mark.parametrize("bits", [28.0, 44.0, 58.0, 88.0])
@pytest.mark.parametrize("L,new", [(300, 128), (6000, 64)])
def test_chunk_beside_a_leading_key_without_value(L, new, bits):
    """A V row of zeros whose key leads by up to 61 nats: all of the output is the others'."""
    c = marked([L, L], {(0, 3): (bits, 0, 0), (1, 0): (bits, 0, 0x80)}, 2, 128, 16, seed=70)
    chunk_some(c, [new, new], 8, [0, 1], [0, 1])


@pytest.mark.parametrize("byte", [241, 244, 247])
@pytest.mark.parametrize("L,new", [(300, 128), (6000, 64)])
def test_chunk_of_the_largest_values(L, new, byte):
    """Outputs up to bf16's largest, beside values 2^100 and more below: finite where the sum is."""
    c = marked([L, L], {(0, 5): (40.0, byte, 0x77), (1, L - 150): (12.0, byte, 0xF7)}, 2, 128, 16, seed=71,
               v_byte=100)
    chunk_some(c, [new, new], 8, [0, 1], [0, 1])


@pytest.mark.parametrize("new", [2, 16, 128])
@pytest.mark.parametrize("v_byte", [0, 3, 60, 200])
def test_values_of_one_magnitude_anywhere(new, v_byte):
    """Caches whose values are all tiny (rows of the least scale, some of them zero) or all huge."""
    c = marked([400, 3000], {(0, 3): (10.0, v_byte, None)}, 2, 64, 32, seed=74, v_byte=v_byte)
    c.v[:, :, 7] = 0
    pool = c.pool()
    q = queries(c, 2 * new, 8)
    out, lse = pool.chunk_attention(q, [new, new], scale=SCALE, return_lse=True)
    assert pool.check_errors() == 0
    check_chunk(c, q, [new, new], SCALE, out, lse)


@pytest.mark.parametrize("new", [4, 64])
def test_split_units_of_the_largest_values(new):
    """Pieces whose outputs are all near bf16's largest are joined without an overflow."""
    c = marked([20000], {}, 1, 128, 16, seed=76, v_byte=247)
    c.v[:] = torch.where(torch.arange(128, device="cuda") % 3 == 0, 0xF7, 0x77).to(torch.uint8)
    chunk_some(c, [new], 8, [0], [0])


ROWS = [(1, 16, 2), (3, 16, 2), (5, 16, 2), (8, 16, 2)]      # 8, 24, 40 and 64 rows a KV head


@pytest.mark.parametrize("N_,hq,hkv", ROWS)
@pytest.mark.parametrize("bits,above", [(-30.0, 44), (-60.0, 52), (-72.0, 60), (-88.0, 70), (-100.0, 70), (-120.0, 100)])
def test_decode_beside_a_large_value_of_little_weight(N_, hq, hkv, bits, above):
    """A token's value is far above the others' and its weight farther below: the output is the others'."""
    lens = [700, 9000, 260]
    c = marked(lens, {(b, lens[b] // 2): (bits, 127 + above, None) for b in range(3)}, hkv, 128, 16, seed=72)
    pool = c.pool()
    q = queries(c, 3, N_ * hq)
    out, lse = pool.decode_attention(q, N_, scale=SCALE, return_lse=True)
    assert pool.check_errors() == 0
    check_decode(c, q, N_, SCALE, out, lse)


@pytest.mark.parametrize("N_,hq,hkv", ROWS)
@pytest.mark.parametrize("bits", [28.0, 58.0, 80.0])
def test_decode_beside_a_leading_key_without_value(N_, hq, hkv, bits):
    lens = [700, 9000, 260]
    c = marked(lens, {(0, 5): (bits, 0, 0), (1, 4000): (bits, 0, 0x80), (2, 259): (bits, 0, 0)}, hkv, 128, 16, seed=73)
    pool = c.pool()
    q = queries(c, 3, N_ * hq)
    out, lse = pool.decode_attention(q, N_, scale=SCALE, return_lse=True)
    assert pool.check_errors() == 0
    check_decode(c, q, N_, SCALE, out, lse)


# (scale byte of the others' V, bits of the marked token's score, its byte): the reference of P rises by 2^126 and more
# while the others keep a part of the weights
RISES = [(127, 10.0, 247), (127, 20.0, 240), (87, 5.0, 247), (70, 18.0, 180), (68, 8.0, 187), (20, 3.0, 150), (5, 0.0, 247)]


@pytest.mark.parametrize("N_,hq,hkv", ROWS)
@pytest.mark.parametrize("v_byte,bits,byte", RISES)
def test_decode_keeps_the_weights_before_a_value_of_far_larger_scale(N_, hq, hkv, v_byte, bits, byte):
    lens = [700, 9000, 260]
    marks = {(b, n * 2 // 3): (bits, byte, 0x70) for b, n in enumerate(lens)}
    c = marked(lens, marks, hkv, 128, 16, seed=77, v_byte=v_byte)
    pool = c.pool()
    q = queries(c, 3, N_ * hq)
    out, lse = pool.decode_attention(q, N_, scale=SCALE, return_lse=True)
    assert pool.check_errors() == 0
    check_decode(c, q, N_, SCALE, out, lse)


@pytest.mark.parametrize("v_byte,bits,byte", RISES)
@pytest.mark.parametrize("copies", [1, 160])
def test_chunk_keeps_the_weights_before_a_value_of_far_larger_scale(v_byte, bits, byte, copies):
    """160 requests of one unit each: none is split."""
    c = share(marked([9000], {(0, 6000): (bits, byte, 0x70)}, 1, 128, 16, seed=78, v_byte=v_byte), copies)
    chunk_some(c, [32] * copies, 8, [0, copies - 1], [0])


# scale bytes of V, with the codes of the row (0: a zero row)
KINDS = [(0, 0), (0, 0), (0, 0x78), (5, 0x78), (60, 0xF8), (80, 0x78), (100, 0x78), (127, 0xF8), (150, 0x78), (170, 0x78),
         (200, 0xF8), (240, 0x78)]


def mixed(lens, hkv, seed, kinds, most, v_byte=127):
    g = torch.Generator().manual_seed(seed)
    draw = lambda n: int(torch.randint(n, (1,), generator=g))               # noqa: E731
    marks = {}
    for b, n in enumerate(lens):
        for _ in range(8):
            byte, code = kinds[draw(len(kinds))]
            bits = draw(2 * most) - most + 0.5
            marks[b, draw(n) if draw(3) else min(draw(3), n - 1)] = (bits, byte, code)
    return marked(lens, marks, hkv, 128, 16, seed=seed, v_byte=v_byte)


@pytest.mark.parametrize("N_,hq,hkv", ROWS)
@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("kinds,most", [(KINDS, 100), (KINDS[:2], 70), (KINDS[:6], 45), (KINDS[5:9], 100)])
def test_decode_of_weights_and_values_of_all_magnitudes(N_, hq, hkv, seed, kinds, most):
    """Zero rows, rows of tiny and of huge values with weights far above and below the others', anywhere."""
    lens = [700, 9000, 260, 64, 1500]
    c = mixed(lens, hkv, 100 + seed, kinds, most)
    pool = c.pool()
    q = queries(c, len(lens), N_ * hq)
    out, lse = pool.decode_attention(q, N_, scale=SCALE, return_lse=True)
    assert pool.check_errors() == 0
    check_decode(c, q, N_, SCALE, out, lse)


@pytest.mark.parametrize("n", [3, 7, 70, 200])
@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("kinds,most", [(KINDS, 100), (KINDS[:2], 70), (KINDS[:6], 45), (KINDS[5:9], 100)])
def test_chunks_of_weights_and_values_of_all_magnitudes(n, seed, kinds, most):
    lens, new = [700, 5000, 260, 1500], [n, n // 2, n, n]
    c = mixed(lens, 2, 200 + seed, kinds, most)
    pool = c.pool()
    q = queries(c, sum(new), 16)
    out, lse = pool.chunk_attention(q, new, scale=SCALE, return_lse=True)
    assert pool.check_errors() == 0
    check_chunk(c, q, new, SCALE, out, lse)


@pytest.mark.parametrize("new", [3, 100])
def test_queries_with_large_channels(new):
    """Query channels 2^13 apart (massive activations): the small ones are held to 2^-17.8 of the largest, as the
    tolerance has it for every query."""
    c = marked([2000], {}, 2, 128, 16, seed=75)
    q = queries(c, new, 8)
    q[..., 17] = 8192.0
    q[..., 40] = -3000.0
    c.k[..., 17] = 0x08                  # 2^-6: its product with the large channel is of ordinary size
    c.k[..., 40] = 0
    pool = c.pool()
    out, lse = pool.chunk_attention(q, [new], scale=0.1, return_lse=True)
    assert pool.check_errors() == 0
    check_chunk(c, q, [new], 0.1, out, lse)


@pytest.mark.parametrize("scale", [2.4e38, -3e38, float("nan"), float("-inf")])
def test_a_scale_that_leaves_fp32_in_bits_is_refused(scale):
    c = marked([40], {}, 1, 64, 16, seed=2)
    pool = c.pool()
    for call in (lambda: pool.decode_attention(c.q(1, 2), 1, scale=scale),
                 lambda: pool.chunk_attention(c.q(4, 2), [4], scale=scale)):
        with pytest.raises(N.ShkvError) as e:
            call()
        assert e.value.status == N.SHKV_ERR_INVALID_ARG


def test_marked_scores_are_what_they_say():
    c = marked([40], {(0, 7): (32.0, 120, None), (0, 9): (-60.0, 127, None)}, 1, 64, 16, seed=1)
    k, _ = c.rows(0)
    bits = (k[:, 0, 0] * 8.0 * SCALE * np.log2(np.e)).cpu()
    assert abs(bits[7] / 32 - 1) <= 2.0 ** -4 and abs(bits[9] / -60 - 1) <= 2.0 ** -4
    assert not bits[[i for i in range(40) if i not in (7, 9)]].any()
