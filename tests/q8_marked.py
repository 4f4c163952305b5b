"""Caches whose marked tokens have a chosen weight and a chosen value scale: shared by the tests of how the
8-bit cache's attentions hold weights and values of very different magnitudes.

Every query has 8 in channel 0 and every key 0 there, but for the marked tokens, whose keys are 0 elsewhere:
a marked token's score is known exactly, the others' are those of the remaining channels, some 1 nat wide."""
import math

import torch

from .q8_common import Cache

SCALE = 0.75
Q0 = 8.0
OTHERS_K = 116                           # scale byte of the other tokens' keys: scores of about 0.5 nats
UNIT = SCALE * Q0 * math.log2(math.e)    # bits of score of a key of 1 in channel 0


def marked(lens, marks, hkv, d, page, seed, v_byte=127, common=True):
    """marks: {(request, token): (bits of score above 0, V scale byte, the V row's codes or None)}."""
    c = Cache(lens, hkv, d, page, seed=seed)
    c.sc[:, :, 0], c.sc[:, :, 1] = OTHERS_K, v_byte
    c.k[:, :, :, 0] = 0
    if common:                           # a common part in every V: errors of one sign add up
        v = torch.randn(c.v.shape, generator=c.g).mul_(60).add_(150).clamp_(-448, 448)
        c.v.copy_(v.to(torch.float8_e4m3fn).view(torch.uint8))
    for (b, t), (bits, byte, codes) in marks.items():
        p, s = int(c.table[b, t // page]), t % page
        m, e = math.frexp(abs(bits) / UNIT)          # |bits| = m * 2^e * UNIT, 16 steps of m
        code = torch.tensor(m * 256).to(torch.float8_e4m3fn).view(torch.uint8)
        c.k[p, :, s] = 0
        c.k[p, :, s, 0] = int(code) | (0x80 if bits < 0 else 0)
        c.sc[p, :, 0, s] = 127 + e - 8
        c.sc[p, :, 1, s] = byte
        if codes is not None:
            c.v[p, :, s] = codes
    return c


def queries(c, *shape):
    q = c.q(*shape)
    q[..., 0] = Q0
    return q


def share(c, copies):
    """The cache with its requests repeated: the copies read the same pages."""
    c.lens, c.table = c.lens * copies, c.table.repeat(copies, 1)
    return c
