"""Shared by the tests of the 8-bit KV cache: the format and the attention written
out from their definitions in 64 bits (numpy and torch, on the CPU for the
format), pools filled with seeded data, and the tolerance.

Tolerance of an attention output.  With p the exact softmax weights,
A = sum_t p_t |v_t| and L keys:
  * the weights are rounded to fp16 for the product with V: 2^-11 A;
  * a score is a dot product of D terms accumulated in fp32, of a query held
    to 2^-18 of its row's maximum: it is off by at most
    ds = scale * (D * 2^-24 + 2^-18) * max|q| * max_t sum_d |k_td|, a weight by
    2 ds of itself (numerator and sum), so 2 ds A;
  * sums over the keys in fp32: L * 2^-24 A, and 2^-18 A for the exponentials,
    the running maximum's rescaling and the join of pieces;
  * a weight under 2^-126 of the row's largest is no normal fp32 number and may
    count as zero: sum_t 2^-126 |v_t| (it matters only beside values 2^100 larger);
  * one rounding to bf16: half a step, 2^-8 of the value.
The log-sum-exp is off by ds + L * 2^-24 + 2^-18 and its own fp32 rounding.
"""
import numpy as np
import torch

from cross_model_shared_gb300 import QuantizedKVPool

E4M3_MAX = 448.0


def e4m3_table() -> np.ndarray:
    out = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = np.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        out[code] = -x if code >> 7 else x
    return out


TABLE = e4m3_table()


def quantise(x: np.ndarray):
    """Codes and scale bytes of fp64 rows [..., D], by search among the 127 non-negative codes."""
    rows = x.reshape(-1, x.shape[-1])
    codes = np.empty(rows.shape, np.uint8)
    scales = np.empty(len(rows), np.uint8)
    pos = TABLE[:127]                                       # 0 .. 448, increasing
    for i, r in enumerate(rows):
        big = np.abs(r).max()
        if not np.isfinite(big):
            codes[i], scales[i] = 0x7F, 255
            continue
        e = -127
        while big > np.ldexp(E4M3_MAX, e):
            e += 1
        y = np.abs(np.ldexp(r, -e))
        hi = np.searchsorted(pos, y).clip(1, 126)
        lo = hi - 1
        up, down = pos[hi] - y, y - pos[lo]
        pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
        codes[i] = pick | (np.signbit(r).astype(np.uint8) << 7)
        scales[i] = e + 127
    return codes.reshape(x.shape), scales.reshape(x.shape[:-1])


def dequantise(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """fp64 values of codes [..., D] with scale bytes [...]."""
    table = torch.from_numpy(TABLE).to(codes.device)
    power = torch.tensor([np.ldexp(1.0, i - 127) for i in range(255)] + [np.nan], dtype=torch.float64,
                         device=codes.device)
    return table[codes.long()] * power[scales.long()][..., None]


class Cache:
    """A pool of random codes and scales with its block table, and what it stands for."""

    def __init__(self, lens, hkv, d, page, seed=0, spare=2, extra=1, scale_lo=117, scale_hi=123, device="cuda"):
        g = torch.Generator(device="cpu").manual_seed(seed)
        pages = [-(-n // page) for n in lens]
        num = sum(pages) + spare
        perm = torch.randperm(num, generator=g).tolist()
        self.table = torch.full((len(lens), max(pages + [1]) + extra), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = torch.tensor(perm[at: at + n], dtype=torch.int32)
            at += n
        self.lens, self.hkv, self.d, self.page, self.num = list(lens), hkv, d, page, num
        # every slot is filled, those behind a request's last token too; no NaN codes
        shape = (num, hkv, page, d)
        draw = lambda: torch.randn(shape, generator=g).mul_(120).clamp_(-448, 448)     # noqa: E731
        self.k = draw().to(torch.float8_e4m3fn).view(torch.uint8).to(device)
        self.v = draw().to(torch.float8_e4m3fn).view(torch.uint8).to(device)
        self.sc = torch.randint(scale_lo, scale_hi + 1, (num, hkv, 2, page), generator=g, dtype=torch.uint8).to(device)
        self.g, self.device = g, device

    def pool(self, lens=None, max_batch=None) -> QuantizedKVPool:
        p = QuantizedKVPool(self.num, self.page, self.hkv, self.d, max_batch=max_batch or len(self.lens),
                            max_pages_per_seq=self.table.shape[1], k_pages=self.k, v_pages=self.v, scales=self.sc,
                            initial_seq_lens=self.lens if lens is None else lens)
        p.block_table[: len(self.lens)].copy_(self.table)
        torch.cuda.synchronize()
        return p

    def q(self, *shape):
        return torch.randn(*shape, self.d, generator=self.g).to(torch.bfloat16).to(self.device)

    def rows(self, b, n=None):
        """fp64 K, V [n, hkv, d] of request b."""
        n = self.lens[b] if n is None else n
        pos = torch.arange(n)
        page = self.table[b, pos // self.page].long().to(self.device)
        slot = (pos % self.page).to(self.device)
        return (dequantise(self.k[page, :, slot], self.sc[page, :, 0, slot]),
                dequantise(self.v[page, :, slot], self.sc[page, :, 1, slot]))


def attend(q, k, v, scale, limit=None):
    """fp64 attention of q [rows, d] over k, v [L, d]; row r sees the keys below
    limit[r].  Returns (out, lse, tolerance of out, tolerance of lse)."""
    q = q.double()
    L, d = k.shape
    x = scale * (q @ k.T)
    if limit is not None:
        x = x.masked_fill(torch.arange(L, device=x.device)[None] >= limit[:, None], -np.inf)
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    out = p @ v
    ds = abs(scale) * (d * 2.0 ** -24 + 2.0 ** -18) * q.abs().amax(1) * k.abs().sum(1).max()
    a = p @ v.abs()
    tol = a * (2.0 ** -11 + 2 * ds[:, None] + L * 2.0 ** -24 + 2.0 ** -18) + out.abs() * 2.0 ** -8
    tol = tol + 2.0 ** -126 * v.abs().sum(0)
    return out, lse, tol, ds + L * 2.0 ** -24 + 2.0 ** -18 + lse.abs() * 2.0 ** -23


def check(got, want, tol, what):
    off = (got.double() - want).abs()
    bad = ~(off <= tol + 1e-300)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((off / tol).nan_to_num().max()):.3g} of the tolerance at "
                           f"{tuple(int(i) for i in bad.nonzero()[0])}")


def check_decode(c: Cache, q, n_models, scale, out, lse, requests=None):
    B, rows, d = q.shape
    hq = rows // n_models
    g = hq // c.hkv
    for b in range(B) if requests is None else requests:
        if c.lens[b] == 0:
            assert not out[b].any() and torch.isneginf(lse[b]).all()
            continue
        k, v = c.rows(b)
        for h in range(c.hkv):
            r = torch.tensor([m * hq + h * g + j for m in range(n_models) for j in range(g)], device=q.device)
            o, e, to, te = attend(q[b, r], k[:, h], v[:, h], scale)
            check(out[b, r], o, to, f"out of request {b}, head {h}")
            check(lse[b, r], e, te, f"lse of request {b}, head {h}")


def check_chunk(c: Cache, q, new, scale, out, lse):
    hq = q.shape[1]
    g = hq // c.hkv
    at = 0
    for b, n in enumerate(new):
        if n:
            k, v = c.rows(b)
            limit = (torch.arange(n, device=q.device) + c.lens[b] - n + 1).repeat_interleave(g)
            for h in range(c.hkv):
                s = slice(h * g, (h + 1) * g)
                o, e, to, te = attend(q[at: at + n, s].reshape(n * g, -1), k[:, h], v[:, h], scale, limit)
                check(out[at: at + n, s].reshape(n * g, -1), o, to, f"out of request {b}, head {h}")
                check(lse[at: at + n, s].reshape(-1), e, te, f"lse of request {b}, head {h}")
        at += n
