"""Shared by the tests of eviction by accumulated attention weight: seeded
caches and the definitions in 64 bits.

Tolerance of a mass.  A weight is w = exp(s - lse), s = scale <q, k>, of the lse
that the call was given:
  * s is a sum of D exact products accumulated in fp32 by the tensor core, whose
    additions may truncate: off by at most D * 2^-23 * scale * sum_d |q_d k_d|;
  * scale * log2(e) rounded, and its product with the sum: 2^-23 |s|;
  * lse * log2(e): constant and product rounded, 2^-23 |lse|;
  * their difference rounded, 2^-24 |s - lse|, all these relative to w; the
    exponential's own error, 2^-22; a w under 2^-126 may count as 0;
  * R weights added in fp32: R * 2^-24 of their sum;
  * decay * old + sum: a rounding of the product and one of the sum, 2^-24 each
    of its operand and of the result (decay itself is an fp32 number: 2^-24).
"""
import numpy as np
import torch

from cross_model_shared_gb300 import SharedKVPool


class Cache:
    """A bf16 pool of random rows with its block table; every slot is filled."""

    def __init__(self, lens, hkv, d, page, seed=0, spare=2, extra=1, big=2.0, device="cuda"):
        self.g = torch.Generator().manual_seed(seed)
        pages = [-(-n // page) for n in lens]
        num = sum(pages) + spare
        perm = torch.randperm(num, generator=self.g).tolist()
        self.table = torch.full((len(lens), max(pages + [1]) + extra), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = torch.tensor(perm[at: at + n], dtype=torch.int32)
            at += n
        self.free = perm[at:]
        self.lens, self.hkv, self.d, self.page, self.num, self.device = list(lens), hkv, d, page, num, device
        k = torch.randn(num, hkv, page, d, generator=self.g)
        k[..., ::16] *= big
        self.k = k.to(torch.bfloat16).to(device)
        self.v = torch.randn(num, hkv, page, d, generator=self.g).to(torch.bfloat16).to(device)

    def pool(self, lens=None, max_batch=None) -> SharedKVPool:
        p = SharedKVPool(self.num, self.page, self.hkv, self.d, max_batch=max_batch or len(self.lens),
                         max_pages_per_seq=self.table.shape[1], k_pages=self.k, v_pages=self.v,
                         initial_seq_lens=self.lens if lens is None else lens)
        p.block_table[: len(self.lens)].copy_(self.table)
        torch.cuda.synchronize()
        return p

    def randn(self, *shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=self.g).to(dtype).to(self.device)

    def mass(self, extra=0, batch=None):
        return torch.rand(batch or len(self.lens), self.hkv, max(self.lens + [1]) + extra,
                          generator=self.g).to(self.device)

    def rows(self, b, pages=None, table=None, n=None):
        """fp64 rows [hkv, n, d] of request b's K (or of `pages`)."""
        n = self.lens[b] if n is None else n
        table = self.table if table is None else table
        pos = torch.arange(n)
        page = table[b].cpu()[pos // self.page].long().to(self.device)
        return (self.k if pages is None else pages)[page, :, (pos % self.page).to(self.device)].double().transpose(0, 1)


def scores(q, k, scale, causal):
    """q [n, hq, d], k [hkv, L, d] -> fp64 scores [hkv, n * G, L] (-inf where
    unseen) and scale * sum |q k| of each."""
    n, hq, d = q.shape
    hkv, L = k.shape[:2]
    G = hq // hkv
    x = q.double().view(n, hkv, G, d).transpose(0, 1).reshape(hkv, n * G, d)
    s = scale * (x @ k.transpose(1, 2))
    a = abs(scale) * (x.abs() @ k.abs().transpose(1, 2))
    if causal:
        pos = torch.arange(L - n, L, device=q.device).repeat_interleave(G)
        unseen = torch.arange(L, device=q.device)[None] > pos[:, None]
        s = s.masked_fill(unseen, -np.inf)
        a = a.masked_fill(unseen, 0.0)
    return s, a


def lse_of(c: Cache, q, scale, causal):
    """fp32 log-sum-exps of q [B, n, hq, d]; -inf for requests of no token."""
    B, n, hq, _ = q.shape
    out = torch.full((B, n, hq), -np.inf, device=q.device)
    for b in range(B):
        if c.lens[b]:
            s, _ = scores(q[b], c.rows(b), scale, causal)
            out[b] = torch.logsumexp(s, -1).view(c.hkv, n, -1).transpose(0, 1).reshape(n, hq).float()
    return out


def check_mass(c: Cache, q, lse, scale, causal, decay, old, got, requests=None):
    """`got` against the definition, request by request; q [B, n, hq, d], lse
    [B, n, hq], old masses (None: none); what lies behind the lengths is not
    looked at."""
    B, n, hq, d = q.shape
    R = n * (hq // c.hkv)
    decay = float(np.float32(decay))
    for b in range(B) if requests is None else requests:
        L = c.lens[b]
        if not L:
            continue
        s, a = scores(q[b], c.rows(b), scale, causal)
        e = lse[b].double().view(n, c.hkv, hq // c.hkv).transpose(0, 1).reshape(c.hkv, R, 1)
        w = torch.where(torch.isneginf(e) | torch.isneginf(s), torch.zeros_like(s), torch.exp(s - e))
        rel = d * 2.0 ** -23 * a + 2.0 ** -23 * (s.abs() + e.abs()) + 2.0 ** -24 * (s - e).abs() + 2.0 ** -22
        total = w.sum(1)
        tol = torch.where(w > 0, w * rel, torch.zeros_like(w)).sum(1) + R * 2.0 ** -24 * total + R * 2.0 ** -126
        kept = torch.zeros_like(total)
        if old is not None and decay != 0:
            kept = decay * old[b, :, :L].double()
        want = kept + total
        tol = tol + 2.0 ** -24 * kept.abs() + 2.0 ** -24 * want.abs()
        off = (got[b, :, :L].double() - want).abs()
        bad = ~((off <= tol) | (torch.isnan(want) & torch.isnan(got[b, :, :L])))
        assert not bad.any(), (f"request {b}: {int(bad.sum())} of {bad.numel()} outside, worst "
                               f"{float((off / tol).nan_to_num().max()):.3g} of the tolerance at "
                               f"{tuple(int(i) for i in bad.nonzero()[0])}")


def selected(row, keep, sink, recent):
    """The positions kept of one row of masses (numpy fp32), from the definition."""
    L = len(row)
    if keep >= L:
        return np.arange(L)
    key = np.where(np.isnan(row), np.float32(np.inf), row)
    order = np.lexsort((np.arange(L), -key, ~np.isnan(row)))       # NaN first, then larger, then lower position
    always = (np.arange(L) < sink) | (np.arange(L) >= L - recent)
    chosen = np.flatnonzero(always)
    rest = order[~always[order]][: keep - len(chosen)]
    return np.sort(np.concatenate([chosen, rest]))


def check_selection(mass, lens, keep, sink, recent, index):
    m, got = mass.cpu().numpy(), index.cpu().numpy()
    for b, (L, k) in enumerate(zip(lens, keep)):
        for g in range(m.shape[1]):
            want = selected(m[b, g, :L], k, sink, recent)
            assert np.array_equal(got[b, g, : len(want)], want), (b, g)
            assert (got[b, g, len(want):] == -1).all(), (b, g)


def evicted(c: Cache, index, keep, new_table, lens=None, table=None):
    """(k pages, v pages) after the move, slot by slot; nothing else changed."""
    k, v = c.k.clone(), c.v.clone()
    lens = c.lens if lens is None else lens
    table = (c.table if table is None else table).cpu()
    new, index = new_table.cpu(), index.cpu()
    P = c.page
    for b, n in enumerate(keep):
        if n >= lens[b]:
            continue
        j = torch.arange(n)
        to = new[b][j // P].long()
        for g in range(c.hkv):
            i = index[b, g, :n].long()
            at = table[b][i // P].long()
            for pages, old in ((k, c.k), (v, c.v)):
                pages[to, g, j % P] = old[at, g, i % P]
    return k, v
