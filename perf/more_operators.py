"""Measured cases of the shared KV cache's eviction by accumulated attention weight.

A cache that only grows runs out of pages.  Four operators let it shrink to the tokens that its readers attend to:

* decode_mass:   add to every cached token's mass the softmax weights that the stacked rows of one decode step gave it;
* prefill_mass:  the same for the causal softmax of a chunk of new tokens, or of a window of its last ones;
* select_tokens: for every request and KV head the tokens of most mass, with the first and the last ones always;
* evict_tokens:  move the selected tokens' K, V and mass into new pages, and the request to them.

`own` chooses what `run` computes with: False, plain torch operations in 32 bits; True, the framework's kernels.
"""
import math
import random

import torch

own = False


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # the tiny configuration: one request, two decoders; latency
        dict(name="decode mass tiny", op="decode", B=1, N=2, hq=8, hkv=2, d=64, page=16, lo=256, hi=256, decay=1.0,
             empty=0, lens_seed=1),
        # two decoders over a batch of ordinary contexts
        dict(name="decode mass 8 rows", op="decode", B=32, N=2, hq=32, hkv=8, d=128, page=16, lo=1024, hi=8192,
             decay=1.0, empty=1, lens_seed=2),
        # eight decoders, long mixed contexts, 40 stacked rows per KV head, masses that fade
        dict(name="decode mass 40 rows", op="decode", B=24, N=8, hq=40, hkv=8, d=128, page=32, lo=4096, hi=65536,
             decay=0.98, empty=0, lens_seed=3),
        # the last tokens of prompts of many lengths vote on what to keep
        dict(name="prefill mass window", op="prefill", B=16, n=32, of=64, hq=32, hkv=8, d=128, page=16, lo=900,
             hi=15000, decay=0.0, empty=0, lens_seed=4),
        # one long document extended by one chunk, every new token counted
        dict(name="prefill mass document", op="prefill", B=1, n=2048, of=2048, hq=40, hkv=8, d=128, page=32, lo=40000,
             hi=40000, decay=1.0, empty=0, lens_seed=5),
        # whole prompts of a small model with 64-wide heads and an odd group
        dict(name="prefill mass prompts", op="prefill", B=5, n=777, of=777, hq=14, hkv=2, d=64, page=16, lo=777,
             hi=1900, decay=1.0, empty=0, lens_seed=6),
        # one short session over its budget; latency
        dict(name="select short", op="select", B=1, hkv=2, lo=300, hi=300, keep=0.5, sink=4, recent=32, empty=0,
             lens_seed=7),
        # a serving batch shrinks to a quarter
        dict(name="select batch", op="select", B=64, hkv=8, lo=1024, hi=8192, keep=0.25, sink=4, recent=128, empty=1,
             lens_seed=8),
        # four very long contexts
        dict(name="select long", op="select", B=4, hkv=8, lo=131584, hi=131584, keep=0.125, sink=16, recent=1024,
             empty=0, lens_seed=9),
        # one short session over its budget; latency
        dict(name="evict short", op="evict", B=1, hkv=2, d=64, page=16, lo=300, hi=300, keep=0.5, sink=4, recent=32,
             empty=0, lens_seed=10),
        # a serving batch shrinks to half; some requests are within their budget and stay
        dict(name="evict batch", op="evict", B=48, hkv=8, d=128, page=16, lo=700, hi=8192, keep=0.5, sink=4,
             recent=128, empty=1, lens_seed=11),
        # long sessions shrink to a quarter
        dict(name="evict long", op="evict", B=4, hkv=8, d=128, page=32, lo=65536, hi=131584, keep=0.25, sink=16,
             recent=1024, empty=0, lens_seed=12),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "prefill", "select", "evict"])
    hkv = rng.choice([1, 2, 4, 8])
    B = _log_uniform(rng, 1, 64)
    c = dict(op=op, B=B, hkv=hkv, empty=rng.choice([0, 0, 0, 1]) if B > 1 else 0, lens_seed=rng.randrange(1 << 30))
    if op != "select":
        c["d"], c["page"] = rng.choice([64, 128, 128]), rng.choice([16, 32])
    if op in ("select", "evict"):
        c["hi"] = _log_uniform(rng, 100, max(100, min(131072, 250000 // B)))
        c["lo"] = max(60, c["hi"] // 8)
        c["keep"] = rng.choice([0.05, 0.1, 0.25, 0.5, 0.75, 0.9])
        c["sink"] = rng.choice([0, 1, 4, 16])
        c["recent"] = _log_uniform(rng, 1, max(2, c["hi"] // 32))
        return c
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    c["hq"] = g * hkv
    c["decay"] = rng.choice([0.0, 0.9, 1.0])
    if op == "decode":
        c["N"] = rng.choice([n for n in (1, 2, 3, 4, 5, 8) if n * g <= 64])
        c["lo"], c["hi"] = 1, _log_uniform(rng, 16, max(64, min(131072, 400000 // B)))
    else:
        pairs = 3 * 10 ** 9 // (B * c["hq"])               # of a new and a cached token, for one head of one request
        c["n"] = _log_uniform(rng, 1, max(1, min(8000 // B, int(math.sqrt(pairs / 2)))))
        c["of"] = c["n"] + rng.choice([0, 0, 1, 64])
        c["lo"] = c["of"]
        c["hi"] = c["of"] + _log_uniform(rng, 1, max(1, min(50000 // B, pairs // c["n"] - c["of"])))
    return c


def _lengths(case):
    """(cached tokens, kept tokens) of each request."""
    rng = random.Random(case["lens_seed"])
    total = [_log_uniform(rng, case["lo"], case["hi"]) for _ in range(case["B"])]
    if case["empty"]:
        total[-1] = case["lo"] if case["op"] == "prefill" else 0
    if case["op"] not in ("select", "evict"):
        return total, None
    # at least the tokens that always stay; a request within that budget is left as it is
    least = case["sink"] + case["recent"]
    return total, [max(least, int(case["keep"] * L)) if b % 8 != 5 else L for b, L in enumerate(total)]


def _moved(case):
    """(length, kept) of the requests that are over their budget."""
    total, keep = _lengths(case)
    return [(L, k) for L, k in zip(total, keep) if k < L]


def work(case):
    hkv, op = case["hkv"], case["op"]
    total, keep = _lengths(case)
    if op == "select":
        kept = sum(min(k, L) for k, L in zip(keep, total))
        return {"bytes": 4 * hkv * (sum(L for L, _ in _moved(case)) + kept), "flops": hkv * sum(total)}
    d = case["d"]
    if op == "evict":
        moved = _moved(case)
        kept = sum(k for _, k in moved)
        return {"bytes": hkv * (kept * (8 * d + 8) + 4 * sum(L for L, _ in moved)), "flops": 0}
    cached = sum(total)
    old = 4 if case["decay"] else 0
    if op == "decode":
        rows = case["N"] * case["hq"]
        return {"bytes": cached * hkv * (2 * d + 4 + old) + case["B"] * rows * (2 * d + 4),
                "flops": 2 * d * rows * cached}
    n, hq = case["n"], case["hq"]
    seen = sum(n * (L - n) + n * (n + 1) // 2 for L in total)
    return {"bytes": cached * hkv * (2 * d + 4 + old) + case["B"] * n * hq * (2 * d + 4), "flops": 2 * d * hq * seen}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _table(rng, total, page, spare):
    """A table of distinct pages in no order, [B, most pages + 2], and the ids left over."""
    pages = [-(-n // page) for n in total]
    ids = list(range(sum(pages) + spare))
    rng.shuffle(ids)
    table = torch.full((len(total), max(pages) + 2), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.tensor(ids[at: at + n], dtype=torch.int32)
        at += n
    return table, ids[at:], len(ids)


def _mass(g, B, hkv, T):
    """Masses as attention leaves them: over many octaves, most tokens next to nothing, and many of exactly nothing."""
    m = torch.exp(2.5 * _randn(g, B, hkv, T) - 4.0)
    m[torch.rand(B, hkv, T, generator=g, device="cuda") < 0.05] = 0.0
    return m


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    total, keep = _lengths(case)
    B, hkv, op = case["B"], case["hkv"], case["op"]
    s = dict(case=case, total=total, keep=keep, width=max(max(total), 1))
    s["mass"] = _mass(g, B, hkv, s["width"] + 3)
    if keep is not None:
        s["most"] = max(max(min(k, L) for k, L in zip(keep, total)), 1)
    if op == "select":
        return s
    d, P = case["d"], case["page"]
    rng = random.Random(int(seed))
    spare = 3 if op != "evict" else 3 + sum(-(-k // P) for _, k in _moved(case))
    table, left, num = _table(rng, total, P, spare)
    s.update(num_pages=num, table=table.cuda(), scale=1 / math.sqrt(d))
    k = torch.empty(num, hkv, P, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    step = max(1, (1 << 25) // (P * hkv * d))
    for i in range(0, num, step):          # every slot holds a value, those behind the last token too
        n = min(step, num - i)
        x = _randn(g, n, hkv, P, d)
        x[..., :: d // 4] *= 2.0           # a few large channels
        k[i: i + n] = x
        v[i: i + n] = _randn(g, n, hkv, P, d)
    s.update(k=k, v=v)
    if op == "evict":
        # what a selection left: ascending positions, random apart from the first and the last
        new = torch.full((B, max(1, max((-(-n // P) for _, n in _moved(case)), default=1))), -1, dtype=torch.int32)
        index = torch.full((B, hkv, s["most"]), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, (L, n) in enumerate(zip(total, keep)):
            n = min(n, L)
            noise = torch.rand(hkv, L, generator=g, device="cuda")
            noise[:, : case["sink"]] = 2.0
            noise[:, max(0, L - case["recent"]):] = 2.0
            index[b, :, :n] = torch.sort(torch.topk(noise, n, dim=1).indices, 1).values.int()
            if n < L:
                pages = -(-n // P)
                new[b, :pages] = torch.tensor(left[at: at + pages], dtype=torch.int32)
                at += pages
        s.update(index=index, new=new.cuda())
        return s
    if op == "decode":
        s["q"] = _randn(g, B, case["N"] * case["hq"], d).to(torch.bfloat16)
        s["lse"] = _lse(s, s["q"].view(B, case["N"], case["hq"], d), False).view(B, -1)
    else:                                  # the window's queries are the last of a chunk's
        n = case["n"]
        q = _randn(g, B, case["of"], case["hq"], d).to(torch.bfloat16)[:, case["of"] - n:]
        lse = torch.zeros(B, case["of"], case["hq"], device="cuda")[:, case["of"] - n:]
        lse.copy_(_lse(s, q, True))
        s.update(q=q, lse=lse)
    return s


def _keys(s, b):
    """K of request b in fp32, [hkv, L, d]."""
    c, L = s["case"], s["total"][b]
    ids = s["table"][b, : -(-L // c["page"])].long()
    return s["k"][ids].float().transpose(0, 1).reshape(c["hkv"], -1, c["d"])[:, :L]


def _scores(s, q, b, i, w, causal, k):
    """Scores of query tokens i .. i + w - 1 of request b, fp32 [hkv, w * G, L]; what a row does not see is -inf."""
    c, n = s["case"], q.shape[1]
    G, L = c["hq"] // c["hkv"], s["total"][b]
    x = q[b, i: i + w].float().view(w, c["hkv"], G, -1).permute(1, 0, 2, 3).reshape(c["hkv"], w * G, -1)
    x = torch.matmul(x, k.transpose(1, 2)) * s["scale"]
    if causal:
        pos = torch.arange(L - n + i, L - n + i + w, device="cuda").repeat_interleave(G)
        x = x.masked_fill(torch.arange(L, device="cuda")[None, :] > pos[:, None], float("-inf"))
    return x


def _lse(s, q, causal, rows=256):
    """The log-sum-exps that an attention call over the same queries returned, [B, n, hq]."""
    c, n = s["case"], q.shape[1]
    G = c["hq"] // c["hkv"]
    out = torch.full(q.shape[:3], float("-inf"), device="cuda")
    for b in range(c["B"]):
        if s["total"][b] == 0:
            continue
        k = _keys(s, b)
        for i in range(0, n, rows):
            w = min(rows, n - i)
            e = torch.logsumexp(_scores(s, q, b, i, w, causal, k), -1)
            out[b, i: i + w] = e.view(c["hkv"], w, G).transpose(0, 1).reshape(w, -1)
    return out


def prepare(case, seed):
    s = _inputs(case, seed)
    total, B = s["total"], case["B"]
    s["out"] = torch.zeros_like(s["mass"])
    if case["op"] == "evict":
        s["lens"] = torch.tensor(total, dtype=torch.int32, device="cuda")
        s["now"] = s["table"].clone()
    if own:
        from cross_model_shared_gb300 import SharedKVPool
        if case["op"] == "select":         # a selection needs no pages, only the lengths
            pool = SharedKVPool(1, 16, case["hkv"], 128, max_batch=B, max_pages_per_seq=-(-s["width"] // 16),
                                initial_seq_lens=total)
        else:
            pool = SharedKVPool(s["num_pages"], case["page"], case["hkv"], case["d"], max_batch=B,
                                max_pages_per_seq=s["table"].shape[1], k_pages=s["k"], v_pages=s["v"],
                                initial_seq_lens=total)
            pool.block_table.copy_(s["table"])
        s["pool"] = pool
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        pool = s["pool"]
        if op == "decode":
            return pool.decode_mass(s["q"], s["lse"], c["N"], s["mass"], decay=c["decay"], scale=s["scale"],
                                    out=s["out"])
        if op == "prefill":
            return pool.prefill_mass(s["q"], s["lse"], s["mass"], decay=c["decay"], scale=s["scale"], out=s["out"])
        if op == "select":
            return pool.select_tokens(s["mass"], s["keep"], sink=c["sink"], recent=c["recent"])
        # from the table and lengths that a user's program keeps beside the pool's own
        pool.evict_tokens(s["index"], s["keep"], s["new"], mass=s["mass"], out=s["out"],
                          source=(s["table"], s["total"]))
        return s["k"], s["v"], pool.block_table, pool.seq_lens, s["out"]
    return {"decode": _plain_decode, "prefill": _plain_prefill, "select": _plain_select, "evict": _plain_evict}[op](s)


def _plain_sums(s, q, causal, rows=256):
    c, n = s["case"], q.shape[1]
    G = c["hq"] // c["hkv"]
    lse = s["lse"].reshape(c["B"], n, c["hkv"], G)
    for b in range(c["B"]):
        L = s["total"][b]
        if L == 0:
            continue
        k = _keys(s, b)
        total = torch.zeros(c["hkv"], L, device="cuda")
        for i in range(0, n, rows):        # blocks of query tokens, to bound the scores' size
            w = min(rows, n - i)
            e = lse[b, i: i + w].transpose(0, 1).reshape(c["hkv"], w * G)
            total += torch.exp(_scores(s, q, b, i, w, causal, k) - e[..., None]).sum(1)
        s["out"][b, :, :L] = total if c["decay"] == 0 else c["decay"] * s["mass"][b, :, :L] + total
    return s["out"]


def _plain_decode(s):
    c = s["case"]
    return _plain_sums(s, s["q"].view(c["B"], c["N"], c["hq"], c["d"]), False)


def _plain_prefill(s):
    return _plain_sums(s, s["q"], True)


def _plain_select(s):
    c = s["case"]
    out = torch.full((c["B"], c["hkv"], s["most"]), -1, dtype=torch.int32, device="cuda")
    for b, (L, n) in enumerate(zip(s["total"], s["keep"])):
        if n >= L:
            out[b, :, :L] = torch.arange(L, dtype=torch.int32, device="cuda")
            continue
        m = s["mass"][b, :, :L].clone()
        m[:, : c["sink"]] = float("inf")
        m[:, L - c["recent"]:] = float("inf")
        first = torch.sort(m, dim=1, descending=True, stable=True).indices[:, :n]
        out[b, :, :n] = torch.sort(first, 1).values.int()
    return out


def _plain_evict(s):
    P = s["case"]["page"]
    hkv = s["case"]["hkv"]
    head = torch.arange(hkv, device="cuda")[:, None]
    for b, (L, n) in enumerate(zip(s["total"], s["keep"])):
        if n >= L:
            continue
        i = s["index"][b, :, :n].long()
        j = torch.arange(n, device="cuda")
        src, dst = s["table"][b].long()[i // P], s["new"][b].long()[j // P]
        for pages in (s["k"], s["v"]):
            pages[dst[None], head, (j % P)[None]] = pages[src, head, i % P]
        s["out"][b, :, :n] = s["mass"][b].gather(1, i)
        s["out"][b, :, n:L] = 0.0
        pages = -(-n // P)
        s["now"][b, :pages] = s["new"][b, :pages]
        s["now"][b, pages:] = -1
        s["lens"][b] = n
    return s["k"], s["v"], s["now"], s["lens"], s["out"]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    hkv, op, total = case["hkv"], case["op"], s["total"]
    if op == "select":                     # whole numbers, one key at a time: larger mass first, then lower position
        out = torch.full((case["B"], hkv, s["most"]), -1, dtype=torch.int32)
        mass = s["mass"].double().cpu()
        for b, (L, n) in enumerate(zip(total, s["keep"])):
            n = min(n, L)
            for h in range(hkv):
                always = set(range(min(case["sink"], L))) | set(range(max(0, L - case["recent"]), L))
                row = mass[b, h].tolist()
                order = sorted((t for t in range(L) if t not in always), key=lambda t: (-row[t], t)) if n < L else []
                chosen = sorted(list(always) + order[: n - len(always)]) if n < L else range(L)
                out[b, h, :n] = torch.tensor(list(chosen), dtype=torch.int32)
        return out.cuda()
    P, d = case["page"], case["d"]
    if op == "evict":                      # copies: slot by slot in the flat views of the pools
        k, v, out = s["k"].clone(), s["v"].clone(), torch.zeros_like(s["mass"])
        table, lens = s["table"].clone(), torch.tensor(total, dtype=torch.int32, device="cuda")
        for b, (L, n) in enumerate(zip(total, s["keep"])):
            if n >= L:
                continue
            for h in range(hkv):
                at = s["index"][b, h, :n].long()
                page = torch.div(at, P, rounding_mode="floor")
                from_row = (s["table"][b].long()[page] * hkv + h) * P + at - page * P
                slot = torch.arange(n, device="cuda")
                page = torch.div(slot, P, rounding_mode="floor")
                to_row = (s["new"][b].long()[page] * hkv + h) * P + slot - page * P
                for got, src in ((k, s["k"]), (v, s["v"])):
                    got.view(-1, d).index_copy_(0, to_row, src.view(-1, d).index_select(0, from_row))
                out[b, h, :n] = s["mass"][b, h].index_select(0, at)
            table[b].fill_(-1)
            table[b, : (n + P - 1) // P] = s["new"][b, : (n + P - 1) // P]
            lens[b] = n
        return k, v, table, lens, out
    n, hq = (case["N"] if op == "decode" else case["n"]), case["hq"]
    G = hq // hkv
    out = torch.zeros(s["mass"].shape, dtype=torch.float64, device="cuda")
    q = s["q"].reshape(case["B"], n, hq, d)
    lse = s["lse"].reshape(case["B"], n, hq).double()
    for b, L in enumerate(total):
        ids = s["table"][b, : -(-L // P)].long()
        for h in range(hkv if L else 0):
            k = s["k"][ids, h].double().flatten(0, 1)[:L]
            for j in range(h * G, h * G + G):
                for i in range(0, n, 1024):
                    w = min(1024, n - i)
                    x = s["scale"] * (q[b, i: i + w, j].double() @ k.T) - lse[b, i: i + w, j][:, None]
                    if op == "prefill":    # query token i sits at position L - n + i
                        seen = torch.ones(w, L, dtype=torch.bool, device="cuda").tril(L - n + i)
                        x = torch.where(seen, x, -math.inf)
                    out[b, h, :L] += torch.exp(x).sum(0)
            if case["decay"]:
                out[b, h, :L] += case["decay"] * s["mass"][b, h, :L].double()
    return out
