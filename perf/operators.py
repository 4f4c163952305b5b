"""Measured cases of the 8-bit shared KV cache's operators.

The cache keeps every token's K and V of a KV head as e4m3 values with one power-of-two scale (e8m0)
for the token's `head_dim` values.  Four operators work on it:

* append: quantise the K/V of new tokens into the pages as they are written;
* read:   read a range of every request's tokens back as contiguous bf16 rows;
* decode: attention of the stacked query rows of several decoders over the cache (one step);
* chunk:  causal attention of a ragged chunk of new tokens per request over the cache.

`own` chooses what `run` computes with: False, plain torch operations in 32 bits; True, the
framework's kernels.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of a serving batch writes one token per request
        dict(name="append one step", op="append", B=64, hkv=8, d=128, page=16, lo=256, hi=2048, new_lo=1, new_hi=1,
             empty=0, lens_seed=1),
        # prompts of a mixed batch arrive behind cached prefixes; odd lengths, a slice of a fused projection
        dict(name="append prompts", op="append", B=24, hkv=8, d=128, page=16, lo=1, hi=3000, new_lo=97, new_hi=4001,
             empty=1, lens_seed=2),
        # a short session handed back to a 16-bit consumer
        dict(name="read short", op="read", B=3, hkv=2, d=64, page=16, lo=100, hi=700, new_lo=33, new_hi=600, empty=0,
             lens_seed=3),
        # long sessions handed over between clusters
        dict(name="read long", op="read", B=8, hkv=8, d=128, page=32, lo=16384, hi=32768, new_lo=8001, new_hi=32768,
             empty=0, lens_seed=4),
        # the tiny configuration: one request, two decoders; latency
        dict(name="decode tiny", op="decode", B=1, N=2, hq=8, hkv=2, d=64, page=16, lo=256, hi=256, empty=0,
             lens_seed=5),
        # two decoders over a batch of ordinary contexts, one padded slot
        dict(name="decode 8 rows", op="decode", B=32, N=2, hq=32, hkv=8, d=128, page=16, lo=1024, hi=8192, empty=1,
             lens_seed=6),
        # eight decoders, long mixed contexts, 40 stacked rows per KV head
        dict(name="decode 40 rows", op="decode", B=24, N=8, hq=40, hkv=8, d=128, page=32, lo=4096, hi=65536, empty=0,
             lens_seed=7),
        # four very long contexts, eight decoders: work split over the tokens
        dict(name="decode long", op="decode", B=4, N=8, hq=16, hkv=8, d=128, page=16, lo=131584, hi=131584, empty=0,
             lens_seed=8),
        # verification of a few drafted tokens per request, ragged
        dict(name="chunk drafts", op="chunk", B=32, hq=32, hkv=8, d=128, page=16, lo=1000, hi=8000, new_lo=1,
             new_hi=8, empty=1, lens_seed=9),
        # turns of many sessions prefilled together behind their cached prefixes
        dict(name="chunk turns", op="chunk", B=12, hq=32, hkv=8, d=128, page=16, lo=600, hi=9000, new_lo=60,
             new_hi=1100, empty=0, lens_seed=10),
        # one long document extended by one chunk
        dict(name="chunk document", op="chunk", B=1, hq=40, hkv=8, d=128, page=32, lo=40000, hi=40000, new_lo=2048,
             new_hi=2048, empty=0, lens_seed=11),
        # a small model with 64-wide heads and an odd group, ragged short turns
        dict(name="chunk narrow heads", op="chunk", B=9, hq=14, hkv=2, d=64, page=16, lo=40, hi=2500, new_lo=1,
             new_hi=300, empty=1, lens_seed=12),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "decode", "chunk"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 32])
    hkv = rng.choice([1, 2, 4, 8])
    B = _log_uniform(rng, 1, 64)
    empty = rng.choice([0, 0, 0, 1]) if B > 1 else 0
    c = dict(op=op, B=B, hkv=hkv, d=d, page=page, empty=empty, lens_seed=rng.randrange(1 << 30))
    if op == "append":
        c["new_lo"], c["new_hi"] = 1, _log_uniform(rng, 1, max(1, 60000 // B) if B > 15 else 4000)
        c["lo"], c["hi"] = 1, _log_uniform(rng, 1, 3000)
    elif op == "read":
        c["lo"], c["hi"] = 1, _log_uniform(rng, 16, max(16, min(32768, 200000 // B)))
        c["new_lo"], c["new_hi"] = 1, c["hi"]
    elif op == "decode":
        g = rng.choice([1, 2, 3, 4, 5, 7, 8])
        n = rng.choice([n for n in (1, 2, 3, 4, 5, 8) if n * g <= 64])
        c["N"], c["hq"] = n, g * hkv
        c["lo"], c["hi"] = 1, _log_uniform(rng, 16, max(64, min(131072, 500000 // B)))
    else:
        g = rng.choice([1, 2, 3, 4, 5, 7, 8])
        c["hq"] = g * hkv
        c["hi"] = _log_uniform(rng, 64, max(64, min(32768, 100000 // B)))
        c["new_lo"], c["new_hi"] = 1, _log_uniform(rng, 1, max(1, min(c["hi"], 8000 // B)))
        c["lo"] = c["new_hi"]
    return c


def _lengths(case):
    """(cached tokens, new or read tokens, first token of the append or the read range) of each request."""
    rng = random.Random(case["lens_seed"])
    B, op = case["B"], case["op"]
    total, new, start = [], [], []
    for b in range(B):
        L = _log_uniform(rng, case["lo"], case["hi"])
        n = _log_uniform(rng, case["new_lo"], case["new_hi"]) if "new_lo" in case else 0
        s = 0
        if op == "append":                 # n tokens behind s cached ones
            s, L = L, L + n
        elif op == "read":                 # tokens [s, s + n)
            n = min(n, L)
            s = rng.randint(0, L - n)
        elif op == "chunk":                # the last n of L
            n = min(n, L)
            s = L - n
        if b >= B - case["empty"]:         # padded slots
            L, n, s = (s, 0, s) if op == "append" else (0, 0, 0)
        total.append(L)
        new.append(n)
        start.append(s)
    return total, new, start


def work(case):
    total, new, start = _lengths(case)
    hkv, d = case["hkv"], case["d"]
    token = hkv * (2 * d + 2)              # e4m3 K and V and their two scale bytes
    wide = hkv * 2 * d * 2                 # the same in bf16
    if case["op"] in ("append", "read"):
        return {"bytes": sum(new) * (token + wide), "flops": sum(new) * hkv * 2 * d}
    if case["op"] == "decode":
        rows = case["N"] * case["hq"]
        return {"bytes": sum(total) * token + case["B"] * rows * (4 * d + 4), "flops": 4 * d * rows * sum(total)}
    hq = case["hq"]
    seen = sum(n * s + n * (n + 1) // 2 for n, s in zip(new, start))
    read = sum(L for L, n in zip(total, new) if n)
    return {"bytes": read * token + sum(new) * hq * (4 * d + 4), "flops": 4 * d * hq * seen}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _kv(g, n, hkv, d, keys):
    """K or V of n tokens, fp32 [n, hkv, d]: keys have a few large channels, values a magnitude per token."""
    x = _randn(g, n, hkv, d)
    if keys:
        x[..., :: max(1, d // 4)] *= 6.0
    else:
        x *= torch.exp2(_randn(g, n, hkv, 1))
    return x


def _power(byte):
    """2^(byte - 127) in fp32, exact, from the bits (an exponentiation may be off by a last bit)."""
    b = byte.int()
    return torch.where(b > 0, b << 23, torch.full_like(b, 1 << 22)).view(torch.float32)


def _quantise(x):
    """fp32 [..., d] -> (e4m3 [..., d], e8m0 bytes [...]): the least power of two 2^e with max|x| <= 448 * 2^e,
    rounded to nearest even."""
    a = x.abs().amax(-1)
    m, e = torch.frexp(a)
    e = (e - 9 + (m > 0.875).int()).clamp(-127, 127)
    e = torch.where(a > 0, e, torch.full_like(e, -127))
    bad = ~torch.isfinite(a)
    q = (x * _power(127 - e)[..., None]).to(torch.float8_e4m3fn)
    q = torch.where(bad[..., None], torch.full_like(q.view(torch.uint8), 0x7F), q.view(torch.uint8))
    return q.view(torch.float8_e4m3fn), torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    total, new, start = _lengths(case)
    B, hkv, d, P = case["B"], case["hkv"], case["d"], case["page"]
    rng = random.Random(int(seed))
    pages = [-(-n // P) for n in total]
    ids = list(range(sum(pages) + 3))
    rng.shuffle(ids)
    table = torch.full((B, max(pages) + 2), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = torch.tensor(ids[at: at + n], dtype=torch.int32)
        at += n
    num = len(ids)
    s = dict(case=case, total=total, new=new, start=start, table=table.cuda(), num_pages=num, scale=1 / math.sqrt(d))
    k8 = torch.empty(num, hkv, P, d, dtype=torch.uint8, device="cuda")
    v8 = torch.empty_like(k8)
    sc = torch.empty(num, hkv, 2, P, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (P * hkv * d))
    for i in range(0, num, step):          # every slot holds a value, those behind the last token too
        n = min(step, num - i)
        for j, dst in enumerate((k8, v8)):
            q, e = _quantise(_kv(g, n * P, hkv, d, j == 0).view(n, P, hkv, d).transpose(1, 2))
            dst[i: i + n] = q.contiguous().view(torch.uint8)
            sc[i: i + n, :, j] = e
    s.update(k8=k8, v8=v8, sc=sc)
    if case["op"] == "append":             # K and V lie side by side, as a fused projection leaves them
        n = sum(new)
        kv = torch.cat([_kv(g, n, hkv, d, True), _kv(g, n, hkv, d, False)], 1).to(torch.bfloat16)
        s["k_new"], s["v_new"] = kv[:, :hkv], kv[:, hkv:]
    elif case["op"] == "decode":
        s["q"] = _randn(g, B, case["N"] * case["hq"], d).to(torch.bfloat16)
    elif case["op"] == "chunk":
        s["q"] = _randn(g, sum(new), case["hq"], d).to(torch.bfloat16)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from cross_model_shared_gb300 import QuantizedKVPool
        lens = s["start"] if case["op"] == "append" else s["total"]
        pool = QuantizedKVPool(s["num_pages"], case["page"], case["hkv"], case["d"], max_batch=case["B"],
                               max_pages_per_seq=s["table"].shape[1], k_pages=s["k8"], v_pages=s["v8"],
                               scales=s["sc"], initial_seq_lens=lens)
        pool.block_table.copy_(s["table"])
        s["pool"] = pool
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        pool = s["pool"]
        if op == "append":
            pool.append_kv(s["k_new"], s["v_new"], s["new"], start=s["start"])
            return _pages(s)
        if op == "read":
            return pool.read_kv(s["start"], s["new"])
        if op == "decode":
            return pool.decode_attention(s["q"], s["case"]["N"], scale=s["scale"], return_lse=True)
        return pool.chunk_attention(s["q"], s["new"], scale=s["scale"], return_lse=True)
    return {"append": _plain_append, "read": _plain_read, "decode": _plain_decode, "chunk": _plain_chunk}[op](s)


def _pages(s):
    """The cache itself: e4m3 values and e8m0 scales."""
    return (s["k8"].view(torch.float8_e4m3fn), s["v8"].view(torch.float8_e4m3fn),
            s["sc"].view(torch.float8_e8m0fnu))


def _slots(s):
    """(page, slot) of every token of the ranges [start, start + new), in order."""
    P, dev = s["case"]["page"], s["table"].device
    n = torch.tensor(s["new"], device=dev)
    b = torch.repeat_interleave(torch.arange(len(s["new"]), device=dev), n, output_size=sum(s["new"]))
    first = torch.cumsum(n, 0) - n
    pos = torch.arange(sum(s["new"]), device=dev) - first[b] + torch.tensor(s["start"], device=dev)[b]
    return s["table"][b, pos // P].long(), pos % P


def _plain_append(s):
    page, slot = _slots(s)
    for j, (x, dst) in enumerate(((s["k_new"], s["k8"]), (s["v_new"], s["v8"]))):
        q, e = _quantise(x.float())
        dst[page, :, slot] = q.view(torch.uint8)
        s["sc"][page, :, j, slot] = e
    return _pages(s)


def _plain_read(s):
    page, slot = _slots(s)
    out = []
    for j, src in enumerate((s["k8"], s["v8"])):
        x = src[page, :, slot].view(torch.float8_e4m3fn).float()
        out.append((x * _power(s["sc"][page, :, j, slot])[..., None]).to(torch.bfloat16))
    return tuple(out)


def _cached(s, b):
    """K and V of request b in fp32, [hkv, L, d] each."""
    c = s["case"]
    L = s["total"][b]
    ids = s["table"][b, : -(-L // c["page"])].long()
    out = []
    for j, src in enumerate((s["k8"], s["v8"])):
        x = src[ids].view(torch.float8_e4m3fn).float() * _power(s["sc"][ids, :, j])[..., None]
        out.append(x.transpose(0, 1).reshape(c["hkv"], -1, c["d"])[:, :L])
    return out


def _softmax_attend(q, k, v, scale, hidden=None):
    x = torch.matmul(q, k.transpose(1, 2)) * scale
    if hidden is not None:
        x = x.masked_fill(hidden, float("-inf"))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / total, (m + torch.log(total))[..., 0]


def _plain_decode(s):
    c = s["case"]
    B, N, hkv, d = c["B"], c["N"], c["hkv"], c["d"]
    g = c["hq"] // hkv
    out = torch.zeros_like(s["q"])
    lse = torch.full(s["q"].shape[:2], float("-inf"), device="cuda")
    for b in range(B):
        if s["total"][b] == 0:
            continue
        k, v = _cached(s, b)
        q = s["q"][b].float().view(N, hkv, g, d).transpose(0, 1).reshape(hkv, N * g, d)
        o, e = _softmax_attend(q, k, v, s["scale"])
        out[b] = o.view(hkv, N, g, d).transpose(0, 1).reshape(-1, d).to(torch.bfloat16)
        lse[b] = e.view(hkv, N, g).transpose(0, 1).reshape(-1)
    return out, lse


def _plain_chunk(s, rows=512):
    c = s["case"]
    hkv, hq, d = c["hkv"], c["hq"], c["d"]
    g = hq // hkv
    out = torch.zeros_like(s["q"])
    lse = torch.zeros(s["q"].shape[:2], device="cuda")
    at = 0
    for b, n in enumerate(s["new"]):
        if n == 0:
            continue
        k, v = _cached(s, b)
        keys = torch.arange(s["total"][b], device="cuda")
        for i in range(0, n, rows):        # blocks of new tokens, to bound the scores' size
            w = min(rows, n - i)
            q = s["q"][at + i: at + i + w].float().view(w, hkv, g, d).permute(1, 0, 2, 3).reshape(hkv, w * g, d)
            last = s["start"][b] + i + w
            pos = torch.arange(s["start"][b] + i, last, device="cuda").repeat_interleave(g)
            o, e = _softmax_attend(q, k[:, :last], v[:, :last], s["scale"], keys[None, :last] > pos[:, None])
            out[at + i: at + i + w] = o.view(hkv, w, g, d).permute(1, 0, 2, 3).reshape(w, hq, d).to(torch.bfloat16)
            lse[at + i: at + i + w] = e.view(hkv, w, g).transpose(0, 1).reshape(w, hq)
        at += n
    return out, lse


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_values():
    """The value of each of the 256 codes, from the format's definition."""
    got = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = math.nan if (e, m) == (15, 7) else m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        got.append(-x if code >> 7 else x)
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def _powers():
    """2^(i - 200) for i in 0 .. 400, exact."""
    return torch.tensor([math.ldexp(1.0, i - 200) for i in range(401)], dtype=torch.float64, device="cuda")


def _value_rows(s, values, powers, which, ids, head):
    """The 64-bit values of pages `ids` of one KV head, [tokens, d]."""
    codes = s["k8" if which == 0 else "v8"][ids, head].long()
    power = powers[s["sc"][ids, head, which].long() + (200 - 127)]
    return (values[codes] * power[..., None]).flatten(0, 1)


def exact(case, seed):
    s = _inputs(case, seed)
    P, hkv, d, op = case["page"], case["hkv"], case["d"], case["op"]
    values, powers = _e4m3_values(), _powers()
    if op in ("append", "read"):
        k, v, sc = s["k8"], s["v8"], s["sc"]
        if op == "append":
            k, v = (values[x.int()] for x in (k, v))
            sc = powers[sc.long() + (200 - 127)]
        got, at = [[], []], 0
        for b, n in enumerate(s["new"]):
            pos = torch.arange(s["start"][b], s["start"][b] + n, device="cuda")
            page, slot = s["table"][b][pos // P].long(), pos % P
            for j, dst in enumerate((k, v)):
                if op == "read":
                    x = values[dst[page, :, slot].long()]
                    got[j].append(x * powers[sc[page, :, j, slot].long() + (200 - 127)][..., None])
                    continue
                x = (s["k_new"], s["v_new"])[j][at: at + n].double()
                big = x.abs().amax(-1)
                e = torch.floor(torch.log2(big.clamp(min=2.0 ** -130))).long() - 9       # 448 * 2^e <= big
                for _ in range(3):         # ... up to the least power that holds it
                    e = e + (big > E4M3_MAX * powers[e + 200]).long()
                e = e.clamp(min=-127)
                y = x / powers[e + 200][..., None]
                binade = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))).long()
                binade = binade + (y.abs() >= powers[binade + 201]).long() - (
                    (y.abs() < powers[binade + 200]) & (binade > -6)).long()
                grid = powers[binade + 200 - 3]
                dst[page, :, slot] = torch.round(y / grid) * grid
                sc[page, :, j, slot] = powers[e + 200]
            at += n
        return (k, v, sc) if op == "append" else tuple(torch.cat(x) for x in got)
    hq = case["hq"]
    g = hq // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(case["B"]):
        L, n = s["total"][b], s["new"][b]
        ids = s["table"][b, : -(-L // P)].long()
        for h in range(hkv):
            if L == 0 or (op == "chunk" and n == 0):
                continue
            k, v = (_value_rows(s, values, powers, j, ids, h)[:L] for j in (0, 1))
            if op == "decode":
                for m in range(case["N"]):
                    r = slice(m * hq + h * g, m * hq + h * g + g)
                    x = s["scale"] * (s["q"][b, r].double() @ k.T)
                    lse[b, r] = torch.logsumexp(x, 1)
                    out[b, r] = torch.exp(x - lse[b, r][:, None]) @ v
                continue
            for i in range(0, n, 1024):    # new token i sees the keys up to its own position
                w = min(1024, n - i)
                past = L - n + i
                for r in range(h * g, h * g + g):
                    x = s["scale"] * (s["q"][at + i: at + i + w, r].double() @ k[: past + w].T)
                    x[:, past:].masked_fill_(torch.ones(w, w, dtype=torch.bool, device="cuda").triu(1), -math.inf)
                    e = torch.logsumexp(x, 1)
                    lse[at + i: at + i + w, r] = e
                    out[at + i: at + i + w, r] = torch.exp(x - e[:, None]) @ v[: past + w]
        at += n
    return out, lse
