"""Measured cases of the 8-bit paged cache and of query and key norms.

``append_kv`` takes norms of queries and keys for each head in the pass that
rotates and writes them (ops "norm", a 16-bit cache), and writes caches of
8-bit values with a power of two for each vector (ops "quant"); ``read_kv``
takes cached rows back to 16 bits, and ``paged_attention`` attends to the 8-bit
cache directly.

``run`` computes a case with elementary torch operations, or, where ``own`` is
true, with the framework's calls.  ``exact`` computes it in 64 bits, sequence
by sequence, from the definitions.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
EPS = 1e-6


# ---------------------------------------------------------------------------
# the cases

def listed():
    return [
        # one decoding sequence without drafts, normed queries and keys: latency
        dict(name="norm-one", op="norm", batch=1, new=1, ctx=700, ragged=False, hq=32, hkv=8, d=128, page=64,
             dtype="bf16", heads_first=True, rot=128, interleaved=False, mix=21),
        # one verification round of 256 sequences with K = 5 drafts: K + 1 new tokens each
        dict(name="norm-round", op="norm", batch=256, new=6, ctx=120, ragged=True, hq=32, hkv=8, d=128, page=64,
             dtype="bf16", heads_first=True, rot=128, interleaved=False, mix=22),
        # prompts entering a 16-bit cache; half of each head is rotated, in adjacent pairs
        dict(name="norm-prompts", op="norm", batch=11, new=4099, ctx=0, ragged=True, hq=16, hkv=4, d=96, page=16,
             dtype="fp16", heads_first=False, rot=48, interleaved=True, mix=23),
        # the verification round, written in 8 bits
        dict(name="quant-round", op="quant", batch=256, new=6, ctx=120, ragged=True, hq=32, hkv=8, d=128, page=64,
             dtype="bf16", heads_first=True, rot=128, interleaved=False, normed=True, mix=24),
        # prompts entering an 8-bit cache, without norms
        dict(name="quant-prompts", op="quant", batch=7, new=5003, ctx=0, ragged=True, hq=32, hkv=8, d=128, page=32,
             dtype="bf16", heads_first=False, rot=64, interleaved=False, normed=False, mix=25),
        # a short sequence taken back to 16 bits: latency
        dict(name="read-one", op="read", batch=1, new=701, ctx=0, ragged=False, hq=32, hkv=8, d=128, page=64,
             dtype="bf16", heads_first=True, mix=26),
        # many sequences taken back, as when they move to another cache
        dict(name="read-batch", op="read", batch=64, new=4099, ctx=0, ragged=True, hq=32, hkv=8, d=128, page=64,
             dtype="bf16", heads_first=True, mix=27),
        # one token of one sequence over a short 8-bit context: latency
        dict(name="attend8-one", op="attend", batch=1, new=1, ctx=1000, ragged=False, hq=32, hkv=8, d=128, page=64,
             dtype="bf16", heads_first=True, window=0, mix=28),
        # the verification round's target pass: K + 1 = 6 tokens over ragged contexts
        dict(name="attend8-round", op="attend", batch=256, new=6, ctx=4096, ragged=True, hq=32, hkv=8, d=128, page=64,
             dtype="bf16", heads_first=True, window=0, mix=29),
        # two long documents, K + 1 tokens each: little work in rows, a long axis
        dict(name="attend8-long", op="attend", batch=2, new=6, ctx=131071, ragged=False, hq=16, hkv=4, d=64, page=16,
             dtype="fp16", heads_first=False, window=0, mix=30),
        # chunks of prompts over what is cached already, beside short ones
        dict(name="attend8-chunks", op="attend", batch=5, new=1025, ctx=7000, ragged=True, hq=32, hkv=8, d=128, page=32,
             dtype="bf16", heads_first=True, window=0, mix=31),
        # two whole prompts: bound by products
        dict(name="attend8-prompts", op="attend", batch=2, new=4097, ctx=0, ragged=False, hq=32, hkv=8, d=128, page=64,
             dtype="bf16", heads_first=False, window=0, mix=32),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "quant", "read", "attend", "attend"))
    hkv = rng.choice((1, 2, 4, 8))
    c = dict(op=op, hq=hkv * rng.choice((1, 2, 3, 4, 7, 8)), hkv=hkv, d=rng.choice((64, 128, 128, 96, 80)),
             page=rng.choice((16, 32, 64, 128, 48)), dtype=rng.choice(("bf16", "fp16")),
             heads_first=rng.random() < 0.5, ragged=rng.random() < 0.7, mix=rng.randrange(100, 1 << 20))
    if op in ("norm", "quant"):
        c["new"] = _log(rng, 1, 4096)
        c["batch"] = _log(rng, 1, max(1, min(256, 16384 // c["new"])))
        c["ctx"] = _log(rng, 1, 1000)
        c["rot"] = c["d"] if rng.random() < 0.7 else c["d"] // 2
        c["interleaved"] = rng.random() < 0.3
        if op == "quant":
            c["normed"] = rng.random() < 0.5
        return c
    if op == "read":
        c["new"] = _log(rng, 1, 16384)
        c["batch"] = _log(rng, 1, max(1, min(64, 131072 // c["new"])))
        c["ctx"] = _log(rng, 1, 1000) if rng.random() < 0.3 else 0
        return c
    if rng.random() < 0.7:       # rounds: few new tokens over what is cached
        c["new"] = _log(rng, 1, 65)
        c["ctx"] = _log(rng, 16, 65536)
        c["batch"] = _log(rng, 1, max(1, min(256, 524288 // (c["ctx"] + c["new"]),
                                             4000000 // (c["new"] * (c["ctx"] + c["new"])) + 1)))
    else:                        # chunks of prompts
        c["new"] = _log(rng, 65, 4096)
        c["ctx"] = _log(rng, 1, 4096)
        c["batch"] = rng.randint(1, max(1, 4096 // c["new"]))
    c["window"] = rng.choice((0, 0, 0, rng.randint(1, 2000)))
    return c


def lengths(case):
    """(new tokens or rows read, length with them) of every sequence."""
    r = random.Random(case["mix"])
    new, total = [], []
    for _ in range(case["batch"]):
        n, c = case["new"], case["ctx"]
        if case["ragged"]:
            # rounds keep their K + 1 tokens, prompts end anywhere; contexts from an eighth to all
            n = n if n <= 6 else r.randint(max(1, n // 8), n)
            c = r.randint(c // 8, c) if c else 0
        new.append(n)
        total.append(n + c)
    return new, total


# ---------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    dt = DTYPES[s["dtype"]]
    new, total = lengths(s)
    B, ps, hq, hkv, d = s["batch"], s["page"], s["hq"], s["hkv"], s["d"]
    N = sum(new)
    need = [-(-t // ps) for t in total]
    wide = max(need)
    pool = sum(need) + 3
    # pages in the order in which a busy allocator hands them out: any
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    pages = torch.zeros(B, wide, dtype=torch.int32, device="cuda")
    have = torch.tensor(need, device="cuda").view(-1, 1) > torch.arange(wide, device="cuda")
    pages[have] = perm[:sum(need)]
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s.update(pages=pages, q_start=torch.tensor(start, dtype=torch.int32, device="cuda"),
             kv_len=torch.tensor(total, dtype=torch.int32, device="cuda"),
             n_max=max(new), l_max=max(total), n_all=N)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale

    for name in ("k", "v"):
        shape = (pool, hkv, ps) if s["heads_first"] else (pool, ps, hkv)
        if s["op"] == "norm":
            cache = normal(*shape, d).to(dt)
        else:
            # vectors of different size, as tokens and heads differ
            cache, scale = _quantise(normal(*shape, d) * torch.exp(normal(*shape, 1, scale=0.4)))
            s[name + "_scale"] = scale.transpose(1, 2) if s["heads_first"] else scale
        s[name + "_cache"] = cache.transpose(1, 2) if s["heads_first"] else cache
        del cache
    if s["op"] != "read":
        # a spread of 1.5 gives scores with a few dominant keys per row, as trained heads have
        s["q"] = normal(N, hq, d, scale=1.5).to(dt)
    if s["op"] in ("norm", "quant"):
        s["k"] = (normal(N, hkv, d) * torch.exp(normal(N, hkv, 1, scale=0.4))).to(dt)
        s["v"] = (normal(N, hkv, d) * torch.exp(normal(N, hkv, 1, scale=0.4))).to(dt)
        half = torch.arange(s["rot"] // 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = torch.pow(10000.0, -2.0 * half / s["rot"])
        s["q_norm"] = s["k_norm"] = None
        if s["op"] == "norm" or s["normed"]:
            s["q_norm"] = (1 + normal(d, scale=0.2)).to(dt)
            s["k_norm"] = (1 + normal(d, scale=0.2)).to(dt)
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    if own:
        return _run_own(s)
    return {"norm": _plain_append, "quant": _plain_append, "read": _plain_read, "attend": _plain_attend}[s["op"]](s)


def _run_own(s):
    import speculative_decoding_verification_08_gb300 as sv
    table = s["pages"], s["q_start"], s["kv_len"]
    caches = s["k_cache"], s["v_cache"]
    if s["op"] == "norm":
        q = sv.append_kv(s["k"], s["v"], *caches, *table, inv_freq=s["inv_freq"], q=s["q"],
                         interleaved=s["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    scales = dict(k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["op"] == "quant":
        q = sv.append_kv(s["k"], s["v"], *caches, *table, inv_freq=s["inv_freq"], q=s["q"],
                         interleaved=s["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, **scales)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"], **scales}
    if s["op"] == "read":
        k, v = sv.read_kv(*caches, *table, rows=s["n_all"], dtype=DTYPES[s["dtype"]], **scales)
        return {"k": k, "v": v}
    return {"out": sv.paged_attention(s["q"], *caches, *table, window=s["window"], **scales)}


def _quantise(y):
    """e4m3 codes and e8m0 scales of vectors y [..., d] in fp32: the smallest
    power of two from 2^-100 to 2^100 that brings the largest magnitude to 448
    or less."""
    m, x = torch.frexp(y.abs().amax(-1))
    e = (x - 9 + (m > 0.875)).masked_fill(m == 0, -100).clamp(-100, 100)
    code = (y * _power(-e).unsqueeze(-1)).to(E4M3)
    return code, (e + 127).to(torch.uint8).view(E8M0)


def _power(e):
    """2^e in fp32, to the last bit (exp2 and ldexp may miss it)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _owners(s):
    """For every new token: its sequence, its place among the new ones, its slot."""
    t = torch.arange(s["n_all"], device="cuda")
    b = torch.searchsorted(s["q_start"][1:].long(), t, right=True)
    j = t - s["q_start"].long()[b]
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    return b, j, s["kv_len"].long()[b] - n[b] + j


def _plain_append(s):
    b, _, slot = _owners(s)
    page = s["pages"][b, slot // s["page"]].long()
    at = slot % s["page"]
    ang = slot.double().view(-1, 1) * s["inv_freq"]
    cos, sin = torch.cos(ang).float().unsqueeze(1), torch.sin(ang).float().unsqueeze(1)
    rot = s["rot"]

    def turned(x, weight):
        y = x.float()
        if weight is not None:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.float()
        if s["interleaved"]:
            a, c = y[..., 0:rot:2], y[..., 1:rot:2]
        else:
            a, c = y[..., :rot // 2], y[..., rot // 2:rot]
        ra, rc = a * cos - c * sin, a * sin + c * cos
        r = torch.stack((ra, rc), -1).flatten(-2) if s["interleaved"] else torch.cat((ra, rc), -1)
        return torch.cat((r, y[..., rot:]), -1)

    k = turned(s["k"], s["k_norm"])
    out = {"q": turned(s["q"], s["q_norm"]).to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "norm":
        s["k_cache"][page, at] = k.to(s["k"].dtype)
        s["v_cache"][page, at] = s["v"]
        return out
    for name, y in (("k", k), ("v", s["v"].float())):
        code, scale = _quantise(y)
        s[name + "_cache"].view(torch.uint8)[page, at] = code.view(torch.uint8)
        s[name + "_scale"].view(torch.uint8)[page, at] = scale.view(torch.uint8)
        out[name + "_scale"] = s[name + "_scale"]
    return out


def _values(s, name, page, at):
    """Cached vectors at (page, at), in fp32."""
    x = s[name + "_cache"].view(torch.uint8)[page, at].view(E4M3).float()
    e = s[name + "_scale"].view(torch.uint8)[page, at].int() - 127
    return x * _power(e).unsqueeze(-1)


def _plain_read(s):
    b, _, slot = _owners(s)
    page, at = s["pages"][b, slot // s["page"]].long(), slot % s["page"]
    dt = DTYPES[s["dtype"]]
    return {"k": _values(s, "k", page, at).to(dt), "v": _values(s, "v", page, at).to(dt)}


def _plain_attend(s):
    B, L, n_max, hkv, d = s["batch"], s["l_max"], s["n_max"], s["hkv"], s["d"]
    G = s["hq"] // hkv
    b, j, _ = _owners(s)
    pos = torch.arange(L, device="cuda")
    page = s["pages"][:, pos // s["page"]].long()
    at = (pos % s["page"]).expand(B, L)
    k = _values(s, "k", page, at).permute(0, 2, 3, 1)              # [B][hkv][d][L]
    v = _values(s, "v", page, at).permute(0, 2, 1, 3)              # [B][hkv][L][d]
    q = torch.zeros(B, n_max, s["hq"], d, device="cuda")
    q[b, j] = s["q"].float()
    q = q.view(B, n_max, hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * n_max, d)
    w = (q @ k) * (1.0 / math.sqrt(d))
    del q, k
    w = w.view(B, hkv, G, n_max, L)
    n = (s["q_start"][1:] - s["q_start"][:-1]).view(B, 1, 1)
    last = s["kv_len"].view(B, 1, 1) - n + torch.arange(n_max, device="cuda").view(1, n_max, 1)
    seen = pos <= last
    if s["window"]:
        seen = seen & (pos > last - s["window"])
    seen = seen.view(B, 1, 1, n_max, L)
    w.masked_fill_(~seen, float("-inf"))
    top = w.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))
    w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = w.view(B, hkv, G * n_max, L) @ v
    total = total.view(B, hkv, G * n_max, 1)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    o = o.view(B, hkv, G, n_max, d).permute(0, 3, 1, 2, 4).reshape(B, n_max, s["hq"], d)
    return {"out": o[b, j].to(s["q"].dtype)}


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    new, total = lengths(case)
    N, d, hq, hkv = sum(new), case["d"], case["hq"], case["hkv"]
    if case["op"] in ("norm", "quant"):
        kept = 2 * d if case["op"] == "norm" else d + 1            # bytes of a cached vector
        normed = case["op"] == "norm" or case["normed"]
        heads = hq + hkv
        return {"bytes": N * (2 * 2 * d * hq + 2 * hkv * (2 * d + kept)) + 12 * N,
                "flops": N * heads * (3.0 * case["rot"] + (4.0 * d if normed else 0.0))
                + (0.0 if case["op"] == "norm" else 4.0 * N * hkv * d)}
    if case["op"] == "read":
        return {"bytes": 2 * N * hkv * (3 * d + 1) + 4 * N / case["page"], "flops": 2.0 * N * hkv * d}
    win = case["window"]
    keys = pairs = 0
    for n, t in zip(new, total):
        first = t - n + 1                                          # keys the first new token may see
        keys += min(t, n - 1 + win) if win else t
        if not win:
            pairs += n * first + n * (n - 1) // 2
        else:
            grow = max(0, min(n, win - first))                     # tokens that see fewer than the window
            pairs += grow * first + grow * (grow - 1) // 2 + (n - grow) * win
    return {"bytes": 2 * 2 * N * hq * d + 2 * keys * hkv * (d + 1) + 4 * keys / case["page"],
            "flops": 4.0 * pairs * hq * d}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(s)
    return _exact_read(s) if case["op"] == "read" else _exact_append(s)


def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_append(s):
    starts, lens, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["pages"].tolist()
    rot, half = s["rot"], s["rot"] // 2
    first = torch.arange(half, device="cuda") * (2 if s["interleaved"] else 1)
    second = first + (1 if s["interleaved"] else half)
    quant = s["op"] == "quant"
    out = {"q": s["q"].double(), "k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
    if quant:
        for name in ("k_scale", "v_scale"):
            out[name] = _two_to(s[name].view(torch.uint8).long() - 127)
    for b in range(s["batch"]):
        t0, t1 = starts[b], starts[b + 1]
        slot = torch.arange(lens[b] - (t1 - t0), lens[b], device="cuda")
        turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                           slot.double().view(-1, 1, 1) * s["inv_freq"])
        k, v, q = s["k"][t0:t1].double(), s["v"][t0:t1].double(), s["q"][t0:t1].double()
        for x, weight in ((k, s["k_norm"]), (q, s["q_norm"])):
            if weight is not None:
                x *= weight.double() / torch.sqrt(x.square().sum(-1, keepdim=True) / s["d"] + EPS)
            y = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = y.real, y.imag
        out["q"][t0:t1] = q
        page, at = torch.tensor(table[b], device="cuda")[slot // s["page"]], slot % s["page"]
        for name, x in (("k", k), ("v", v)):
            if quant:
                # what the codes stand for before they are rounded
                top = x.abs().amax(-1)
                near = torch.ceil(torch.log2(top / 448)).clamp(-100, 100)       # or one step off
                scale = _two_to(near + 1)
                while bool((low := (top <= 224 * scale) & (scale > 2.0 ** -100)).any()):
                    scale = torch.where(low, scale / 2, scale)
                out[name + "_scale"][page, at] = scale
                x = x / scale.unsqueeze(-1)
            out[name + "_cache"][page, at] = x
    return out


def _exact_read(s):
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    got = {}
    for name in ("k", "v"):
        parts = []
        for b in range(s["batch"]):
            mine = s["pages"][b, :-(-lens[b] // s["page"])].long()
            x = s[name + "_cache"].view(torch.uint8)[mine].view(E4M3).double()
            x = x * _two_to(s[name + "_scale"].view(torch.uint8)[mine].long() - 127).unsqueeze(-1)
            parts.append(x.reshape(-1, s["hkv"], s["d"])[lens[b] - starts[b + 1] + starts[b]:lens[b]])
        got[name] = torch.cat(parts)
    return got


def _exact_attend(s):
    starts, lens = s["q_start"].tolist(), s["kv_len"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    G, ps = s["hq"] // s["hkv"], s["page"]
    for b in range(s["batch"]):
        t0, t1, L = starts[b], starts[b + 1], lens[b]
        n = t1 - t0
        mine = s["pages"][b, :-(-L // ps)].long()
        reach = torch.arange(L - n, L, device="cuda").view(-1, 1)
        at = torch.arange(L, device="cuda").view(1, -1)
        hide = at > reach
        if s["window"]:
            hide |= at <= reach - s["window"]
        for h in range(s["hkv"]):
            k, v = (s[x + "_cache"].view(torch.uint8)[mine, :, h].view(E4M3).double()
                    * _two_to(s[x + "_scale"].view(torch.uint8)[mine, :, h].long() - 127).unsqueeze(-1)
                    for x in ("k", "v"))
            k, v = k.reshape(-1, s["d"])[:L], v.reshape(-1, s["d"])[:L]
            for i in range(h * G, h * G + G):
                a = (s["q"][t0:t1, i].double() @ k.t() / math.sqrt(s["d"])).masked_fill_(hide, -math.inf)
                out[t0:t1, i] = torch.softmax(a, dim=-1) @ v
    return {"out": out}
