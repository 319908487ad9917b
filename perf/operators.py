"""Measured cases of the paged-cache and sampling operators.

Three operators serve the target side of a speculative round: ``append_kv``
rotates the new tokens' queries and keys and writes keys and values into a
paged cache, ``paged_attention`` lets the new tokens (a draft chain, a prompt
chunk or one token) attend to that cache, and ``warp_sample`` turns logits
into the warped probability rows verification takes and draws tokens from
them with given uniforms.

``run`` computes a case with elementary torch operations, or, where ``own`` is
true, with the framework's calls.  ``exact`` computes it in 64 bits, sequence
by sequence and row by row, from the definitions.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# the cases

def listed():
    return [
        # one decoding sequence without drafts: the smallest append, pure latency
        dict(name="append-one", op="append", batch=1, new=1, ctx=700, ragged=False, hq=32, hkv=8, d=128,
             page=64, dtype="bf16", heads_first=True, rot=128, interleaved=False, mix=1),
        # one verification round of 256 sequences with K = 5 drafts: K + 1 new tokens each
        dict(name="append-round", op="append", batch=256, new=6, ctx=1000, ragged=True, hq=32, hkv=8, d=128,
             page=64, dtype="bf16", heads_first=True, rot=128, interleaved=False, mix=2),
        # prompts entering the cache; half of each head is rotated, in adjacent pairs
        dict(name="append-prompts", op="append", batch=11, new=4099, ctx=0, ragged=True, hq=16, hkv=16, d=64,
             page=16, dtype="fp16", heads_first=False, rot=32, interleaved=True, mix=3),
        # one token of one sequence over a short context: latency
        dict(name="attend-one", op="attend", batch=1, new=1, ctx=1000, ragged=False, hq=32, hkv=8, d=128,
             page=64, dtype="bf16", heads_first=True, window=0, mix=4),
        # the verification round's target pass: K + 1 = 6 tokens over ragged contexts
        dict(name="attend-round", op="attend", batch=256, new=6, ctx=4096, ragged=True, hq=32, hkv=8, d=128,
             page=64, dtype="bf16", heads_first=True, window=0, mix=5),
        # two long documents, K + 1 tokens each: little work in rows, a long axis
        dict(name="attend-long", op="attend", batch=2, new=6, ctx=131071, ragged=False, hq=16, hkv=4, d=64,
             page=16, dtype="fp16", heads_first=False, window=0, mix=6),
        # chunks of prompts over what is cached already, beside short ones
        dict(name="attend-chunks", op="attend", batch=5, new=1025, ctx=7000, ragged=True, hq=32, hkv=8, d=128,
             page=32, dtype="bf16", heads_first=True, window=0, mix=7),
        # two whole prompts: the largest, bound by products
        dict(name="attend-prompts", op="attend", batch=2, new=8192, ctx=0, ragged=False, hq=32, hkv=8, d=128,
             page=64, dtype="bf16", heads_first=False, window=0, mix=8),
        # one sequence's next token, all filters on: latency
        dict(name="sample-one", op="sample", rows=1, v=32000, dtype="fp32", draw=True, probs=False,
             spread=3.0, filters=7, mix=9),
        # a draft step of 256 sequences: the drawn tokens and the rows q that verification takes
        dict(name="sample-draft", op="sample", rows=256, v=128256, dtype="fp32", draw=True, probs=True,
             spread=2.5, filters=7, mix=10),
        # temperature alone over a large vocabulary, tokens only
        dict(name="sample-plain", op="sample", rows=64, v=262144, dtype="fp32", draw=True, probs=False,
             spread=2.0, filters=0, mix=11),
        # the target rows p of a round (K + 1 = 6 per sequence) from 16-bit logits
        dict(name="sample-target", op="sample", rows=768, v=128256, dtype="bf16", draw=False, probs=True,
             spread=3.0, filters=6, mix=12),
    ]


def _log(rng, lo, hi):
    n = max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n + 1 if n == LEFT_OUT else n


#: The one size that the ranges leave out.
LEFT_OUT = 3 << 10


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "sample"))
    mix = rng.randrange(100, 1 << 20)
    if op == "sample":
        v = _log(rng, 1000, 262144)
        return dict(op=op, rows=_log(rng, 1, min(768, 768 * 128256 // v)), v=v,
                    dtype=rng.choice(("fp32", "fp32", "bf16", "fp16")), draw=True, probs=rng.random() < 0.5,
                    spread=round(rng.uniform(1.0, 4.0), 2), filters=rng.randrange(8), mix=mix)
    hkv = rng.choice((1, 2, 4, 8))
    c = dict(op=op, hq=hkv * rng.choice((1, 2, 3, 4, 7, 8)), hkv=hkv, d=rng.choice((64, 128, 128, 96, 80)),
             page=rng.choice((16, 32, 64, 128, 48)), dtype=rng.choice(("bf16", "fp16")),
             heads_first=rng.random() < 0.5, ragged=rng.random() < 0.7, mix=mix)
    if c["hq"] * c["d"] == LEFT_OUT:
        c["d"] = 64
    if op == "append":
        c["new"] = _log(rng, 1, 4096)
        c["batch"] = _log(rng, 1, max(1, min(256, 16384 // c["new"])))
        c["ctx"] = _log(rng, 1, 1000)
        c["rot"] = c["d"] if rng.random() < 0.7 else c["d"] // 2
        c["interleaved"] = rng.random() < 0.3
        return c
    if rng.random() < 0.6:       # rounds: few new tokens over what is cached
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
    """(new tokens, length after the append) of every sequence."""
    r = random.Random(case["mix"])
    new, total = [], []
    for _ in range(case["batch"]):
        n, c = case["new"], case["ctx"]
        if case["ragged"]:
            # rounds keep their K + 1 tokens, prompts end anywhere; contexts from an eighth to all
            n = n if n <= 6 else r.randint(max(1, n // 8), n)
            c = r.randint(c // 8, c) if c else 0
        c += LEFT_OUT in (c, n + c)
        new.append(n + (n == LEFT_OUT))
        total.append(new[-1] + c)
    return new, total


# ---------------------------------------------------------------------------
# inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    return _prepare_sample(s, g) if case["op"] == "sample" else _prepare_cache(s, g)


def _prepare_cache(s, g):
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
        return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dt)

    for name in ("k_cache", "v_cache"):
        if s["heads_first"]:
            s[name] = normal(pool, hkv, ps, d).transpose(1, 2)
        else:
            s[name] = normal(pool, ps, hkv, d)
    # a spread of 1.5 gives scores with a few dominant keys per row, as trained heads have
    s["q"] = normal(N, hq, d, scale=1.5)
    if s["op"] == "append":
        s["k"], s["v"] = normal(N, hkv, d), normal(N, hkv, d)
        half = torch.arange(s["rot"] // 2, dtype=torch.float64, device="cuda")
        s["inv_freq"] = torch.pow(10000.0, -2.0 * half / s["rot"])
    return s


def _prepare_sample(s, g):
    R, V = s["rows"], s["v"]
    z = torch.randn(R, V, generator=g, device="cuda")
    # rows of different sharpness
    z *= s["spread"] * torch.empty(R, 1, device="cuda").uniform_(0.7, 1.3, generator=g)
    s["z"] = z.to(DTYPES[s["dtype"]])
    s["u"] = torch.rand(R, generator=g, device="cuda", dtype=torch.float64) if s["draw"] else None
    s["temperature"] = torch.empty(R, device="cuda").uniform_(0.6, 1.2, generator=g)
    f = s["filters"]
    off = torch.rand(3, R, generator=g, device="cuda") < 0.2     # requests that leave a filter off
    k = torch.randint(1, 200, (R,), generator=g, device="cuda", dtype=torch.int32)
    p = torch.empty(R, device="cuda").uniform_(0.7, 0.99, generator=g)
    m = torch.empty(R, device="cuda").uniform_(0.001, 0.1, generator=g)
    s["top_k"] = k.masked_fill(off[0], 0) if f & 1 else None
    s["top_p"] = p.masked_fill(off[1], 1.0) if f & 2 else None
    s["min_p"] = m.masked_fill(off[2], 0.0) if f & 4 else None
    return s


# ---------------------------------------------------------------------------
# one pass

def run(s):
    if own:
        return _run_own(s)
    return {"append": _plain_append, "attend": _plain_attend, "sample": _plain_sample}[s["op"]](s)


def _run_own(s):
    import speculative_decoding_verification_08_gb300 as sv
    if s["op"] == "append":
        q = sv.append_kv(s["k"], s["v"], s["k_cache"], s["v_cache"], s["pages"], s["q_start"], s["kv_len"],
                         inv_freq=s["inv_freq"], q=s["q"], interleaved=s["interleaved"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "attend":
        return {"out": sv.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["pages"], s["q_start"],
                                          s["kv_len"], window=s["window"])}
    token, probs = sv.warp_sample(s["z"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                                  top_p=s["top_p"], min_p=s["min_p"], probs=s["probs"])
    return {k: x for k, x in (("token", token), ("probs", probs)) if x is not None}


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

    def rotate(x):
        y = x.float()
        if s["interleaved"]:
            a, c = y[..., 0:rot:2], y[..., 1:rot:2]
        else:
            a, c = y[..., :rot // 2], y[..., rot // 2:rot]
        ra, rc = a * cos - c * sin, a * sin + c * cos
        turned = torch.stack((ra, rc), -1).flatten(-2) if s["interleaved"] else torch.cat((ra, rc), -1)
        return torch.cat((turned, y[..., rot:]), -1).to(x.dtype)

    s["k_cache"][page, at] = rotate(s["k"])
    s["v_cache"][page, at] = s["v"]
    return {"q": rotate(s["q"]), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s):
    B, L, n_max, hkv, d = s["batch"], s["l_max"], s["n_max"], s["hkv"], s["d"]
    G = s["hq"] // hkv
    b, j, _ = _owners(s)
    pos = torch.arange(L, device="cuda")
    page = s["pages"][:, pos // s["page"]].long()
    at = (pos % s["page"]).expand(B, L)
    k = s["k_cache"][page, at].float().permute(0, 2, 3, 1)         # [B][hkv][d][L]
    v = s["v_cache"][page, at].float().permute(0, 2, 1, 3)         # [B][hkv][L][d]
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


def _plain_sample(s):
    # borders of the filters and of the draw are decided in 64 bits
    z = s["z"].double()
    R, V = z.shape
    x = z / s["temperature"].double().view(-1, 1)
    w = torch.exp(x - x.amax(-1, keepdim=True))
    order = torch.sort(s["z"], dim=-1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    rank = torch.arange(V, device="cuda")
    keep = torch.ones(R, V, dtype=torch.bool, device="cuda")
    if s["top_k"] is not None:
        k = s["top_k"].long().view(-1, 1)
        keep &= (rank < k) | (k <= 0)
    if s["top_p"] is not None:
        p = s["top_p"].double().view(-1, 1)
        kept = ws * keep
        before = kept.cumsum(-1) - kept
        keep &= (before < p * kept.sum(-1, keepdim=True)) | (p >= 1) | (rank == 0)
    if s["min_p"] is not None:
        keep &= (ws >= s["min_p"].double().view(-1, 1)) | (rank == 0)
    w = torch.zeros_like(w).scatter_(1, order, ws * keep)
    total = w.sum(-1, keepdim=True)
    out = {}
    if s["u"] is not None:
        run_ = w.cumsum(-1)
        t = (run_ <= s["u"].view(-1, 1) * total).sum(-1)
        last = V - 1 - (w > 0).flip(-1).to(torch.int8).argmax(-1)
        out["token"] = torch.minimum(t, last).to(torch.int32)
    if s["probs"]:
        out["probs"] = (w / total).float()
    return out


# ---------------------------------------------------------------------------
# what a pass cannot do without

def work(case):
    if case["op"] == "sample":
        R, V = case["rows"], case["v"]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": R * V * (size + (4 if case["probs"] else 0)) + R * 32, "flops": 4.0 * R * V}
    new, total = lengths(case)
    N, d, hq, hkv = sum(new), case["d"], case["hq"], case["hkv"]
    if case["op"] == "append":
        return {"bytes": 2 * 2 * N * d * (hq + 2 * hkv) + 12 * N, "flops": 3.0 * N * (hq + hkv) * case["rot"]}
    win = case["window"]
    keys = pairs = 0
    for n, t in zip(new, total):
        first = t - n + 1                                        # keys the first new token may see
        keys += min(t, n - 1 + win) if win else t
        if not win:
            pairs += n * first + n * (n - 1) // 2
        else:
            grow = max(0, min(n, win - first))                   # tokens that see fewer than the window
            pairs += grow * first + grow * (grow - 1) // 2 + (n - grow) * win
    return {"bytes": 2 * (2 * N * hq * d + 2 * keys * hkv * d) + 4 * keys / case["page"],
            "flops": 4.0 * pairs * hq * d}


# ---------------------------------------------------------------------------
# the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](s)


def _exact_append(s):
    starts, lens, table = s["q_start"].tolist(), s["kv_len"].tolist(), s["pages"].tolist()
    keys, values = s["k_cache"].double(), s["v_cache"].double()
    q = s["q"].double()
    rot, half = s["rot"], s["rot"] // 2
    first = torch.arange(half, device="cuda") * (2 if s["interleaved"] else 1)
    second = first + (1 if s["interleaved"] else half)
    for b in range(s["batch"]):
        t0, t1 = starts[b], starts[b + 1]
        slot = torch.arange(lens[b] - (t1 - t0), lens[b], device="cuda")
        turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                           slot.double().view(-1, 1, 1) * s["inv_freq"])
        k = s["k"][t0:t1].double()
        for x in (k, q[t0:t1]):
            y = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = y.real, y.imag
        page = torch.tensor(table[b], device="cuda")[slot // s["page"]]
        keys[page, slot % s["page"]] = k
        values[page, slot % s["page"]] = s["v"][t0:t1].double()
    return {"q": q, "k_cache": keys, "v_cache": values}


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
            k = s["k_cache"][mine, :, h].reshape(-1, s["d"])[:L].double()
            v = s["v_cache"][mine, :, h].reshape(-1, s["d"])[:L].double()
            for i in range(h * G, h * G + G):
                a = (s["q"][t0:t1, i].double() @ k.t() / math.sqrt(s["d"])).masked_fill_(hide, -math.inf)
                out[t0:t1, i] = torch.softmax(a, dim=-1) @ v
    return {"out": out}


def _exact_sample(s):
    R, V = s["z"].shape
    tokens, rows = [], []
    for r in range(R):
        z = s["z"][r].double()
        weight = torch.exp((z - z.max()) / s["temperature"][r].double())
        # ascending by value and, among equals, from the highest index down: read backwards
        best = (V - 1 - torch.sort(z.flip(0), stable=True).indices).flip(0)
        count = V
        if s["top_k"] is not None and 0 < int(s["top_k"][r]) < V:
            count = int(s["top_k"][r])
        mass = weight[best[:count]]
        if s["top_p"] is not None and float(s["top_p"][r]) < 1:
            goal = s["top_p"][r].double() * mass.sum()
            upto = torch.cat((mass.new_zeros(1), mass.cumsum(0)[:-1]))
            count = max(1, int((upto < goal).sum()))
        if s["min_p"] is not None:
            count = max(1, min(count, int((mass >= s["min_p"][r].double()).sum())))
        left = torch.zeros_like(weight)
        left[best[:count]] = weight[best[:count]]
        sums = left.cumsum(0)
        if s["u"] is not None:
            t = int(torch.searchsorted(sums, (s["u"][r] * sums[-1]).view(1), right=True))
            tokens.append(min(t, int(left.nonzero().max())))
        if s["probs"]:
            rows.append(left / sums[-1])
    out = {}
    if s["u"] is not None:
        out["token"] = torch.tensor(tokens, dtype=torch.int32, device="cuda")
    if s["probs"]:
        out["probs"] = torch.stack(rows)
    return out
