"""64-bit references of the paged-cache calls and of warp_sample, and batch
builders, for the tests (plain loops over sequences and rows; test
infrastructure only)."""
import math

import numpy as np
import torch


class CacheBatch:
    """A paged cache with scattered pages and a batch of (n, length) sequences
    on `device`; unused slots hold NaN."""

    def __init__(self, seqs, hkv, d, page, dtype, device="cuda", heads_first=False, seed=0,
                 fill=True, extra_tokens=0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.hkv, self.d, self.page, self.dtype = seqs, hkv, d, page, dtype
        self.device = device
        need = [-(-t // page) for _, t in seqs]
        self.wide = max(need + [1])
        pool = sum(need) + 2
        perm = torch.randperm(pool, generator=g).tolist()
        table = torch.full((len(seqs), self.wide), -7, dtype=torch.int32)   # entries nobody reads
        at = 0
        for b, c in enumerate(need):
            table[b, :c] = torch.tensor(perm[at:at + c], dtype=torch.int32)
            at += c
        starts = [0]
        for n, _ in seqs:
            starts.append(starts[-1] + n)
        self.N = starts[-1] + extra_tokens
        shape = (pool, hkv, page, d) if heads_first else (pool, page, hkv, d)
        k = torch.full(shape, float("nan"))
        v = torch.full(shape, float("nan"))
        if heads_first:
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        if fill:
            for b, (_, t) in enumerate(seqs):
                for s in range(t):
                    p = int(table[b, s // page])
                    k[p, s % page] = torch.randn(hkv, d, generator=g) * spread
                    v[p, s % page] = torch.randn(hkv, d, generator=g)
        self.k, self.v = k.to(dtype).to(device), v.to(dtype).to(device)
        self.pages = table.to(device)
        self.q_start = torch.tensor(starts, dtype=torch.int32, device=device)
        self.kv_len = torch.tensor([t for _, t in seqs], dtype=torch.int32, device=device)
        self.table, self.starts = table, starts
        self.gen = g

    def tokens(self, heads, scale=1.0):
        x = torch.randn(self.N, heads, self.d, generator=self.gen) * scale
        return x.to(self.dtype).to(self.device)

    def args(self):
        return self.k, self.v, self.pages, self.q_start, self.kv_len

    def sequence(self, cache, b):
        """[length][hkv][d] of sequence b in fp64."""
        t = self.seqs[b][1]
        if t == 0:
            return torch.zeros(0, self.hkv, self.d, dtype=torch.float64)
        p = self.table[b, :-(-t // self.page)].long()
        return cache.cpu()[p].reshape(-1, self.hkv, self.d)[:t].double()


def attention(cb, q, scale, window):
    """(out, tolerance) in fp64, per element.

    Tolerance: the weights are rounded to the cache's type (eps / 2 of the
    mass-weighted |v|), the result is rounded once (eps / 2 of it); scores carry
    fp32 errors of at most (d + 4) 2^-24 of sum |q||k| scale, which act on the
    weights' exponents, exp2 one of 2^-21, and the fp32 sums over the keys one
    of (L / 8 + 64) 2^-23."""
    eps = torch.finfo(cb.dtype).eps / 2
    G = q.shape[1] // cb.hkv
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol = torch.zeros(q.shape, dtype=torch.float64)
    qd = q.cpu().double()
    for b, (n, L) in enumerate(cb.seqs):
        if n == 0:
            continue
        K, V = cb.sequence(cb.k, b), cb.sequence(cb.v, b)
        pos = torch.arange(L)
        for j in range(n):
            last = L - n + j
            seen = pos <= last
            if window:
                seen &= pos > last - window
            if not bool(seen.any()):
                continue
            t = cb.starts[b] + j
            k, v = K[seen], V[seen]
            for h in range(q.shape[1]):
                g = h // G
                s = (k[:, g] @ qd[t, h]) * scale
                mag = float((k[:, g].abs() @ qd[t, h].abs()).max()) * abs(scale)
                p = torch.softmax(s, 0)
                o = p @ v[:, g]
                a = p @ v[:, g].abs()
                out[t, h] = o
                tol[t, h] = eps * (a + o.abs()) + a * (2 * (cb.d + 4) * 2.0 ** -24 * mag + 2.0 ** -21
                                                       + (len(s) / 8 + 64) * 2.0 ** -23)
    return out, tol


def rotate(x, pos, inv_freq, interleaved):
    """(x rotated, tolerance) in fp64: fp32 products and sums of values good to
    2^-22 (cos, sin, angle), then one rounding of the result."""
    half = inv_freq.numel()
    eps = torch.finfo(x.dtype).eps / 2
    y = x.cpu().double()
    o, tol = y.clone(), torch.zeros_like(y)
    if half:
        i = torch.arange(half)
        a, c = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = pos.double().view(-1, 1, 1) * inv_freq.cpu().view(1, 1, -1)
        cos, sin = torch.cos(ang), torch.sin(ang)
        o[..., a] = y[..., a] * cos - y[..., c] * sin
        o[..., c] = y[..., a] * sin + y[..., c] * cos
        mag = (y[..., a].abs() + y[..., c].abs()) * 2.0 ** -21
        tol[..., a] = o[..., a].abs() * eps + mag
        tol[..., c] = o[..., c].abs() * eps + mag
    return o, tol


def warp_row(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, u=None):
    """(probs f64, kept mask, token) of one row of logits by the definition."""
    z = np.asarray(z, dtype=np.float64)
    V = z.size
    w = np.exp((z - z.max()) / temperature)
    order = np.lexsort((np.arange(V), -z))
    m = top_k if 0 < top_k < V else V
    s = w[order[:m]]
    if top_p < 1:
        before = np.concatenate(([0.0], np.cumsum(s)[:-1]))
        m = max(1, int((before < top_p * s.sum()).sum()))
    if min_p > 0:
        m = max(1, min(m, int((s >= min_p).sum())))
    kept = np.zeros(V, dtype=bool)
    kept[order[:m]] = True
    w = np.where(kept, w, 0.0)
    token = None
    if u is not None:
        over = np.nonzero(np.cumsum(w) > u * w.sum())[0]
        token = int(over[0]) if over.size else int(np.nonzero(w)[0][-1])
    return w / w.sum(), kept, token


def default_scale(d):
    return 1.0 / math.sqrt(d)
