"""Speculative decoding against a target with a paged cache, end to end on the
GPU: a small decoder with random weights is the target, its first layer alone
the draft.

Each round the draft proposes tokens (``warp_sample`` draws them and returns the
rows q they were drawn from), the target runs once over [pending, drafts]
(``append_kv``, ``paged_attention``), its logits are warped alike into the rows
p (``warp_sample``), and the verification decides (``verify_round`` through
``PendingTokenDecoder``).  Rejected drafts leave the cache by rollback.

With ``--eight`` the caches hold 8-bit values; with ``--norms`` queries and keys
are normed by heads before they turn.

    python examples/paged_decoding.py [--new 64] [--k 5] [--sampling] [--eight] [--norms]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import speculative_decoding_verification_08_gb300 as sv  # noqa: E402
from speculative_decoding_verification_08_gb300.decoder import PendingTokenDecoder  # noqa: E402
from speculative_decoding_verification_08_gb300.paged import PagedCache, rope_frequencies  # noqa: E402


class TinyDecoder:
    """A decoder with random weights: attention over a paged cache and a gated
    feed-forward per layer.  ``layers`` of it may be run."""

    def __init__(self, vocab=4096, dim=256, layers=2, heads=4, kv_heads=2, head_dim=64, seed=0,
                 eight=False, norms=False):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(a, b, scale=1.0):
            w = torch.randn(a, b, generator=g, device="cuda") * (scale * a ** -0.5)
            return w.to(torch.bfloat16)

        self.heads, self.kv_heads, self.head_dim, self.layers = heads, kv_heads, head_dim, layers
        self.embed = weight(vocab, dim, vocab ** 0.5)
        # later layers change the first one's answer by little, so that its
        # logits make a useful draft
        self.blocks = [dict(qkv=weight(dim, (heads + 2 * kv_heads) * head_dim),
                            out=weight(heads * head_dim, dim, 0.3 if i else 1.0),
                            up=weight(dim, 4 * dim), down=weight(2 * dim, dim, 0.3 if i else 1.0))
                       for i in range(layers)]
        self.head = weight(dim, vocab, 4.0)
        self.inv_freq = rope_frequencies(head_dim, device="cuda")
        self.eight = eight
        # (drawn last: the other weights are the same with and without)
        self.norms = [{f"{x}_norm": (1 + weight(head_dim, 1).view(-1)) if norms else None for x in "qk"}
                      for _ in range(layers)]

    def cache(self, layers, pages=64, page_size=16):
        return PagedCache(layers, pages, page_size, self.kv_heads, self.head_dim,
                          dtype=torch.float8_e4m3fn if self.eight else torch.bfloat16, inv_freq=self.inv_freq)

    @staticmethod
    def norm(x):
        y = x.float()
        return (y * torch.rsqrt(y.pow(2).mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def forward(self, cache, seq, tokens, layers):
        """Logits [len(tokens)][vocab] of the tokens, which enter the cache."""
        n, d = len(tokens), self.head_dim
        cache.begin({seq: n})
        x = self.embed[torch.tensor(tokens, device="cuda")]
        for i, b in enumerate(self.blocks[:layers]):
            qkv = (self.norm(x) @ b["qkv"]).view(n, -1, d)
            q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
            q = cache.append(i, q, k, v, **self.norms[i])
            x = x + cache.attend(i, q).reshape(n, -1) @ b["out"]
            gate, up = (self.norm(x) @ b["up"]).chunk(2, dim=-1)
            x = x + (torch.nn.functional.silu(gate) * up) @ b["down"]
        return self.norm(x) @ self.head


class Warp:
    """The filters both distributions go through: temperature, top-k, top-p,
    min-p, for any number of rows."""

    def __init__(self, temperature=0.8, top_k=50, top_p=0.95, min_p=0.02):
        self.values = dict(temperature=(temperature, torch.float32), top_k=(top_k, torch.int32),
                           top_p=(top_p, torch.float32), min_p=(min_p, torch.float32))

    def __call__(self, z, u=None):
        rows = z.shape[0]
        filters = {k: torch.full((rows,), x, dtype=t, device="cuda") for k, (x, t) in self.values.items()}
        return sv.warp_sample(z, u, probs=True, **filters)


class PagedTarget:
    """The target as ``PendingTokenDecoder`` drives it: forward() over new tokens,
    rollback() of rejected ones."""

    def __init__(self, model, warp, layers=None):
        self.model, self.warp = model, warp
        self.layers = model.layers if layers is None else layers
        self.cache = model.cache(self.layers)

    def forward(self, tokens):
        return self.warp(self.model.forward(self.cache, 0, tokens, self.layers))[1]

    def rollback(self, n):
        self.cache.rollback(0, n)


class PagedDraft:
    """Draft steps of the first layer, on a cache of its own that follows the
    committed prefix."""

    def __init__(self, model, warp, seed=1, greedy=True):
        self.model, self.warp, self.greedy = model, warp, greedy
        self.cache, self.seen = model.cache(1), []
        self.gen = torch.Generator(device="cuda").manual_seed(seed)

    def __call__(self, prefix, k):
        # drop what the verification did not keep, then catch up
        same = 0
        while same < min(len(self.seen), len(prefix) - 1) and self.seen[same] == prefix[same]:
            same += 1
        if len(self.seen) > same:
            self.cache.rollback(0, len(self.seen) - same)
            self.seen = self.seen[:same]
        tokens, rows, feed = [], [], list(prefix[same:])
        for _ in range(k):
            z = self.model.forward(self.cache, 0, feed, 1)[-1:]
            self.seen += feed
            u = torch.rand(1, generator=self.gen, device="cuda", dtype=torch.float64)
            token, q = self.warp(z, u)
            t = int(q[0].argmax()) if self.greedy else int(token[0])
            tokens.append(t)
            rows.append(q[0])
            feed = [t]
        return tokens, torch.stack(rows)


def decode(prompt, max_new=64, k=5, greedy=True, seed=0, **model):
    """(tokens, tokens a round on average) of a generation with the tiny model."""
    model, warp = TinyDecoder(**model), Warp()
    dec = PendingTokenDecoder(PagedDraft(model, warp, greedy=greedy), PagedTarget(model, warp), k=k,
                              greedy=greedy, seed=seed)
    out = dec.generate(prompt, max_new)
    return out, sum(n + 1 for _, n, _ in dec.trace) / len(dec.trace)


def plain(prompt, max_new=64, **model):
    """The same target without speculation, one token at a time."""
    target = PagedTarget(TinyDecoder(**model), Warp())
    feed, out = list(prompt), []
    while len(out) < max_new:
        feed = [int(target.forward(feed)[-1].argmax())]
        out += feed
    return out


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--new", type=int, default=64)
    ap.add_argument("--k", type=int, default=5)
    ap.add_argument("--sampling", action="store_true")
    ap.add_argument("--eight", action="store_true")
    ap.add_argument("--norms", action="store_true")
    a = ap.parse_args()
    prompt = [11, 222, 3333, 44, 5]
    model = dict(eight=a.eight, norms=a.norms)
    out, rate = decode(prompt, a.new, a.k, not a.sampling, **model)
    print("tokens:", out)
    print(f"{rate:.2f} tokens a target pass")
    if not a.sampling:
        same = sum(x == y for x, y in zip(out, plain(prompt, a.new, **model)))
        print(f"{same} of {len(out)} as without speculation")


if __name__ == "__main__":
    main()
