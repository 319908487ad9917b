"""64-bit references of head norms and of the 8-bit cache, for the tests (plain
loops; test infrastructure only)."""
import math

import torch

from cache_refs import CacheBatch, rotate

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def power(e):
    """2^e, exact, for an integer tensor."""
    return torch.ldexp(torch.ones(e.shape, dtype=torch.float64), e)


def scale_exponents(y):
    """Exponent of each vector's scale [...], y [..., d] finite f64: the smallest
    e in [-100, 100] with max |y| <= 448 * 2^e."""
    top = y.abs().amax(-1)
    e = torch.full(top.shape, -100, dtype=torch.int32)
    for c in range(-100, 100):
        e = torch.where(top > 448 * 2.0 ** c, c + 1, e)
    return e


def quantise(y):
    """(codes, scales) of finite fp32 vectors y [..., d] on the CPU."""
    e = scale_exponents(y.double())
    code = (y.double() * power(-e).unsqueeze(-1)).clamp(-448, 448).float().to(E4M3)
    return code, (e + 127).to(torch.uint8).view(E8M0)


def values(code, scale):
    """What codes [..., d] and scales [...] stand for, f64, on the CPU."""
    b = scale.cpu().view(torch.uint8).int()
    s = power(torch.where(b == 255, 127, b) - 127)
    s = torch.where(b == 255, math.nan, s)
    return code.cpu().float().double() * s.unsqueeze(-1)


def normed(x, weight, eps):
    """(x normed by heads, relative tolerance) in fp64.  fp32: a sum of d squares
    (d / 8 + 4 roundings in a row, halved by the root), the root and quotient of
    2^-22 together, and two products."""
    y = x.cpu().double()
    d = y.shape[-1]
    if weight is None:
        return y, 0.0
    r = torch.rsqrt(y.square().mean(-1, keepdim=True) + eps)
    return y * r * weight.cpu().double(), (d / 16 + 8) * 2.0 ** -23


def turned(x, weight, eps, pos, inv_freq, interleaved):
    """(normed and rotated x, tolerance before its one rounding), f64."""
    y, rel = normed(x, weight, eps)
    if inv_freq is None:
        return y, y.abs() * rel
    half = inv_freq.numel()
    o, _ = rotate(y, pos, inv_freq, interleaved)
    i = torch.arange(half)
    a, c = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    tol = y.abs() * rel
    both = (y[..., a].abs() + y[..., c].abs()) * (rel + 2.0 ** -21)
    tol[..., a], tol[..., c] = both, both
    return o, tol


class EightBatch(CacheBatch):
    """A CacheBatch whose caches are 8-bit: codes and scales; unused slots hold the
    code NaN and the scale NaN."""

    def __init__(self, seqs, hkv, d, page, dtype, heads_first=False, seed=0, fill=True, extra_tokens=0, spread=1.0,
                 scale_spread=1.0):
        super().__init__(seqs, hkv, d, page, torch.float32, device="cpu", heads_first=heads_first, seed=seed,
                         fill=fill, extra_tokens=extra_tokens, spread=spread)
        self.dtype, self.device = dtype, "cuda"
        for name in ("pages", "q_start", "kv_len"):
            setattr(self, name, getattr(self, name).cuda())
        for name in ("k", "v"):
            x = getattr(self, name)
            size = torch.exp(torch.randn(*x.shape[:3], generator=self.gen) * scale_spread)
            x = x * size.unsqueeze(-1)
            used = ~torch.isnan(x).any(-1)
            code, scale = quantise(torch.where(used.unsqueeze(-1), x, 0.0))
            code.view(torch.uint8)[~used] = 0x7f
            scale.view(torch.uint8)[~used] = 255
            if heads_first:
                code, scale = (y.view(torch.uint8).transpose(1, 2).contiguous().transpose(1, 2) for y in (code, scale))
            setattr(self, name + "8", code.cuda().view(E4M3))
            setattr(self, name + "s", scale.cuda().view(E8M0))
            # what the cache stands for
            setattr(self, name, values(code.contiguous().view(E4M3), scale.contiguous().view(E8M0)))

    def eight(self):
        return self.k8, self.v8, self.pages, self.q_start, self.kv_len

    def scales(self):
        return dict(k_scale=self.ks, v_scale=self.vs)

    def refresh(self):
        """Takes what the caches stand for from the device again."""
        self.k, self.v = values(self.k8, self.ks), values(self.v8, self.vs)
