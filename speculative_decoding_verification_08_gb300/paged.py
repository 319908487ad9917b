"""A paged key/value cache for several sequences, on top of ``append_kv`` and
``paged_attention``: the pages, the page table and the lengths that those calls
take, and the rollback of rejected drafts.

One ``PagedCache`` holds the keys and values of one or more layers; all layers
share the page table.  A pass over new tokens is::

    cache.begin({seq: n_new, ...})            # pages for them, the batch's arrays
    for layer in range(layers):
        q = cache.append(layer, q, k, v)      # rotated by position, written
        x = cache.attend(layer, q)
    ...
    cache.rollback(seq, n_rejected)           # the last tokens leave again

Token rows are ordered by sequence, in the order ``begin`` was given them.
Rolled-back slots are simply written again by the next pass; pages that no
token uses any more go back to the pool.

With ``dtype=torch.float8_e4m3fn`` the cache holds 8-bit values and a power of
two for each vector; tokens stay in 16 bits, and ``read`` takes sequences back
to them.
"""
from __future__ import annotations

from typing import Dict, List, Optional

from . import SpecVerifyError, _torch, append_kv, paged_attention, read_kv


def rope_frequencies(rot_dim: int, base: float = 10000.0, device=None):
    """Radians per position of each of a head's rot_dim / 2 pairs, f64:
    base^(-2 i / rot_dim)."""
    torch = _torch()
    if rot_dim < 0 or rot_dim % 4:
        raise ValueError("rot_dim must be a multiple of 4")
    i = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
    return torch.pow(float(base), -2.0 * i / max(rot_dim, 1))


class PagedCache:
    """Keys and values of ``layers`` layers in ``num_pages`` pages of
    ``page_size`` slots (heads first within a page: a head's slots lie
    together).  ``inv_freq`` as for ``append_kv`` (None: no rotation).  dtype:
    the tokens' (bfloat16 by default), or float8_e4m3fn, whose scales are
    ``k_scale`` and ``v_scale`` (None otherwise)."""

    def __init__(self, layers: int, num_pages: int, page_size: int, kv_heads: int, head_dim: int,
                 dtype=None, device=None, inv_freq=None, interleaved: bool = False):
        torch = _torch()
        if layers < 1 or num_pages < 1:
            raise ValueError("layers and num_pages must be >= 1")
        self.device = torch.device("cuda") if device is None else torch.device(device)
        dtype = torch.bfloat16 if dtype is None else dtype
        shape = (layers, num_pages, kv_heads, page_size, head_dim)
        # zeros: a page's unused slots are never read as numbers, but a cache
        # of old bits would make dumps hard to read
        self.k = torch.zeros(shape, dtype=dtype, device=self.device).transpose(2, 3)
        self.v = torch.zeros(shape, dtype=dtype, device=self.device).transpose(2, 3)
        self.k_scale = self.v_scale = None
        if dtype == torch.float8_e4m3fn:
            # (bytes of zero: the smallest scale, for codes of zero)
            self.k_scale, self.v_scale = (
                torch.zeros(shape[:-1], dtype=torch.uint8, device=self.device).view(torch.float8_e8m0fnu).transpose(2, 3)
                for _ in range(2))
        self.page_size, self.inv_freq, self.interleaved = page_size, inv_freq, interleaved
        self.free: List[int] = list(range(num_pages - 1, -1, -1))
        self.owned: Dict[object, List[int]] = {}
        self.length: Dict[object, int] = {}
        self._batch = None

    def begin(self, new: Dict[object, int]) -> None:
        """Makes room for new[seq] more tokens of every seq (a new one is added)
        and sets up the arrays of a pass over them.  Nothing changes when the
        pool has too few pages left."""
        torch = _torch()
        if not new:
            raise ValueError("a pass needs at least one sequence")
        need = {}
        for seq, n in new.items():
            if n < 1:
                raise ValueError("a pass needs at least one token of each sequence")
            have = len(self.owned.get(seq, ()))
            total = self.length.get(seq, 0) + n
            need[seq] = max(0, -(-total // self.page_size) - have)
        if sum(need.values()) > len(self.free):
            raise SpecVerifyError(f"out of pages: {sum(need.values())} wanted, {len(self.free)} free")
        for seq, n in new.items():
            pages = self.owned.setdefault(seq, [])
            for _ in range(need[seq]):
                pages.append(self.free.pop())
            self.length[seq] = self.length.get(seq, 0) + n
        rows = [self.owned[seq] for seq in new]
        wide = max(len(r) for r in rows)
        table = torch.tensor([r + [0] * (wide - len(r)) for r in rows], dtype=torch.int32)
        starts = [0]
        for n in new.values():
            starts.append(starts[-1] + n)
        self._batch = (table.to(self.device),
                       torch.tensor(starts, dtype=torch.int32).to(self.device),
                       torch.tensor([self.length[s] for s in new], dtype=torch.int32).to(self.device))

    def _pass(self):
        if self._batch is None:
            raise SpecVerifyError("begin() comes first")
        return self._batch

    def _scales(self, layer: int):
        return {} if self.k_scale is None else dict(k_scale=self.k_scale[layer], v_scale=self.v_scale[layer])

    def append(self, layer: int, q, k, v, ws=None, q_norm=None, k_norm=None, eps: float = 1e-6):
        """Writes the pass's keys and values of a layer; returns q rotated.
        (ws as for ``append_kv``: a pass captured into a graph needs one; norms
        as there.)"""
        return append_kv(k, v, self.k[layer], self.v[layer], *self._pass(), inv_freq=self.inv_freq,
                         q=q, interleaved=self.interleaved, q_norm=q_norm, k_norm=k_norm, eps=eps, ws=ws,
                         **self._scales(layer))

    def attend(self, layer: int, q, scale: Optional[float] = None, window: int = 0, ws=None):
        """The pass's queries over a layer of the cache."""
        return paged_attention(q, self.k[layer], self.v[layer], *self._pass(), scale=scale,
                               window=window, ws=ws, **self._scales(layer))

    def read(self, layer: int, seqs=None, dtype=None, ws=None) -> Dict[object, tuple]:
        """What a layer holds of the sequences (all by default): seq -> (k, v),
        [length][kv_heads][head_dim], in 16 bits (``dtype`` as for ``read_kv``)."""
        torch = _torch()
        seqs = list(self.length if seqs is None else seqs)
        lengths = [self._held(s) for s in seqs]
        rows = [self.owned[s] for s in seqs]
        wide = max([len(r) for r in rows] + [1])
        starts = [0]
        for n in lengths:
            starts.append(starts[-1] + n)
        k, v = read_kv(self.k[layer], self.v[layer],
                       torch.tensor([r + [0] * (wide - len(r)) for r in rows], dtype=torch.int32)
                       .view(len(seqs), wide).to(self.device),
                       torch.tensor(starts, dtype=torch.int32).to(self.device),
                       torch.tensor(lengths, dtype=torch.int32).to(self.device), rows=starts[-1], dtype=dtype, ws=ws,
                       **self._scales(layer))
        return {s: (k[a:b], v[a:b]) for s, a, b in zip(seqs, starts, starts[1:])}

    def rollback(self, seq, n: int) -> None:
        """Drops a sequence's last n tokens."""
        held = self._held(seq)
        if n < 0 or n > held:
            raise ValueError(f"cannot drop {n} of {held} tokens")
        self.length[seq] = held - n
        self._trim(seq)
        self._batch = None

    def drop(self, seq) -> None:
        """Forgets a sequence; its pages go back to the pool."""
        self._held(seq)
        self.length[seq] = 0
        self._trim(seq)
        del self.length[seq], self.owned[seq]
        self._batch = None

    def _held(self, seq) -> int:
        if seq not in self.length:
            raise ValueError(f"no sequence {seq!r} in the cache")
        return self.length[seq]

    def _trim(self, seq) -> None:
        keep = -(-self.length[seq] // self.page_size)
        pages = self.owned[seq]
        while len(pages) > keep:
            self.free.append(pages.pop())
