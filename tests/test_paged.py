"""PagedCache: its pages and lengths (CPU), and a decoder over it end to end
(GPU): a speculated stream is the one the target gives alone."""
import importlib.util
import os

import pytest
import torch

import speculative_decoding_verification_08_gb300 as sv
from speculative_decoding_verification_08_gb300.paged import PagedCache, rope_frequencies
from cache_refs import attention, CacheBatch, default_scale, rotate

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def host_cache(pages=6, page_size=8):
    return PagedCache(2, pages, page_size, 1, 8, device="cpu")


def test_pages_follow_the_lengths():
    c = host_cache()
    c.begin({"a": 5, "b": 9})
    table, start, length = c._pass()
    assert start.tolist() == [0, 5, 14] and length.tolist() == [5, 9]
    assert len(c.owned["a"]) == 1 and len(c.owned["b"]) == 2 and len(c.free) == 3
    assert table[0, 0] == c.owned["a"][0] and table[1].tolist() == c.owned["b"]
    c.begin({"b": 1, "a": 4})                      # another order, one more page for a
    _, start, length = c._pass()
    assert start.tolist() == [0, 1, 5] and length.tolist() == [10, 9]
    used = c.owned["a"] + c.owned["b"]
    assert len(set(used)) == 4 and not set(used) & set(c.free)
    c.rollback("b", 3)                             # 7 tokens: one page goes back
    assert c.length["b"] == 7 and len(c.owned["b"]) == 1 and len(c.free) == 3
    with pytest.raises(sv.SpecVerifyError):
        c._pass()                                  # the arrays of the pass are stale
    c.rollback("a", 9)
    assert c.length["a"] == 0 and c.owned["a"] == [] and len(c.free) == 5
    c.drop("b")
    assert sorted(c.free) == list(range(6)) and "b" not in c.length


def test_a_full_pool_refuses_and_changes_nothing():
    c = host_cache(pages=2)
    c.begin({"a": 8})
    before = (dict(c.length), list(c.free), {k: list(v) for k, v in c.owned.items()})
    with pytest.raises(sv.SpecVerifyError):
        c.begin({"a": 1, "b": 8})
    assert before == (c.length, c.free, c.owned)
    for bad in (lambda: c.begin({"a": 0}), lambda: c.rollback("a", 9), lambda: c.rollback("a", -1),
                lambda: c.begin({}), lambda: c.rollback("z", 0), lambda: c.drop("z")):
        with pytest.raises(ValueError):
            bad()


def test_frequencies():
    f = rope_frequencies(8, 100.0)
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75]).double())
    assert rope_frequencies(0).numel() == 0
    with pytest.raises(ValueError):
        rope_frequencies(6)


def example():
    spec = importlib.util.spec_from_file_location("paged_decoding", os.path.join(ROOT, "examples", "paged_decoding.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.gpu
def test_passes_and_rollbacks_leave_the_right_cache():
    """A prompt, a round with drafts, a rollback and another round: the last
    pass's output is that of the final sequence."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.build()
    d, f = 64, rope_frequencies(64, device="cuda")
    c = PagedCache(1, 20, 16, 2, d, inv_freq=f)
    g = torch.Generator().manual_seed(3)
    rnd = lambda n, h: torch.randn(n, h, d, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
    kept, held = {0: [], 1: []}, {}

    def step(new):
        n = sum(new.values())
        q, k, v = rnd(n, 4), rnd(n, 2), rnd(n, 2)
        c.begin(new)
        q = c.append(0, q, k, v)
        at = 0
        for s, m in new.items():
            kept[s] += [(k[at + i], v[at + i]) for i in range(m)]
            at += m
        held.update(q=q, out=c.attend(0, q), new=new)

    step({0: 40, 1: 3})
    step({0: 6, 1: 6})
    for s, n in ((0, 4), (1, 5)):
        c.rollback(s, n)
        del kept[s][-n:]
    step({1: 6, 0: 6})
    # the same from scratch
    seqs = [(6, len(kept[s])) for s in held["new"]]
    cb = CacheBatch(seqs, 2, d, 16, torch.bfloat16, fill=False)
    for b, s in enumerate(held["new"]):
        k = torch.stack([x for x, _ in kept[s]])
        v = torch.stack([x for _, x in kept[s]])
        kr = rotate(k, torch.arange(len(kept[s])), f, False)[0].to(torch.bfloat16)
        for i in range(len(kept[s])):
            p = int(cb.table[b, i // 16])
            cb.k[p, i % 16], cb.v[p, i % 16] = kr[i].cuda(), v[i]
    want, tol = attention(cb, held["q"], default_scale(d), 0)
    # keys may be rounded the other way where cos and sin differ in the last bit
    off = (held["out"].cpu().double() - want).abs()
    assert bool((off <= 2 * tol + 2.0 ** -8 * want.abs().max()).all())


@pytest.mark.gpu
def test_speculation_does_not_change_the_greedy_stream():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.build()
    m = example()
    prompt = [11, 222, 3333, 44, 5]
    out, rate = m.decode(prompt, 48, 5, greedy=True)
    # the target's rows depend on how many tokens share a pass only through
    # roundings of the library products; the streams may part at a near tie
    ref = m.plain(prompt, 48)
    same = 0
    while same < 48 and out[same] == ref[same]:
        same += 1
    assert len(out) == 48 and same >= 16, (same, out, ref)
    assert rate > 1.2


@pytest.mark.gpu
def test_sampled_stream_is_reproducible():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.build()
    m = example()
    a, rate = m.decode([7, 8, 9], 32, 4, greedy=False, seed=5)
    b, _ = m.decode([7, 8, 9], 32, 4, greedy=False, seed=5)
    assert a == b and len(a) == 32 and 1.0 <= rate <= 5.0
