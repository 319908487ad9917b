"""append_kv and paged_attention against their 64-bit definitions, at the sizes
and masks where they can go wrong.  Unused slots of every page hold NaN, and
the page table's unread entries are invalid."""
import math

import pytest
import torch

import speculative_decoding_verification_08_gb300 as sv
from cache_refs import CacheBatch, attention, default_scale, rotate

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.build()
    return sv.load()


def within(got, want, tol):
    off = (got.cpu().double() - want).abs()
    bad = ~(off <= tol)
    assert not bool(bad.any()), f"{int(bad.sum())} values off, worst {float(off.max())}"


def freqs(rot, device="cuda"):
    i = torch.arange(rot // 2, dtype=torch.float64, device=device)
    return torch.pow(10000.0, -2.0 * i / max(rot, 1))


# ---------------------------------------------------------------------------
# append

APPEND = [
    # sequences (new, length), q heads, kv heads, d, page, type, rot, interleaved, heads first
    ([(1, 1)], 1, 1, 64, 16, BF, 64, False, False),
    ([(1, 701)], 32, 8, 128, 64, BF, 128, False, True),
    ([(6, 6), (6, 70), (6, 129)], 8, 2, 128, 64, HF, 128, False, True),
    ([(0, 33), (5, 40), (0, 0), (17, 17)], 6, 2, 96, 48, BF, 48, False, False),
    ([(33, 97), (1, 20)], 4, 4, 80, 16, HF, 40, False, True),
    ([(9, 64), (3, 3)], 3, 1, 64, 8, BF, 32, True, False),
    ([(9, 9), (2, 31)], 7, 1, 8, 8, HF, 4, True, True),
    ([(4, 9)], 2, 2, 24, 24, BF, 0, False, False),
]


@pytest.mark.parametrize("case", APPEND)
def test_append_rotates_and_writes_only_its_slots(case):
    seqs, hq, hkv, d, page, dt, rot, inter, first = case
    cb = CacheBatch(seqs, hkv, d, page, dt, heads_first=first, fill=False, seed=3)
    k, v, q = cb.tokens(hkv), cb.tokens(hkv), cb.tokens(hq)
    kept = [x.clone() for x in (k, v, q)]
    f = freqs(rot) if rot else None
    ws = sv.CacheWorkspace()
    got = sv.append_kv(k, v, *cb.args(), inv_freq=f, q=q, interleaved=inter, ws=ws)
    assert ws.status() == 0
    for x, y in zip((k, v, q), kept):
        assert torch.equal(x, y)
    pos = torch.cat([torch.arange(t - n, t) for n, t in seqs])
    fr = f if rot else torch.zeros(0, dtype=torch.float64)
    within(got, *rotate(q, pos, fr, inter))
    kr, kt = rotate(k, pos, fr, inter)
    kc, vc = cb.k.cpu(), cb.v.cpu()
    written = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for b, (n, t) in enumerate(seqs):
        for j in range(n):
            s = t - n + j
            p, at, row = int(cb.table[b, s // page]), s % page, cb.starts[b] + j
            written[p, at] = True
            within(kc[p, at], kr[row], kt[row])
            assert torch.equal(vc[p, at], v[row].cpu())
    assert bool(torch.isnan(kc[~written]).all()) and bool(torch.isnan(vc[~written]).all())


def test_append_many_tokens_takes_several_per_block():
    cb = CacheBatch([(9000, 9000), (7400, 7411)], 1, 16, 64, BF, fill=False)
    k, v = cb.tokens(1), cb.tokens(1)
    f = freqs(16)
    assert sv.append_kv(k, v, *cb.args(), inv_freq=f) is None
    pos = torch.cat((torch.arange(9000), torch.arange(11, 7411)))
    kr, kt = rotate(k, pos, f, False)
    lens = [t for _, t in cb.seqs]
    for b, (n, t) in enumerate(cb.seqs):
        got = cb.sequence(cb.k, b)[t - n:]
        within(got, kr[cb.starts[b]:cb.starts[b + 1]], kt[cb.starts[b]:cb.starts[b + 1]])
        assert torch.equal(cb.sequence(cb.v, b)[t - n:], v[cb.starts[b]:cb.starts[b + 1]].cpu().double())
    assert lens == [9000, 7411]


def test_append_positions_far_out_and_in_place_on_a_slice():
    """Angles of positions near 2^30 keep their digits; q and k are slices of
    one fused projection and q is rotated in place."""
    cb = CacheBatch([(5, 12)], 2, 64, 16, HF, fill=False)
    fused = torch.randn(5, 8 * 64, generator=torch.Generator().manual_seed(1)).to(HF).cuda()
    q = fused[:, :4 * 64].view(5, 4, 64)
    k = fused[:, 4 * 64:6 * 64].view(5, 2, 64)
    v = fused[:, 6 * 64:].view(5, 2, 64)
    pos = torch.tensor([0, 1, 1 << 20, (1 << 30) + 7, 3], dtype=torch.int32, device="cuda")
    f = freqs(64)
    want, tol = rotate(q, pos.cpu(), f, False)
    kw, kt = rotate(k, pos.cpu(), f, False)
    assert sv.append_kv(k, v, *cb.args(), inv_freq=f, q=q, q_out=q, positions=pos) is q
    within(q, want, tol)
    within(cb.sequence(cb.k, 0)[7:], kw, kt)


def test_append_reports_bad_pages_and_lengths_and_leaves_the_rest():
    cb = CacheBatch([(2, 40), (3, 3), (2, 1), (1, 16)], 1, 16, 16, BF, fill=False)
    cb.pages[0, 2] = cb.k.shape[0]          # sequence 0 appends to slots 38, 39
    k, v = cb.tokens(1), cb.tokens(1)
    ws = sv.CacheWorkspace()
    sv.append_kv(k, v, *cb.args(), ws=ws)
    assert ws.status() == sv.STATUS_BAD_PAGE | sv.STATUS_BAD_LENGTH    # 1 slot for 2 new tokens
    assert ws.status() == 0
    written = (~torch.isnan(cb.k.float())).any(-1).any(-1)
    assert int(written.sum()) == 3 + 1 + 1  # sequence 1, the second token of 2, sequence 3
    cb2 = CacheBatch([(2, 40), (3, 3)], 1, 16, 16, BF, fill=False)
    cb2.kv_len[0] = 16 * cb2.wide + 1       # past the page table
    sv.append_kv(cb2.tokens(1), cb2.tokens(1), *cb2.args(), ws=ws)
    assert ws.status() == sv.STATUS_BAD_LENGTH
    assert int((~torch.isnan(cb2.k.float())).any(-1).any(-1).sum()) == 3


# ---------------------------------------------------------------------------
# attention

ATTEND = [
    # sequences (new, length), q heads, kv heads, d, page, type, window, heads first
    ([(1, 1)], 1, 1, 64, 16, BF, 0, False),
    ([(1, 2), (1, 127), (1, 128), (1, 129)], 4, 2, 128, 64, BF, 0, True),
    ([(6, 300), (6, 6), (6, 255), (6, 257)], 8, 2, 128, 64, HF, 0, True),
    ([(1, 1000)], 32, 8, 128, 64, BF, 0, True),
    ([(0, 50), (3, 3), (0, 0), (7, 400)], 6, 2, 96, 48, BF, 0, False),
    ([(33, 33), (31, 200)], 8, 2, 64, 16, HF, 0, False),
    ([(65, 130), (2, 513)], 8, 2, 128, 32, BF, 0, True),
    ([(70, 70)], 8, 1, 80, 16, HF, 0, False),
    ([(130, 300)], 3, 3, 64, 128, BF, 0, True),
    ([(200, 641)], 4, 1, 128, 256, HF, 0, False),
    ([(6, 300), (1, 5), (40, 290)], 4, 2, 64, 16, BF, 1, True),
    ([(6, 300), (40, 290)], 4, 2, 128, 32, HF, 33, False),
    ([(150, 420)], 4, 2, 128, 64, BF, 130, True),
    ([(3, 3), (2, 9)], 2, 1, 8, 8, HF, 0, False),
    ([(5, 3), (4, 0), (2, 1)], 4, 2, 64, 16, BF, 0, True),     # rows before the first slot
    ([(2, 2200)], 2, 1, 128, 16, HF, 0, True),
]


@pytest.mark.parametrize("case", ATTEND)
def test_attention_matches_the_definition(case):
    seqs, hq, hkv, d, page, dt, window, first = case
    cb = CacheBatch(seqs, hkv, d, page, dt, heads_first=first, seed=11)
    q = cb.tokens(hq, 1.5)
    ws = sv.CacheWorkspace()
    want, tol = attention(cb, q, default_scale(d), window)
    for _ in range(2):                      # a second call finds the workspace as the first did
        got = sv.paged_attention(q, *cb.args(), window=window, ws=ws)
        assert ws.status() == 0
        within(got, want, tol)


def test_attention_over_many_sequences():
    """More sequences than one pass of the scheduler's search covers, empty ones
    among them."""
    seqs = [((b * 7) % 4, (b * 7) % 4 + (b * 13) % 37) for b in range(1000)]
    cb = CacheBatch(seqs, 1, 64, 16, BF, seed=14)
    q = cb.tokens(2)
    ws = sv.CacheWorkspace()
    want, tol = attention(cb, q, default_scale(64), 0)
    got = sv.paged_attention(q, *cb.args(), ws=ws)
    assert ws.status() == 0
    within(got, want, tol)


@pytest.mark.parametrize("group,d,page", [(3, 64, 8), (7, 96, 24), (5, 128, 16), (16, 64, 64), (130, 32, 8)])
def test_attention_group_sizes_and_scales(group, d, page):
    cb = CacheBatch([(5, 140), (1, 33), (45, 45)], 1, d, page, BF, seed=group)
    q = cb.tokens(group)
    for scale in (0.2, -0.1, 0.0):
        want, tol = attention(cb, q, scale, 0)
        within(sv.paged_attention(q, *cb.args(), scale=scale), want, tol)


def test_attention_same_bits_again_and_on_another_stream():
    cb = CacheBatch([(6, 900), (1, 77), (50, 300)], 2, 128, 64, BF, seed=5)
    q = cb.tokens(8)
    a = sv.paged_attention(q, *cb.args())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b = sv.paged_attention(q, *cb.args(), stream=s)
    s.synchronize()
    assert torch.equal(a, b)


def test_outputs_on_another_stream_come_from_its_own_memory():
    """A block that the current stream has freed but not finished with is not
    handed out as the output of a call on another stream."""
    cb = CacheBatch([(40, 300), (1, 77)], 2, 128, 64, BF, seed=5)
    q, k, v = cb.tokens(8), cb.tokens(2), cb.tokens(2)
    z, u = torch.randn(41, 1024, device="cuda"), torch.rand(41, dtype=torch.float64, device="cuda")
    big = torch.zeros(1 << 27, device="cuda")
    calls = [lambda **kw: sv.append_kv(k, v, *cb.args(), inv_freq=freqs(128), q=q, **kw),
             lambda **kw: sv.paged_attention(q, *cb.args(), **kw),
             lambda **kw: sv.warp_sample(z, u, probs=True, **kw)[1]]
    want = [f() for f in calls]
    s = torch.cuda.Stream()
    for f in calls:
        f(stream=s)                         # workspace of this stream
    torch.cuda.synchronize()
    for f, w in zip(calls, want):
        late = torch.empty_like(w)
        for _ in range(20):
            big.add_(1)                     # some milliseconds
        late.fill_(9)
        del late
        got = f(stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, w)


def test_attention_large_scores_and_scale():
    """Scores in the thousands: one key takes all the weight, nothing overflows."""
    cb = CacheBatch([(6, 400), (130, 260)], 1, 64, 16, HF, seed=6, spread=12.0)
    q = cb.tokens(2, 12.0)
    for scale in (1.0, -0.5, 0.0):
        want, tol = attention(cb, q, scale, 0)
        within(sv.paged_attention(q, *cb.args(), scale=scale), want, tol)


def test_attention_strided_queries_and_out():
    cb = CacheBatch([(6, 50), (3, 140)], 2, 64, 16, BF, seed=7)
    wide = torch.randn(9, 6, 128, generator=cb.gen).to(BF).cuda()
    q = wide[:, 1:5, 64:]
    out = torch.full((9, 8, 72), 5.0, dtype=BF, device="cuda")
    got = sv.paged_attention(q, *cb.args(), out=out[:, 2:6, 8:])
    want, tol = attention(cb, q, default_scale(64), 0)
    within(got, want, tol)
    assert bool((out[:, :2] == 5).all()) and bool((out[:, 6:] == 5).all())
    assert bool((out[..., :8] == 5).all())


def test_attention_pages_over_two_gigabytes_apart():
    """Offsets into the cache pass 32 bits."""
    page, d = 64, 128
    pool = (1 << 31) // (page * d) + 64                # over 2^31 elements in one cache
    k = torch.zeros(pool, page, 1, d, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    far = CacheBatch([(2, 100)], 1, d, page, BF, seed=8)
    ids = [pool - 1, 3]
    for i, p in enumerate(ids):
        src = int(far.table[0, i])
        k[p], v[p] = far.k[src], far.v[src]
    pages = torch.tensor([ids], dtype=torch.int32, device="cuda")
    q = far.tokens(4)
    want, tol = attention(far, q, default_scale(d), 0)
    within(sv.paged_attention(q, k, v, pages, far.q_start, far.kv_len), want, tol)
    kn, vn = far.tokens(1), far.tokens(1)
    far.kv_len[0] = 2                                  # tokens 0 and 1: the far page
    sv.append_kv(kn, vn, k, v, pages, far.q_start, far.kv_len)
    assert torch.equal(k[pool - 1, :2], kn) and torch.equal(v[pool - 1, :2], vn)


def test_attention_reports_bad_pages_and_lengths():
    cb = CacheBatch([(2, 200), (3, 90), (1, 10)], 1, 64, 16, BF, seed=9)
    q = cb.tokens(2)
    want, tol = attention(cb, q, default_scale(64), 0)
    cb.pages[0, 3] = -1
    out = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    ws = sv.CacheWorkspace()
    sv.paged_attention(q, *cb.args(), out=out, ws=ws)
    assert ws.status() == sv.STATUS_BAD_PAGE
    within(out[2:], want[2:], tol[2:])
    assert bool(torch.isfinite(out).all())
    cb.pages[0, 3] = int(cb.table[0, 3])
    cb.kv_len[1] = 16 * cb.wide + 1
    out.fill_(7.0)
    sv.paged_attention(q, *cb.args(), out=out, ws=ws)
    assert ws.status() == sv.STATUS_BAD_LENGTH
    assert bool((out[2:5] == 7).all())
    within(out[:2], want[:2], tol[:2])
    within(out[5:], want[5:], tol[5:])


def test_rows_of_no_sequence_are_left_alone():
    cb = CacheBatch([(2, 20), (3, 90)], 1, 64, 16, BF, seed=9, extra_tokens=4)
    q = cb.tokens(2)
    out = torch.full(q.shape, 7.0, dtype=BF, device="cuda")
    sv.paged_attention(q, *cb.args(), out=out)
    assert bool((out[5:] == 7).all())
    want, tol = attention(cb, q, default_scale(64), 0)
    within(out[:5], want[:5], tol[:5])


def test_append_then_attend_in_a_graph():
    """Both calls captured once and replayed on new contents."""
    cb = CacheBatch([(3, 70), (2, 33)], 2, 64, 16, BF, seed=10)
    q, k, v = cb.tokens(4), cb.tokens(2), cb.tokens(2)
    f = freqs(64)
    ws = sv.CacheWorkspace()
    out = torch.empty_like(q)
    qr = torch.empty_like(q)

    def step(stream=None):
        sv.append_kv(k, v, *cb.args(), inv_freq=f, q=q, q_out=qr, ws=ws)
        sv.paged_attention(qr, *cb.args(), out=out, ws=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in (1, 2):
        gen = torch.Generator().manual_seed(seed)
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen).to(BF))
        g.replay()
        torch.cuda.synchronize()
        want, tol = attention(cb, qr, default_scale(64), 0)
        within(out, want, tol)
    assert ws.status() == 0


def test_bindings_refuse_what_does_not_fit():
    cb = CacheBatch([(2, 20)], 1, 64, 16, BF)
    q, k, v = cb.tokens(2), cb.tokens(1), cb.tokens(1)
    E = sv.SpecVerifyError
    a = list(cb.args())
    with pytest.raises(E):
        sv.paged_attention(q.float(), *a)
    with pytest.raises(E):
        sv.paged_attention(q[..., :32], *a)
    with pytest.raises(E):
        sv.paged_attention(q.transpose(1, 2), *a)
    with pytest.raises(E):
        sv.paged_attention(q, *a, scale=math.inf)
    with pytest.raises(E):
        sv.paged_attention(q, *a, window=-1)
    with pytest.raises(E):
        sv.paged_attention(q, a[0], a[1].half(), *a[2:])
    with pytest.raises(E):
        sv.paged_attention(q, *a[:2], a[2].long(), *a[3:])
    with pytest.raises(E):
        sv.paged_attention(q, *a[:3], a[3][:1], a[4])
    with pytest.raises(E):
        sv.paged_attention(q, *a[:4], a[4].cpu())
    with pytest.raises(E):
        sv.paged_attention(q, *a[:2], a[2].cpu(), *a[3:])
    with pytest.raises(E):
        sv.append_kv(k, v[:1], *a)
    with pytest.raises(E):
        sv.append_kv(k, v, *a, inv_freq=freqs(64).float())
    with pytest.raises(E):
        sv.append_kv(k, v, *a, inv_freq=freqs(132))
    with pytest.raises(E):
        sv.append_kv(k, v, *a, inv_freq=freqs(6))
    with pytest.raises(E):
        sv.append_kv(k, v, *a, q_out=q)
    off = torch.empty(2 * 64 + 1, dtype=BF, device="cuda")[1:].view(2, 1, 64)
    with pytest.raises(E):
        sv.append_kv(off, v, *a)                       # not 16-byte aligned
    torch.cuda.synchronize()
