"""Attention over 8-bit caches: what one row, one slot or one batch holds does not
reach the others, whichever way a call is computed."""

import pytest
import torch

import speculative_decoding_verification_08_gb300 as sv
from cache_refs import attention, default_scale
from eight_refs import E4M3, EightBatch

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


def place(cb, b, s):
    return int(cb.table[b, s // cb.page]), s % cb.page


# few rows: over the codes; many: read back to 16 bits first
FEW = [(6, 300), (5, 2100)]
MANY = [(150, 400), (170, 300)]


# ---------------------------------------------------------------------------
# vectors that are NaN

@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("seqs", [FEW, MANY])
@pytest.mark.parametrize("scale,window", [(None, 0), (None, 50), (0.0, 0)])
def test_nan_vectors_reach_the_rows_that_see_them(dt, seqs, scale, window):
    """append_kv's code of a vector that is not finite: the scale NaN, codes of zero."""
    cb = EightBatch(seqs, 2, 64, 16, dt, seed=61)
    q = cb.tokens(4)
    ws = sv.CacheWorkspace()

    def call():
        return sv.paged_attention(q, *cb.eight(), scale=scale, window=window, **cb.scales(), ws=ws)
    clean = call()
    assert sv.last_kernel_count() == (2 if seqs is MANY else 1)
    want = torch.zeros(cb.N, 4, dtype=torch.bool)
    # sequence 0, kv head 0: the key of its new token 3; sequence 1, kv head 1: the value of token 4
    for b, j, h, c, s in ((0, 3, 0, cb.k8, cb.ks), (1, 4, 1, cb.v8, cb.vs)):
        n, t = seqs[b]
        p, at = place(cb, b, t - n + j)
        s.view(torch.uint8)[p, at, h] = 255
        c.view(torch.uint8)[p, at, h] = 0
        last = min(n, j + window) if window else n
        want[cb.starts[b] + j:cb.starts[b] + last, 2 * h:2 * h + 2] = True
    got = call()
    assert ws.status() == 0
    assert torch.equal(torch.isnan(got).all(-1).cpu(), want)
    assert torch.equal(got[~want.cuda()], clean[~want.cuda()])


# ---------------------------------------------------------------------------
# the room that sequences are read back to

def test_a_wide_and_mostly_empty_table_takes_little_memory():
    """No more than the cache itself in 16 bits, whatever the table's width; pages
    that sequences share, and one that is none, are read as they are."""
    cb = EightBatch([(150, 400), (170, 300), (140, 140)], 2, 64, 16, BF, seed=63)
    cb.table[2, :4] = cb.table[0, :4]                  # a common beginning of 64 slots
    wide = torch.full((3, 20000), 0, dtype=torch.int32)
    wide[:, :cb.wide] = cb.table
    cb.pages = wide.cuda()
    q = cb.tokens(4)
    sv.paged_attention(q, *cb.eight(), **cb.scales())
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    ws = sv.CacheWorkspace()
    got = sv.paged_attention(q, *cb.eight(), **cb.scales(), ws=ws)
    assert ws.status() == 0 and sv.last_kernel_count() == 2
    taken = torch.cuda.max_memory_allocated() - before - ws.nbytes
    assert taken <= 2 * 2 * cb.k8.numel() + got.numel() * 2 + (1 << 16)
    within(got, *attention(cb, q, default_scale(64), 0))
    cb.pages[1, 2] = cb.k8.shape[0]
    cb.k, cb.v = (torch.cat((x, torch.zeros_like(x[:1]))) for x in (cb.k, cb.v))
    cb.table[1, 2] = cb.k.shape[0] - 1                 # zeros
    got = sv.paged_attention(q, *cb.eight(), **cb.scales(), ws=ws)
    assert ws.status() == sv.STATUS_BAD_PAGE
    within(got, *attention(cb, q, default_scale(64), 0))


def test_without_memory_to_read_back_to_the_codes_are_attended_to():
    page, hkv, d, pool = 64, 8, 128, 2000              # 131 MB of codes, 524 to read back to
    cb = EightBatch([(140, 300), (130, 200)], hkv, d, page, BF, seed=64)
    for name in ("k8", "v8", "ks", "vs"):
        x = getattr(cb, name)
        y = torch.zeros(pool, *x.shape[1:], dtype=torch.uint8, device="cuda")
        y[:x.shape[0]] = x.view(torch.uint8)
        setattr(cb, name, y.view(x.dtype))
    wide = torch.zeros(2, 1200, dtype=torch.int32)
    wide[:, :cb.wide] = cb.table
    cb.pages = wide.cuda()
    q = cb.tokens(8)
    ws = sv.CacheWorkspace()
    want, tol = attention(cb, q, default_scale(d), 0)
    within(sv.paged_attention(q, *cb.eight(), **cb.scales(), ws=ws), want, tol)
    assert sv.last_kernel_count() == 2
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (100 << 20)) / total)
    try:
        got = sv.paged_attention(q, *cb.eight(), **cb.scales(), ws=ws)
        assert sv.last_kernel_count() == 1 and ws.status() == 0
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    within(got, want, tol)


# ---------------------------------------------------------------------------
# rows of a tile

@pytest.mark.parametrize("seqs", [[(3, 200), (2, 1500)], [(6, 40)]])
@pytest.mark.parametrize("dt,small,spread,big", [(BF, 1.0, 1.0, 2.0 ** 24), (BF, 1.0, 1.0, 2.0 ** 90),
                                                 (BF, 2.0 ** -60, 1.0, 2.0 ** 30), (HF, 2.0 ** -8, 256.0, 2.0 ** 21)])
def test_a_large_query_leaves_other_rows_alone(seqs, dt, small, spread, big):
    """Rows of one tile whose queries differ by 2^21 and more: each is as exact as by
    itself, and the others' bits do not change."""
    cb = EightBatch(seqs, 1, 64, 16, dt, seed=65, spread=spread)
    q = cb.tokens(4, small)
    scale = default_scale(64) if small > 1e-3 else 2.0 ** 60 * default_scale(64)
    call = lambda x: sv.paged_attention(x, *cb.eight(), scale=scale, **cb.scales())  # noqa: E731
    clean = call(q)
    within(clean, *attention(cb, q, scale, 0))
    far = q.clone()
    far[1, 2] *= big
    far[cb.N - 1, 0] *= big
    assert bool(torch.isfinite(far).all())
    got = call(far)
    within(got, *attention(cb, far, scale, 0))
    rest = torch.ones(cb.N, 4, dtype=torch.bool, device="cuda")
    rest[1, 2] = rest[cb.N - 1, 0] = False
    assert torch.equal(got[rest], clean[rest])


def test_the_largest_query_leaves_other_rows_alone():
    cb = EightBatch([(4, 700)], 1, 128, 16, BF, seed=66)
    q = cb.tokens(6)
    clean = sv.paged_attention(q, *cb.eight(), **cb.scales())
    q[2, 3] = torch.finfo(BF).max
    got = sv.paged_attention(q, *cb.eight(), **cb.scales())
    rest = torch.ones(4, 6, dtype=torch.bool, device="cuda")
    rest[2, 3] = False
    assert torch.equal(got[rest], clean[rest])


@pytest.mark.parametrize("power", [-110, -30, 60, 110])
def test_far_scales_of_the_call(power):
    """Queries and scale that are each out of the way, their product as usual."""
    cb = EightBatch([(3, 200)], 1, 64, 16, BF, seed=71)
    q = cb.tokens(4)
    want = sv.paged_attention(q, *cb.eight(), scale=0.125, **cb.scales())
    got = sv.paged_attention(q * 2.0 ** -power, *cb.eight(), scale=0.125 * 2.0 ** power, **cb.scales())
    assert torch.equal(got, want)


# ---------------------------------------------------------------------------
# slots whose values are far larger than others'

@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("seqs", [[(6, 300)], [(6, 3000), (2, 70)]])
@pytest.mark.parametrize("up", [20, 60])
def test_values_that_a_row_does_not_see_leave_it_alone(dt, seqs, up):
    """A new token's value 2^up times as large as the others': rows before it keep
    their bits, and with a window those behind it."""
    cb = EightBatch(seqs, 1, 64, 16, dt, seed=67, scale_spread=0.3)
    q = cb.tokens(4)
    n, t = seqs[0]
    before = [sv.paged_attention(q, *cb.eight(), window=w, **cb.scales()) for w in (0, 2)]
    p, at = place(cb, 0, t - n + 2)
    cb.vs.view(torch.uint8)[p, at] += up
    cb.refresh()
    for w, old in zip((0, 2), before):
        got = sv.paged_attention(q, *cb.eight(), window=w, **cb.scales())
        assert torch.equal(got[:2], old[:2]) and torch.equal(got[6:], old[6:])
        if w:
            assert torch.equal(got[4:], old[4:])
        if dt == BF or up == 20:                       # (fp16 results end at 65504)
            want, tol = attention(cb, q, default_scale(64), w)
            fits = want.abs() + tol < torch.finfo(dt).max
            off = (got.cpu().double() - want).abs()
            assert bool((off[fits] <= tol[fits]).all())


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("down", [0, -40, 30])
def test_large_values_with_no_weight(dt, down):
    """Values 2^30 times as large as the others', in slots that a row gives no weight
    (keys opposite to its query), and all of them small or large."""
    cb = EightBatch([(1, 700), (2, 3000)], 1, 64, 16, dt, seed=68, scale_spread=0.0)
    q = cb.tokens(2)
    q[...] = 0
    q[..., 0] = 8.0
    down = max(down, -14) if dt == HF else down        # (results above fp16's smallest)
    down = min(down, 0) if dt == HF else down
    cb.vs.view(torch.uint8)[...] += down % 256
    for b, (_, t) in enumerate(cb.seqs):
        for s in range(0, t, 7):
            p, at = place(cb, b, s)
            cb.k8[p, at, 0] = torch.zeros(64, device="cuda").to(E4M3)
            cb.k8.view(torch.uint8)[p, at, 0, 0] = 0xfe     # -448
            cb.ks.view(torch.uint8)[p, at, 0] = 127 - 2
            cb.vs.view(torch.uint8)[p, at, 0] = (127 - 6 + 30 + down)
    cb.refresh()
    got = sv.paged_attention(q, *cb.eight(), **cb.scales())
    within(got, *attention(cb, q, default_scale(64), 0))


@pytest.mark.parametrize("score", [2.0 ** 20, 2.0 ** 27, 2.0 ** 30, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("values", [-40, -9, 0, 30])
def test_huge_scores(score, values):
    """Scores whose steps in fp32 would swallow the values' scales: one slot has all
    the weight, the last of a pair of opposite ones, and gives its value."""
    cb = EightBatch([(2, 700)], 1, 64, 16, BF, seed=72, scale_spread=0.0)
    q = cb.tokens(4)
    q[...] = 0
    q[..., 0] = score
    cb.vs.view(torch.uint8)[...] += values % 256
    for s in range(0, 698, 99):                        # larger and larger keys, both ways
        for i in (0, 1):
            p, at = place(cb, 0, s + i)
            cb.k8[p, at, 0] = torch.zeros(64, device="cuda").to(E4M3)
            cb.k8.view(torch.uint8)[p, at, 0, 0] = 0x7e if i else 0xfe       # 448, -448
            cb.ks.view(torch.uint8)[p, at, 0] = 127 + s // 99 - 4
    cb.refresh()
    got = sv.paged_attention(q, *cb.eight(), **cb.scales())
    p, at = place(cb, 0, 694)
    want = cb.v[p, at, 0].expand(2, 4, 64)
    within(got, want, want.abs() * 2.0 ** -7)


# ---------------------------------------------------------------------------
# pages that are none

@pytest.mark.parametrize("seqs", [FEW, MANY])
@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("bad", [-1, 1 << 30])
def test_a_page_that_is_none_reads_as_zeros(seqs, window, bad):
    cb = EightBatch(seqs, 2, 64, 16, BF, seed=69)
    q = cb.tokens(4)
    ws = sv.CacheWorkspace()
    # page 3 (of a window none or all see: the one before the first new token)
    at = [3, (seqs[1][1] - seqs[1][0] - 1) // 16]
    cb.k, cb.v = (torch.cat((x, torch.zeros_like(x[:1]))) for x in (cb.k, cb.v))
    for b in (0, 1):
        cb.pages[b, at[b]] = bad
        cb.table[b, at[b]] = cb.k.shape[0] - 1
    got = sv.paged_attention(q, *cb.eight(), window=window, **cb.scales(), ws=ws)
    assert ws.status() == sv.STATUS_BAD_PAGE
    within(got, *attention(cb, q, default_scale(64), window))


# ---------------------------------------------------------------------------
# batches at the border between the two ways

@pytest.mark.parametrize("seqs,kernels", [
    ([(120, 400), (8, 900)], 1), ([(121, 400), (8, 900)], 2), ([(127, 130), (1, 1300)], 1),
    ([(300, 300)] + [(1, 100 + 90 * i) for i in range(20)], 1), ([(500, 700), (6, 1000), (1, 40)], 2)])
@pytest.mark.parametrize("window", [0, 100])
def test_long_and_short_sequences_together(seqs, kernels, window):
    cb = EightBatch(seqs, 2, 64, 16, BF, seed=70, scale_spread=0.5)
    q = cb.tokens(4, 1.5)
    ws = sv.CacheWorkspace()
    got = sv.paged_attention(q, *cb.eight(), window=window, **cb.scales(), ws=ws)
    assert ws.status() == 0 and sv.last_kernel_count() == kernels
    within(got, *attention(cb, q, default_scale(64), window))
