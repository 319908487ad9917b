"""append_kv and paged_attention where the usual batches do not go."""
import contextlib
import ctypes

import pytest
import torch

import speculative_decoding_verification_08_gb300 as sv
from speculative_decoding_verification_08_gb300 import _build, paged as sv_paged
from cache_refs import CacheBatch, attention, default_scale

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


def test_a_captured_call_needs_a_workspace_of_its_own():
    """A graph keeps the workspace's address and may be replayed anywhere, and a
    workspace made during a capture would be zeroed by that graph alone: calls
    without one are refused while the stream is captured."""
    cb = CacheBatch([(3, 700), (2, 33)], 2, 64, 16, BF, seed=20)
    q, k, v = cb.tokens(4), cb.tokens(2), cb.tokens(2)
    z, u = torch.randn(3, 500, device="cuda"), torch.rand(3, dtype=torch.float64, device="cuda")
    calls = [lambda **kw: sv.append_kv(k, v, *cb.args(), q=q, **kw),
             lambda **kw: sv.paged_attention(q, *cb.args(), **kw),
             lambda **kw: sv.warp_sample(z, u, **kw)]
    used = torch.cuda.Stream()                        # a stream that has an implicit workspace already
    for f in calls:
        f(stream=used)
    torch.cuda.synchronize()
    for where in ({}, {"stream": used}):
        for f in calls:
            with pytest.raises(sv.SpecVerifyError, match="ws="):
                with torch.cuda.graph(torch.cuda.CUDAGraph(), **where):
                    f()
    for f in (sv.CacheWorkspace, sv.cache_workspace, lambda: sv.CacheWorkspace(stream=used)):
        with pytest.raises(sv.SpecVerifyError, match="capture"):
            with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=used):
                f()
    torch.cuda.synchronize()
    want = sv.paged_attention(q, *cb.args())
    # two graphs, each with its workspace, in either order
    graphs = []
    for _ in range(2):
        ws, out, g = sv.CacheWorkspace(), torch.empty_like(q), torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sv.paged_attention(q, *cb.args(), out=out, ws=ws)
        graphs.append((g, out, ws))
    for g, out, ws in reversed(graphs):
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert ws.status() == 0 and torch.equal(out, want)


def test_a_captured_pass_over_a_paged_cache():
    c = sv_paged.PagedCache(1, 8, 16, 2, 64)
    g = torch.Generator().manual_seed(25)
    q, k, v = (torch.randn(5, h, 64, generator=g).to(BF).cuda() for h in (4, 2, 2))
    c.begin({0: 5})
    want = c.attend(0, c.append(0, q, k, v))
    c.k.zero_()
    graph, ws = torch.cuda.CUDAGraph(), sv.CacheWorkspace()
    with torch.cuda.graph(graph):
        got = c.attend(0, c.append(0, q, k, v, ws=ws), ws=ws)
    graph.replay()
    assert ws.status() == 0 and torch.equal(got, want)


def test_the_implicit_workspace_by_any_name_of_the_device():
    want = sv.cache_workspace()
    assert sv.cache_workspace("cuda") is want
    assert sv.cache_workspace("cuda:0") is want
    assert sv.cache_workspace(torch.device("cuda")) is want
    s = torch.cuda.Stream()
    assert sv.cache_workspace("cuda", stream=s) is sv.cache_workspace(stream=s)
    assert sv.cache_workspace(stream=s) is not want


def test_counts_left_in_a_workspace_are_reported_and_cleared():
    """The tiles' counters (two per CTA from byte 256 on) hold what no call
    leaves there: the call says so, and the next one is right."""
    cb = CacheBatch([(6, 3000), (2, 700)], 2, 64, 16, BF, seed=24)
    q = cb.tokens(4)
    want, tol = attention(cb, q, default_scale(64), 0)
    ws = sv.CacheWorkspace()
    counters = ws.buf[256:256 + 4 * 2 * 160].view(torch.int32)
    for clear in (ws.status, lambda: (ws.reset(), ws.status())[1]):
        counters.fill_(1 << 20)
        sv.paged_attention(q, *cb.args(), ws=ws)
        assert clear() == (sv.STATUS_OVERFLOW if clear == ws.status else 0)
        assert not bool(counters.any())
        got = sv.paged_attention(q, *cb.args(), ws=ws)
        assert ws.status() == 0
        within(got, want, tol)
        assert not bool(counters.any())


@pytest.fixture(scope="module")
def stalled(tmp_path_factory):
    """The entry points of a build whose attention leaves waits unanswered
    (SV_STALL=1); the extension calls them inside `with`."""
    out = str(tmp_path_factory.mktemp("specverify_stall") / "libspecverify_stall.so")
    other = sv._declare(ctypes.CDLL(_build.build_variant(out, ["-DSV_STALL=1"])))

    @contextlib.contextmanager
    def bound():
        def bind(lib):
            sv._native().bind(*(ctypes.cast(f, ctypes.c_void_p).value
                                for f in (lib.sv_append_kv, lib.sv_paged_attention, lib.sv_warp_sample)),
                              sv.SpecVerifyError, sv._check)
        bind(other)
        try:
            yield
        finally:
            bind(sv.load())
    return bound


@pytest.mark.parametrize("group", [2, 3])             # queries by tensor copies, and by the threads
def test_a_wait_that_runs_out_is_reported_and_the_workspace_serves_again(stalled, group):
    cb = CacheBatch([(6, 880 + b) for b in range(60)] + [(150, 400)] * 8, 2, 64, 16, BF, seed=26)
    q = cb.tokens(2 * group)
    ws = sv.CacheWorkspace()
    want = sv.paged_attention(q, *cb.args(), ws=ws)
    assert ws.status() == 0
    for _ in range(2):
        with stalled():
            sv.paged_attention(q, *cb.args(), ws=ws)
        assert ws.status() == sv.STATUS_TIMEOUT
        got = sv.paged_attention(q, *cb.args(), ws=ws)
        assert ws.status() == 0 and torch.equal(got, want)


@pytest.mark.parametrize("seqs", [[(2, 3000), (40, 300)],          # few tiles, cut between CTAs
                                  [(2, 40 + b % 7) for b in range(400)] + [(130, 200)]])
@pytest.mark.parametrize("group", [2, 3])
def test_a_nan_query_gives_nan_whatever_the_cut(seqs, group):
    cb = CacheBatch(seqs, 2, 64, 16, BF, seed=21)
    q = cb.tokens(2 * group)
    want, tol = attention(cb, q, default_scale(64), 0)
    rows = [(0, 1), (3, 0), (cb.N - 1, 2)]            # (token, head)
    for t, h in rows:
        q[t, h, 5] = float("nan")
    ws = sv.CacheWorkspace()
    got = sv.paged_attention(q, *cb.args(), ws=ws)
    assert ws.status() == 0
    for t, h in rows:
        assert bool(torch.isnan(got[t, h]).all()), (t, h)
        got[t, h], want[t, h] = 0.0, 0.0
    within(got, want, tol)


@pytest.mark.parametrize("bits", [25.25, 23.5, 18.0])
@pytest.mark.parametrize("new", [1, 130])             # rows that split the keys, rows that share them
def test_many_small_weights_beside_a_large_one(bits, new):
    """One key outweighs each of 20,000 others by `bits` octaves: together they
    still count, fp16's range of 24 octaves below one notwithstanding.  Weights
    are held in steps of 2^-31 of one that the row's largest reaches: each is off
    by half a step at most, beside its relative rounding.  400 sequences share
    the pages, so that a CTA sees a tile's keys from the first to the last."""
    L, d, page, B = 20000, 64, 80, 400
    cb = CacheBatch([(new, L)], 1, d, page, HF, fill=False, seed=22)
    cb.k.zero_()
    cb.v.fill_(1.0)
    at = int(cb.table[0, 0])
    cb.k[at, 0, 0, 0] = bits * 0.6931471805599453
    cb.v[at, 0] = 0.0
    q = torch.zeros(B * new, 1, d, dtype=HF, device="cuda")
    q[..., 0] = 1.0
    gap = float(cb.k[at, 0, 0, 0])
    n = (L - new + torch.arange(new, dtype=torch.float64)).repeat(B).view(-1, 1, 1)   # equal slots a row sees
    small = n * torch.exp(torch.tensor(-gap, dtype=torch.float64))
    want = (small / (1 + small)).expand(B * new, 1, d)
    tol = want * (2 * 2.0 ** -11 + 2 * (d + 4) * 2.0 ** -24 * gap + 2.0 ** -21 + (L / 8 + 64) * 2.0 ** -23)
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda") * new
    ws = sv.CacheWorkspace()
    got = sv.paged_attention(q, cb.k, cb.v, cb.pages.expand(B, -1).contiguous(), start, cb.kv_len.expand(B).contiguous(),
                             scale=1.0, ws=ws)
    assert ws.status() == 0
    within(got, want, tol + L * 2.0 ** -32)


def test_the_stride_of_an_axis_of_length_one_means_nothing():
    """One token, one head, one page of one sequence: whatever stride such an
    axis carries, it is never multiplied by anything but zero."""
    cb = CacheBatch([(1, 9)], 1, 64, 16, BF, seed=23)
    q, k, v = cb.tokens(1), cb.tokens(1), cb.tokens(1)
    f = torch.pow(10000.0, -2.0 * torch.arange(32, dtype=torch.float64, device="cuda") / 64)
    page = int(cb.table[0, 0])
    kc, vc = cb.k[page:page + 1].clone(), cb.v[page:page + 1].clone()
    zero = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    odd = lambda x: x.as_strided(x.shape, [7 if n == 1 else s for n, s in zip(x.shape, x.stride())])  # noqa: E731
    want = []
    for g in (lambda x: x, odd):
        ck, cv = kc.clone(), vc.clone()
        r = sv.append_kv(g(k), g(v), g(ck), g(cv), zero, cb.q_start, cb.kv_len, inv_freq=f, q=g(q),
                         q_out=g(torch.empty_like(q)))
        o = sv.paged_attention(g(q), g(ck), g(cv), zero, cb.q_start, cb.kv_len, out=g(torch.empty_like(q)))
        want.append((ck, cv, r, o))
    for a, b in zip(*want):
        assert torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def test_pieces_that_take_longer_than_a_wait_may():
    """48 million slots (one page of zero values, listed over and over, and one of
    others at the end) before four rows of 128 heads: a tile keeps a CTA busy for
    more than the 250 ms after which a wait without progress gives up, and its next
    tile's queries wait for that long.  Scores are 0, so that every sum is exact."""
    page, L, d, G, B = 1 << 18, 48 << 20, 64, 128, 95
    k = torch.randn(2, page, 1, d, generator=torch.Generator().manual_seed(27)).to(BF).cuda()
    v = torch.zeros(2, page, 1, d, dtype=BF, device="cuda")
    row = torch.linspace(-3, 3, d).to(BF)
    v[1] = row.cuda()
    pages = torch.zeros(B, L // page, dtype=torch.int32, device="cuda")
    pages[:, -1] = 1
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda") * 4      # two tiles each
    q = torch.zeros(4 * B, G, d, dtype=BF, device="cuda")
    ws = sv.CacheWorkspace()
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    t[0].record()
    got = sv.paged_attention(q, k, v, pages, start, torch.full((B,), L, dtype=torch.int32, device="cuda"), ws=ws)
    t[1].record()
    assert ws.status() == 0
    assert t[0].elapsed_time(t[1]) > 250
    last = torch.arange(-3, 1, dtype=torch.float64).repeat(B).view(-1, 1, 1)
    want = (row.double() * (page + last) / (L + last)).expand(4 * B, G, d)
    within(got, want, want.abs() * (2.0 ** -8 + 2.0 ** -20))
