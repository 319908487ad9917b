"""8-bit caches and head norms where the usual batches do not go."""
import ctypes
import importlib.util
import math
import os

import pytest
import torch

import speculative_decoding_verification_08_gb300 as sv
from speculative_decoding_verification_08_gb300 import _build
from speculative_decoding_verification_08_gb300.paged import PagedCache, rope_frequencies
from cache_refs import CacheBatch, attention, default_scale
from eight_refs import E4M3, E8M0, EightBatch, turned

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


# ---------------------------------------------------------------------------
# many rows: the sequences are read back first

MANY = [
    ([(300, 700), (5, 900)], 4, 2, 64, 24, HF, 50),
    ([(200, 200), (0, 40), (129, 1000)], 8, 2, 128, 64, BF, 0),
    ([(150, 151)], 6, 6, 48, 8, BF, 0),
    ([(140, 1200), (140, 141)], 2, 1, 96, 16, BF, 3),
]


@pytest.mark.parametrize("case", MANY)
def test_many_rows(case):
    seqs, hq, hkv, d, page, dt, window = case
    cb = EightBatch(seqs, hkv, d, page, dt, seed=31, scale_spread=0.5)
    q = cb.tokens(hq, 1.5)
    ws = sv.CacheWorkspace()
    got = sv.paged_attention(q, *cb.eight(), window=window, **cb.scales(), ws=ws)
    assert ws.status() == 0 and sv.last_kernel_count() == (2 if sum(n for n, _ in seqs) * (hq // hkv) > 128 * len(seqs) else 1)
    within(got, *attention(cb, q, default_scale(d), window))
    cb.pages[0, 0] = -1                                # a page that is none reads as zeros
    sv.paged_attention(q, *cb.eight(), window=window, **cb.scales(), ws=ws)
    if not window:
        assert ws.status() == sv.STATUS_BAD_PAGE


# ---------------------------------------------------------------------------
# references that grow

@pytest.mark.parametrize("dt", [BF, HF])
def test_scores_and_scales_that_keep_growing(dt):
    """Every block's keys outweigh the ones before, and its values are larger: the
    rows' references and that of the scales move again and again."""
    L = 1300
    cb = EightBatch([(5, L), (3, L - 7)], 2, 64, 16, dt, seed=32, scale_spread=0.0)
    # scales are powers of two already: raise them along the sequence
    for b, (_, t) in enumerate(cb.seqs):
        for s in range(t):
            p, at = int(cb.table[b, s // 16]), s % 16
            up_k, up_v = s // 200, s // 50 - 20
            cb.ks.view(torch.uint8)[p, at] += up_k
            cb.vs.view(torch.uint8)[p, at] += up_v % 256
    cb.refresh()
    q = cb.tokens(6, 1.0)
    got = sv.paged_attention(q, *cb.eight(), **cb.scales())
    within(got, *attention(cb, q, default_scale(64), 0))


def test_small_values_beside_large_ones():
    """A row's own values count where another's are 2^18 times as large but out of
    its reach (keys opposite to its query)."""
    cb = EightBatch([(1, 400)], 1, 64, 16, HF, seed=33, scale_spread=0.0)
    q = cb.tokens(1)
    q[0, 0] = 0
    q[0, 0, 0] = 8.0
    code = torch.zeros(64).to(E4M3)
    for s in range(0, 400, 7):                         # far from the query, and large
        p, at = int(cb.table[0, s // 16]), s % 16
        cb.k8[p, at, 0] = code.cuda()
        cb.k8.view(torch.uint8)[p, at, 0, 0] = 0xfe    # -448
        cb.ks.view(torch.uint8)[p, at, 0] = 127 - 2
        cb.vs.view(torch.uint8)[p, at, 0] = 127 - 6 + 18
    cb.refresh()
    got = sv.paged_attention(q, *cb.eight(), **cb.scales())
    within(got, *attention(cb, q, default_scale(64), 0))


# ---------------------------------------------------------------------------
# what is not finite

def test_keys_and_values_that_are_nan_reach_the_rows_that_see_them():
    n, L = 6, 300
    cb = EightBatch([(n, L), (n, L)], 2, 64, 16, BF, seed=34)
    q = cb.tokens(8)
    clean = sv.paged_attention(q, *cb.eight(), **cb.scales())
    # sequence 0, head 0: the key of new token 3; sequence 1, head 1: the value of token 4
    for b, s, h, x in ((0, L - n + 3, 0, cb.ks), (1, L - n + 4, 1, cb.vs)):
        p, at = int(cb.table[b, s // 16]), s % 16
        x.view(torch.uint8)[p, at, h] = 255
        (cb.k8 if x is cb.ks else cb.v8).view(torch.uint8)[p, at, h] = 0
    got = sv.paged_attention(q, *cb.eight(), **cb.scales())
    want = torch.zeros(2 * n, 8, dtype=torch.bool)
    want[3:n, :4] = True
    want[n + 4:, 4:] = True
    assert torch.equal(torch.isnan(got).all(-1).cpu(), want)
    assert torch.equal(got[~want.cuda()], clean[~want.cuda()])


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("length", [40, 3000])          # one CTA's tile, and one cut between several
def test_a_query_that_is_not_finite_gives_nan_alone(bad, length):
    cb = EightBatch([(4, length)], 1, 64, 16, HF, seed=35)
    q = cb.tokens(2)
    clean = sv.paged_attention(q, *cb.eight(), **cb.scales())
    q[2, 1, 17] = bad
    got = sv.paged_attention(q, *cb.eight(), **cb.scales())
    assert bool(torch.isnan(got[2, 1]).all()) and int(torch.isnan(got).sum()) == 64
    rest = torch.ones(4, 2, dtype=torch.bool, device="cuda")
    rest[2, 1] = False
    assert torch.equal(got[rest], clean[rest])


def test_garbage_in_unused_slots_does_not_matter():
    """Codes and scales behind a sequence's end, in its last page and others."""
    cb = EightBatch([(2, 205), (2, 129)], 1, 128, 32, BF, seed=36)
    q = cb.tokens(4)
    want = sv.paged_attention(q, *cb.eight(), **cb.scales())
    held = torch.zeros(cb.k8.shape[:2], dtype=torch.bool)
    for b, (_, t) in enumerate(cb.seqs):
        for s in range(t):
            held[int(cb.table[b, s // 32]), s % 32] = True
    for byte in (0x00, 0x7e, 0xff):
        for x in (cb.k8, cb.v8, cb.ks, cb.vs):
            x.view(torch.uint8)[~held] = byte
        assert torch.equal(sv.paged_attention(q, *cb.eight(), **cb.scales()), want)


# ---------------------------------------------------------------------------
# layouts, places, repeats

def test_layouts_of_caches_and_scales():
    cb = EightBatch([(3, 90), (2, 33)], 3, 64, 16, BF, seed=37)
    q, k, v = cb.tokens(6), cb.tokens(3), cb.tokens(3)

    def relaid(x, order, pad):
        raw = x.view(torch.uint8)
        shape = [raw.shape[i] for i in order] + ([raw.shape[3]] if raw.dim() == 4 else [])
        wide = torch.full([s + pad for s in shape[:-1]] + [shape[-1] + 16 * pad], 0x55, dtype=torch.uint8, device="cuda")
        view = wide[tuple(slice(0, s) for s in shape)]
        back = [order.index(i) for i in range(3)] + ([3] if raw.dim() == 4 else [])
        view = view.permute(back)
        view.copy_(raw)
        return view.view(x.dtype)

    plain = [x.clone() for x in (cb.k8, cb.v8, cb.ks, cb.vs)]
    def passes(k8, v8, ks, vs):  # noqa: E306
        scales = dict(k_scale=ks, v_scale=vs)
        args = k8, v8, cb.pages, cb.q_start, cb.kv_len
        q1 = sv.append_kv(k, v, *args, q=q, q_norm=torch.ones(64, device="cuda"), **scales)
        return (q1, *sv.read_kv(*args, rows=cb.N, **scales), sv.paged_attention(q1, *args, **scales),
                *(x.view(torch.uint8).clone() for x in (k8, v8, ks, vs)))
    want = passes(*(x.clone() for x in plain))
    for order, pad in (((0, 1, 2), 1), ((0, 2, 1), 0), ((2, 0, 1), 1), ((1, 0, 2), 0), ((2, 1, 0), 1)):
        got = passes(*(relaid(x, order, pad) for x in plain))
        for x, y in zip(got, want):
            assert torch.equal(x, y), (order, pad)


def test_scales_that_vectors_share_can_be_read():
    """One scale for a head, as an expanded tensor: read and attended to, not written."""
    cb = EightBatch([(2, 100)], 2, 64, 16, BF, seed=38, scale_spread=0.0)
    one = torch.tensor([[[120, 119]]], dtype=torch.uint8, device="cuda")
    full = one.expand(cb.ks.shape).contiguous().view(E8M0)
    wide = one.expand(cb.ks.shape).view(E8M0)
    q = cb.tokens(4)
    a = sv.paged_attention(q, *cb.eight(), k_scale=full, v_scale=full)
    assert torch.equal(sv.paged_attention(q, *cb.eight(), k_scale=wide, v_scale=wide), a)
    for x, y in zip(sv.read_kv(*cb.eight(), rows=2, k_scale=wide, v_scale=wide),
                    sv.read_kv(*cb.eight(), rows=2, k_scale=full, v_scale=full)):
        assert torch.equal(x, y)
    with pytest.raises(sv.SpecVerifyError):
        sv.append_kv(cb.tokens(2), cb.tokens(2), *cb.eight(), k_scale=wide, v_scale=wide)


def test_offsets_past_32_bits():
    """Pages that begin 2^31 bytes and more into the cache."""
    page, hkv, d, pool = 64, 8, 128, 34000             # 65,536 bytes a page
    k8, v8 = (torch.zeros(pool, hkv, page, d, dtype=torch.uint8, device="cuda").view(E4M3).transpose(1, 2)
              for _ in range(2))
    ks, vs = (torch.zeros(pool, page, hkv, dtype=torch.uint8, device="cuda").view(E8M0) for _ in range(2))
    scales = dict(k_scale=ks, v_scale=vs)
    pages = torch.tensor([[pool - 1, 5, pool - 2]], dtype=torch.int32, device="cuda")
    n = 150
    batch = pages, torch.tensor([0, n], dtype=torch.int32, device="cuda"), torch.tensor([n], dtype=torch.int32,
                                                                                     device="cuda")
    g = torch.Generator().manual_seed(39)
    k, v = (torch.randn(n, hkv, d, generator=g).to(BF).cuda() for _ in range(2))
    sv.append_kv(k, v, k8, v8, *batch, **scales)
    kr, vr = sv.read_kv(k8, v8, *batch, rows=n, **scales)
    for got, want in ((kr, k), (vr, v)):
        top = want.abs().amax(-1, keepdim=True).float()
        assert bool(((got.float() - want.float()).abs() <= want.abs().float() * 2.0 ** -4 + top * 2.0 ** -17).all())
    q = torch.randn(2, 16, d, generator=g).to(BF).cuda()
    batch = pages, torch.tensor([0, 2], dtype=torch.int32, device="cuda"), batch[2]
    out = sv.paged_attention(q, k8, v8, *batch, **scales)
    for j in range(2):
        s = torch.einsum("hd,khd->hk", q[j].double(), kr[:n - 1 + j].double().repeat_interleave(2, 1)) / d ** 0.5
        p = s.softmax(-1)
        vv = vr[:n - 1 + j].double().repeat_interleave(2, 1)
        want = torch.einsum("hk,khd->hd", p, vv)
        room = torch.einsum("hk,khd->hd", p, vv.abs()) * 2.0 ** -7 + 1e-5
        assert bool(((out[j].double() - want).abs() <= room).all())


def test_the_same_bits_every_time():
    cb = EightBatch([(6, 900 + 37 * b) for b in range(30)], 2, 128, 32, BF, seed=40)
    q = cb.tokens(8)
    want = sv.paged_attention(q, *cb.eight(), **cb.scales())
    for _ in range(20):
        assert torch.equal(sv.paged_attention(q, *cb.eight(), **cb.scales()), want)


# ---------------------------------------------------------------------------
# streams, graphs, workspaces

def test_captured_calls_and_other_streams():
    for seqs in ([(3, 700), (2, 33)], [(200, 700), (180, 330)]):
        cb = EightBatch(seqs, 2, 64, 16, BF, seed=41)
        q, k, v = cb.tokens(4), cb.tokens(2), cb.tokens(2)
        w = torch.linspace(0.5, 1.5, 64, device="cuda")
        calls = [lambda **kw: sv.append_kv(k, v, *cb.eight(), q=q, q_norm=w, k_norm=w, **cb.scales(), **kw),
                 lambda **kw: sv.paged_attention(q, *cb.eight(), **cb.scales(), **kw),
                 lambda **kw: torch.stack(sv.read_kv(*cb.eight(), rows=cb.N, **cb.scales(), **kw))]
        want = [f() for f in calls]
        for f in calls:
            with pytest.raises(sv.SpecVerifyError, match="ws="):
                with torch.cuda.graph(torch.cuda.CUDAGraph()):
                    f()
        torch.cuda.synchronize()
        graphs = []
        for _ in range(2):                              # two graphs, each with its workspace
            ws, g = sv.CacheWorkspace(), torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                got = [f(ws=ws) for f in calls]
            graphs.append((g, got, ws))
        for g, got, ws in reversed(graphs):
            for x in got:
                x.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert ws.status() == 0
            for x, y in zip(got, want):
                assert torch.equal(x, y)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = [f(stream=side) for f in calls[:2]]
        with torch.cuda.stream(side):
            got.append(calls[2]())
        side.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_one_workspace_for_both_kinds_of_cache():
    """Calls on 16-bit and 8-bit caches in turn, tiles cut between CTAs in both."""
    a = CacheBatch([(6, 2500)], 2, 64, 16, BF, seed=42)
    b = EightBatch([(6, 2700)], 2, 64, 16, BF, seed=43)
    qa, qb = a.tokens(8), b.tokens(8)
    ws = sv.CacheWorkspace()
    first = None
    for _ in range(3):
        got = (sv.paged_attention(qa, *a.args(), ws=ws), sv.paged_attention(qb, *b.eight(), **b.scales(), ws=ws))
        assert ws.status() == 0
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(got, first))


def test_counts_that_no_call_leaves_are_reported():
    cb = EightBatch([(6, 3000)], 1, 64, 16, BF, seed=44)
    q = cb.tokens(4)
    ws = sv.CacheWorkspace()
    want = sv.paged_attention(q, *cb.eight(), **cb.scales(), ws=ws)
    ws.buf[256:256 + 2048].view(torch.int32).fill_(1 << 20)
    sv.paged_attention(q, *cb.eight(), **cb.scales(), ws=ws)
    assert ws.status() & sv.STATUS_OVERFLOW
    assert torch.equal(sv.paged_attention(q, *cb.eight(), **cb.scales(), ws=ws), want) and ws.status() == 0


def test_a_wait_that_runs_out_is_reported_and_the_workspace_serves_again(tmp_path):
    """A build whose attention leaves waits unanswered (SV_STALL=1)."""
    out = str(tmp_path / "libspecverify_stall.so")
    other = sv._declare(ctypes.CDLL(_build.build_variant(out, ["-DSV_STALL=1"])))

    def bind(lib):
        sv._native().bind8(*(ctypes.cast(f, ctypes.c_void_p).value
                             for f in (lib.sv_append_kv_normed, lib.sv_read_kv, lib.sv_paged_attention_scaled,
                                       lib.sv_paged_attention_scratch_size)))
    cb = EightBatch([(6, 880 + b) for b in range(60)], 2, 64, 16, BF, seed=45)
    q = cb.tokens(4)
    ws = sv.CacheWorkspace()
    want = sv.paged_attention(q, *cb.eight(), **cb.scales(), ws=ws)
    assert ws.status() == 0
    for _ in range(2):
        bind(other)
        try:
            sv.paged_attention(q, *cb.eight(), **cb.scales(), ws=ws)
            assert ws.status() & sv.STATUS_TIMEOUT
        finally:
            bind(sv.load())
        got = sv.paged_attention(q, *cb.eight(), **cb.scales(), ws=ws)
        assert ws.status() == 0 and torch.equal(got, want)


# ---------------------------------------------------------------------------
# refusals

def test_tensors_that_do_not_fit_are_refused():
    cb = EightBatch([(3, 20)], 2, 64, 16, BF, seed=46)
    q, k, v = cb.tokens(4), cb.tokens(2), cb.tokens(2)
    w, s = torch.ones(64, device="cuda"), cb.scales()
    half = torch.zeros(3, 2, 64, dtype=HF, device="cuda")
    bad = [
        lambda: sv.paged_attention(q, *cb.eight()),
        lambda: sv.paged_attention(q, *cb.eight(), k_scale=cb.ks),
        lambda: sv.paged_attention(q, *cb.eight(), k_scale=cb.ks.view(torch.uint8), v_scale=cb.vs),
        lambda: sv.paged_attention(q, *cb.eight(), k_scale=cb.ks[:, :, :1], v_scale=cb.vs),
        lambda: sv.paged_attention(q.float(), *cb.eight(), **s),
        lambda: sv.paged_attention(q, cb.k8.float().to(BF), cb.v8.float().to(BF), *cb.eight()[2:], **s),
        lambda: sv.paged_attention(q[:, :3], *cb.eight(), **s),
        lambda: sv.paged_attention(q, *cb.eight(), out=q.float(), **s),
        lambda: sv.append_kv(k, v, *cb.eight()),
        lambda: sv.append_kv(half, v, *cb.eight(), **s),
        lambda: sv.append_kv(k, v, *cb.eight(), q=q, q_norm=w.half(), **s),
        lambda: sv.append_kv(k, v, *cb.eight(), q=q, q_norm=w[:32], **s),
        lambda: sv.append_kv(k, v, *cb.eight(), q=q, q_norm=w.cpu(), **s),
        lambda: sv.append_kv(k, v, *cb.eight(), q=q, q_norm=w, k_norm=w.to(BF), **s),
        lambda: sv.append_kv(k, v, *cb.eight(), q_norm=w, **s),
        lambda: sv.append_kv(k, v, *cb.eight(), k_norm=w, eps=-1.0, **s),
        lambda: sv.append_kv(k, v, *cb.eight(), k_norm=w, eps=math.nan, **s),
        lambda: sv.read_kv(*cb.eight(), **s),
        lambda: sv.read_kv(*cb.eight(), rows=3, dtype=torch.float32, **s),
        lambda: sv.read_kv(*cb.eight(), rows=4, k_out=k, **s),
        lambda: sv.read_kv(*cb.eight(), k_out=k, v_out=half, **s),
        lambda: sv.read_kv(*cb.eight(), rows=3),
        lambda: sv.read_kv(half.view(3, 1, 2, 64), half.view(3, 1, 2, 64), *cb.eight()[2:], rows=3, dtype=BF),
    ]
    before = [x.view(torch.uint8).clone() for x in (cb.k8, cb.v8, cb.ks, cb.vs)]
    for i, f in enumerate(bad):
        with pytest.raises(sv.SpecVerifyError):
            f()
            pytest.fail(f"call {i} was taken")
    for x, y in zip((cb.k8, cb.v8, cb.ks, cb.vs), before):
        assert torch.equal(x.view(torch.uint8), y)


def test_no_rows_and_no_sequences():
    cb = EightBatch([(0, 20), (0, 0)], 2, 64, 16, BF, seed=47)
    q, k, v = cb.tokens(4), cb.tokens(2), cb.tokens(2)
    assert sv.append_kv(k, v, *cb.eight(), q=q, **cb.scales()).shape == (0, 4, 64)
    assert sv.paged_attention(q, *cb.eight(), **cb.scales()).shape == (0, 4, 64)
    assert [tuple(x.shape) for x in sv.read_kv(*cb.eight(), rows=0, **cb.scales())] == [(0, 2, 64)] * 2


# ---------------------------------------------------------------------------
# the cache class and the example

@pytest.mark.parametrize("eight", [False, True])
def test_passes_rollbacks_and_reads_of_a_paged_cache(eight):
    d, f = 64, rope_frequencies(64, device="cuda")
    c = PagedCache(2, 20, 16, 2, d, dtype=E4M3 if eight else BF, inv_freq=f)
    g = torch.Generator().manual_seed(48)
    rnd = lambda n, h: torch.randn(n, h, d, generator=g).to(BF).cuda()  # noqa: E731
    w = (1 + 0.2 * torch.randn(d, generator=g)).cuda()
    kept = {0: [], 1: []}
    for step, new in enumerate(({0: 40, 1: 3}, {0: 6, 1: 6}, {1: 6, 0: 6})):
        n = sum(new.values())
        q, k, v = rnd(n, 4), rnd(n, 2), rnd(n, 2)
        c.begin(new)
        q = c.append(1, q, k, v, q_norm=w, k_norm=w)
        out = c.attend(1, q)
        at = 0
        for s, m in new.items():
            kept[s] += [(k[at + i], v[at + i]) for i in range(m)]
            at += m
        held = c.read(1)
        at = 0
        for s, m in new.items():                        # attention over what is read back
            kr, vr = (x.double().repeat_interleave(2, 1) for x in held[s])
            for j in range(m):
                L = kr.shape[0] - m + j + 1
                p = (torch.einsum("hd,khd->hk", q[at + j].double(), kr[:L]) / d ** 0.5).softmax(-1)
                want, room = (torch.einsum("hk,khd->hd", p, x) for x in (vr[:L], vr[:L].abs()))
                assert bool(((out[at + j].double() - want).abs() <= room * 2.0 ** -7 + 1e-5).all())
            at += m
        if step == 1:
            for s, m in ((0, 4), (1, 5)):
                c.rollback(s, m)
                del kept[s][-m:]
    for s, (kr, vr) in c.read(1).items():               # what was appended, to the cache's precision
        k, v = (torch.stack([x[i] for x in kept[s]]) for i in (0, 1))
        kw, kt = turned(k, w, 1e-6, torch.arange(k.shape[0]), f.cpu(), False)
        step_of = 2.0 ** -4 if eight else 2.0 ** -8
        for got, want, tol in ((kr, kw, kt), (vr, v.cpu().double(), 0.0)):
            top = want.abs().amax(-1, keepdim=True)
            within(got, want, want.abs() * step_of * 1.01 + tol + (top * 2.0 ** -17 if eight else 2.0 ** -25))
    assert c.read(0, [1])[1][0].shape == (len(kept[1]), 2, d) and c.read(0, []) == {}


def test_the_example_runs_on_eight_bits_with_norms():
    spec = importlib.util.spec_from_file_location("paged_decoding", os.path.join(ROOT, "examples", "paged_decoding.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    for greedy in (True, False):
        out, rate = m.decode([11, 222, 3333, 44, 5], 20, 4, greedy=greedy, eight=True, norms=True)
        assert len(out) == 20 and all(0 <= t < 4096 for t in out) and 1 <= rate <= 5
