"""Head norms, the 8-bit cache, its read-back and attention over it against their
64-bit definitions, at the sizes and masks where they can go wrong."""
import math

import pytest
import torch

import speculative_decoding_verification_08_gb300 as sv
from cache_refs import CacheBatch, attention, default_scale
from eight_refs import E4M3, E8M0, EightBatch, power, scale_exponents, turned, values

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


def freqs(rot):
    i = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    return torch.pow(10000.0, -2.0 * i / max(rot, 1))


def positions_of(seqs):
    return torch.cat([torch.arange(t - n, t) for n, t in seqs] + [torch.zeros(0, dtype=torch.long)])


def slots_of(cb):
    """(row, page, slot in page) of every new token."""
    for b, (n, t) in enumerate(cb.seqs):
        for j in range(n):
            s = t - n + j
            yield cb.starts[b] + j, int(cb.table[b, s // cb.page]), s % cb.page


# ---------------------------------------------------------------------------
# norms and rotation

APPEND = [
    # sequences (new, length), q heads, kv heads, d, page, type, rot, interleaved, heads first, norms
    ([(1, 1)], 1, 1, 64, 16, BF, 64, False, False, "qk"),
    ([(1, 701)], 32, 8, 128, 64, BF, 128, False, True, "qk"),
    ([(6, 6), (6, 70), (6, 129)], 8, 2, 128, 64, HF, 128, False, True, "k"),
    ([(0, 33), (5, 40), (0, 0), (17, 17)], 6, 2, 96, 48, BF, 48, False, False, "q"),
    ([(33, 97), (1, 20)], 4, 4, 80, 16, HF, 40, False, True, "qk"),
    ([(9, 64), (3, 3)], 3, 1, 64, 8, BF, 32, True, False, "qk"),
    ([(9, 9), (2, 31)], 7, 1, 16, 8, HF, 4, True, True, "qk"),
    ([(4, 9), (700, 720)], 2, 2, 32, 24, BF, 0, False, False, "qk"),
    ([(2, 9)], 5, 3, 48, 16, BF, 20, False, False, "qk"),
    ([(1300, 1300)], 2, 1, 112, 16, BF, 112, False, False, "qk"),
]


def append_inputs(case, cb, seed):
    seqs, hq, hkv, d, page, dt, rot, inter, first, norms = case
    k, v, q = cb.tokens(hkv, 2.0), cb.tokens(hkv), cb.tokens(hq)
    g = torch.Generator().manual_seed(seed)
    wt = torch.float32 if seed % 2 else dt
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(wt).cuda() if x in norms else None for x in "qk"]
    return k, v, q, w, freqs(rot) if rot else None


@pytest.mark.parametrize("case", APPEND)
@pytest.mark.parametrize("seed", [3, 4])
def test_normed_append_writes_only_its_slots(case, seed):
    seqs, hq, hkv, d, page, dt, rot, inter, first, norms = case
    cb = CacheBatch(seqs, hkv, d, page, dt, heads_first=first, fill=False, seed=seed)
    k, v, q, (qn, kn), f = append_inputs(case, cb, seed)
    kept = [x.clone() for x in (k, v, q)]
    ws = sv.CacheWorkspace()
    got = sv.append_kv(k, v, *cb.args(), inv_freq=f, q=q, interleaved=inter, q_norm=qn, k_norm=kn, eps=1e-5, ws=ws)
    assert ws.status() == 0
    for x, y in zip((k, v, q), kept):
        assert torch.equal(x, y)
    pos, eps = positions_of(seqs), torch.finfo(dt).eps / 2
    fc = f.cpu() if rot else None
    want, tol = turned(q, qn, 1e-5, pos, fc, inter)
    within(got, want, tol + want.abs() * eps + 2.0 ** -25)
    want, tol = turned(k, kn, 1e-5, pos, fc, inter)
    tol = tol + want.abs() * eps + 2.0 ** -25
    kc, vc = cb.k.cpu(), cb.v.cpu()
    written = torch.zeros(kc.shape[:2], dtype=torch.bool)
    for row, p, at in slots_of(cb):
        written[p, at] = True
        within(kc[p, at], want[row], tol[row])
        assert torch.equal(vc[p, at], v[row].cpu())
    assert bool(torch.isnan(kc[~written]).all()) and bool(torch.isnan(vc[~written]).all())


@pytest.mark.parametrize("case", [c for c in APPEND if c[3] % 16 == 0])
@pytest.mark.parametrize("norms", ["", "qk"])
def test_append_to_eight_bits(case, norms):
    """Scales are the definition's wherever the largest magnitude is not within fp32
    error of a border; a code is the nearest to the value, whose fp32 error counts."""
    seqs, hq, hkv, d, page, dt, rot, inter, first, _ = case
    cb = EightBatch(seqs, hkv, d, page, dt, heads_first=first, fill=False, seed=5)
    k, v, q, (qn, kn), f = append_inputs(case[:-1] + (norms,), cb, 5)
    ws = sv.CacheWorkspace()
    got = sv.append_kv(k, v, *cb.eight(), inv_freq=f, q=q, interleaved=inter, q_norm=qn, k_norm=kn, eps=1e-5,
                       **cb.scales(), ws=ws)
    assert ws.status() == 0
    pos, fc = positions_of(seqs), f.cpu() if rot else None
    want, tol = turned(q, qn, 1e-5, pos, fc, inter)
    within(got, want, tol + want.abs() * (torch.finfo(dt).eps / 2) + 2.0 ** -25)
    kw, kt = turned(k, kn, 1e-5, pos, fc, inter)
    vw = v.cpu().double()
    used = torch.zeros(cb.k8.shape[:2], dtype=torch.bool)
    for name, want, tol in (("k", kw, kt), ("v", vw, torch.zeros_like(vw))):
        code, scale = getattr(cb, name + "8").cpu().contiguous(), getattr(cb, name + "s").cpu().contiguous()
        byte = scale.view(torch.uint8).int() - 127
        held = values(code, scale)
        for row, p, at in slots_of(cb):
            used[p, at] = True
            e, t = byte[p, at], tol[row].amax(-1)
            top = want[row].abs().amax(-1)
            low, high = scale_exponents((top - t).clamp(min=0).unsqueeze(-1)), scale_exponents((top + t).unsqueeze(-1))
            assert bool(((e >= low) & (e <= high)).all())
            # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale where it is subnormal
            step = torch.maximum(want[row].abs() * 2.0 ** -4, power(e).unsqueeze(-1) * 2.0 ** -10)
            within(held[p, at], want[row], step + tol[row] * 1.07)
        raw = code.view(torch.uint8)
        assert bool((raw[~used] == 0x7f).all()) and bool((scale.view(torch.uint8)[~used] == 255).all())


def test_eight_bit_values_nearest_and_scales_exact():
    """Values without an error in fp32: codes and scales to the bit, ties to even,
    at the borders of the scales, for the smallest and the largest numbers."""
    rows = [torch.linspace(-448, 448, 64), torch.linspace(-1, 1, 64) ** 3 * 448.0, torch.arange(64) * 7.0,
            torch.arange(64) * 7.0 + 8, torch.full((64,), 2.0 ** -20), torch.zeros(64), torch.arange(64) * 2.0 ** -130,
            torch.cat((torch.full((32,), 3e38), torch.linspace(-1, 1, 32))), torch.arange(64) * 2.0 ** 95,
            torch.arange(64) * 2.0 ** -108, torch.cat((torch.tensor([449.0]), torch.zeros(63))),
            17 + torch.arange(64) / 4]
    v = torch.stack(rows).to(BF).view(len(rows), 1, 64)
    cb = EightBatch([(len(rows), len(rows))], 1, 64, 16, BF, fill=False)
    sv.append_kv(v.cuda(), v.cuda(), *cb.eight(), **cb.scales())
    e = scale_exponents(v.double())
    want = (v.double() * power(-e).unsqueeze(-1)).clamp(-448, 448).float().to(E4M3)
    for code, scale in ((cb.k8, cb.ks), (cb.v8, cb.vs)):
        for row, p, at in slots_of(cb):
            assert int(scale.view(torch.uint8)[p, at, 0]) == int(e[row, 0]) + 127, row
            assert torch.equal(code[p, at].cpu().float(), want[row].float()), row


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_vector_that_is_not_finite_is_nan_as_a_whole(bad):
    cb = EightBatch([(3, 20)], 2, 64, 16, BF, fill=False)
    k, v, q = cb.tokens(2), cb.tokens(2), cb.tokens(4)
    k[1, 0, 5] = bad
    v[2, 1, 63] = bad
    sv.append_kv(k, v, *cb.eight(), inv_freq=freqs(64), q=q, k_norm=torch.ones(64, device="cuda"), **cb.scales())
    kr, vr = sv.read_kv(*cb.eight(), rows=3, **cb.scales())
    kn, vn = torch.isnan(kr), torch.isnan(vr)
    for got, at in ((kn, (1, 0)), (vn, (2, 1))):
        assert bool(got[at].all()) and int(got.sum()) == 64
    assert not bool(torch.isinf(kr).any()) and not bool(torch.isinf(vr).any())


def test_queries_in_place_on_slices_and_far_positions():
    cb = EightBatch([(5, 12)], 2, 64, 16, HF, fill=False)
    fused = torch.randn(5, 8 * 64, generator=torch.Generator().manual_seed(1)).to(HF).cuda()
    q, k, v = fused[:, :256].view(5, 4, 64), fused[:, 256:384].view(5, 2, 64), fused[:, 384:].view(5, 2, 64)
    pos = torch.tensor([0, 1, 1 << 20, (1 << 30) + 7, 3], dtype=torch.int32, device="cuda")
    w = torch.linspace(0.5, 2, 64, device="cuda")
    f = freqs(64)
    want, tol = turned(q, w, 1e-6, pos.cpu(), f.cpu(), False)
    kw, _ = turned(k, w, 1e-6, pos.cpu(), f.cpu(), False)
    assert sv.append_kv(k, v, *cb.eight(), inv_freq=f, q=q, q_out=q, positions=pos, q_norm=w, k_norm=w,
                        **cb.scales()) is q
    within(q, want, tol + want.abs() * 2.0 ** -11 + 2.0 ** -25)
    got, _ = sv.read_kv(*cb.eight(), rows=5, **cb.scales())
    top = kw.abs().amax(-1, keepdim=True)
    within(got, kw, kw.abs() * 2.0 ** -4 + top * (2.0 ** -17 + 2.0 ** -18))


def test_pages_and_lengths_that_do_not_fit():
    cb = EightBatch([(3, 20), (2, 5), (2, 2)], 1, 32, 16, BF, fill=False, extra_tokens=2)
    cb.pages[0, 1] = 99                       # slots 16..: no such page
    cb.kv_len[2] = 1                          # the first of two new tokens would be in slot -1
    k, v, q = cb.tokens(1), cb.tokens(1), cb.tokens(2)
    ws = sv.CacheWorkspace()
    before = cb.k8.clone()
    out = torch.full_like(q, 7.0)
    sv.append_kv(k, v, *cb.eight(), inv_freq=freqs(32), q=q, q_out=out, q_norm=torch.ones(32, device="cuda"),
                 **cb.scales(), ws=ws)
    assert ws.status() == sv.STATUS_BAD_PAGE | sv.STATUS_BAD_LENGTH
    assert bool((out[-2:] == 7).all()) and not bool((out[:-2] == 7).any())
    changed = (cb.k8.view(torch.uint8) != before.view(torch.uint8)).any(-1).any(-1)
    assert int(changed.sum()) == 3            # two of sequence 1, slot 0 of sequence 2
    ko = torch.full((9, 1, 32), 7.0, dtype=BF, device="cuda")
    vo = ko.clone()
    sv.read_kv(*cb.eight(), k_out=ko, v_out=vo, **cb.scales(), ws=ws)
    assert ws.status() == sv.STATUS_BAD_PAGE | sv.STATUS_BAD_LENGTH
    for x in (ko, vo):
        assert bool((x[:3] == 0).all()) and bool((x[5] == 0).all()) and bool((x[-2:] == 7).all())
        assert bool((x[3:5] != 0).any()) and bool((x[6] != 0).any())
    cb.kv_len[1] = -1                         # left out
    out.fill_(7.0)
    sv.append_kv(k, v, *cb.eight(), q=q, q_out=out, q_norm=torch.ones(32, device="cuda"), **cb.scales(), ws=ws)
    assert ws.status() & sv.STATUS_BAD_LENGTH and bool((out[3:5] == 7).all())


# ---------------------------------------------------------------------------
# the way back

READ = [
    # sequences (rows read, length), kv heads, d, page, type, heads first
    ([(1, 1)], 1, 16, 8, BF, False),
    ([(701, 701)], 8, 128, 64, BF, True),
    ([(0, 40), (33, 40), (0, 0), (17, 17)], 2, 96, 48, HF, False),
    ([(5, 300), (300, 300), (1, 7)], 3, 80, 16, BF, True),
    ([(9, 64)] * 30, 1, 64, 32, HF, False),
]


@pytest.mark.parametrize("case", READ)
def test_read_back(case):
    seqs, hkv, d, page, dt, first = case
    cb = EightBatch(seqs, hkv, d, page, dt, heads_first=first, seed=7, extra_tokens=1, scale_spread=2.0)
    ws = sv.CacheWorkspace()
    k = torch.full((cb.N, hkv, 2 * d), 7.0, dtype=dt, device="cuda")[..., d:]
    _, v = sv.read_kv(*cb.eight(), k_out=k, dtype=dt, **cb.scales(), ws=ws)
    assert ws.status() == 0
    # a float16 result below 2^-14 is rounded in steps of 2^-24
    for got, cache in ((k, cb.k), (v, cb.v)):
        for b, (n, t) in enumerate(seqs):
            want = cb.sequence(cache, b)[t - n:]
            tol = torch.zeros_like(want) if dt == BF else torch.full_like(want, 2.0 ** -25)
            within(got[cb.starts[b]:cb.starts[b + 1]], want, tol)
    assert bool((k[-1] == 7).all())


@pytest.mark.parametrize("d,page", [(8, 8), (128, 64), (72, 24)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_read_of_a_sixteen_bit_cache_gives_its_bits(d, page, dt):
    seqs = [(5, 40), (40, 40), (0, 3)]
    cb = CacheBatch(seqs, 3, d, page, dt, heads_first=True, seed=8)
    k, v = sv.read_kv(*cb.args(), rows=cb.N)
    for got, cache in ((k, cb.k), (v, cb.v)):
        for b, (n, t) in enumerate(seqs):
            assert torch.equal(got[cb.starts[b]:cb.starts[b + 1]].cpu().double(), cb.sequence(cache, b)[t - n:])


# ---------------------------------------------------------------------------
# attention

ATTEND = [
    # sequences, q heads, kv heads, d, page, type, heads first, window
    ([(1, 1)], 1, 1, 64, 16, BF, False, 0),
    ([(1, 1000)], 32, 8, 128, 64, BF, True, 0),
    ([(6, 6), (6, 70), (6, 129), (6, 128)], 8, 2, 128, 64, HF, True, 0),
    ([(6, 1500), (6, 2049)], 16, 4, 64, 16, HF, False, 0),
    ([(0, 33), (5, 40), (0, 0), (17, 17)], 6, 2, 96, 48, BF, False, 0),
    ([(33, 97), (1, 20), (3, 513)], 28, 4, 80, 16, HF, True, 0),
    ([(9, 64), (3, 3)], 3, 1, 16, 8, BF, False, 0),
    ([(130, 300), (2, 400)], 4, 1, 128, 32, BF, True, 0),
    ([(7, 900), (40, 300)], 8, 2, 64, 16, BF, False, 100),
    ([(7, 900), (1, 130)], 4, 2, 112, 256, HF, True, 1),
    ([(3, 600)], 40, 1, 128, 16, BF, False, 0),
    ([(17, 700)], 8, 2, 128, 64, BF, False, 300),
]


@pytest.mark.parametrize("case", ATTEND)
def test_attention_over_eight_bits(case):
    seqs, hq, hkv, d, page, dt, first, window = case
    cb = EightBatch(seqs, hkv, d, page, dt, heads_first=first, seed=9, scale_spread=0.5)
    q = cb.tokens(hq, 1.5)
    ws = sv.CacheWorkspace()
    got = sv.paged_attention(q, *cb.eight(), window=window, **cb.scales(), ws=ws)
    assert ws.status() == 0
    within(got, *attention(cb, q, default_scale(d), window))


@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0])
def test_scales_of_either_sign(scale):
    cb = EightBatch([(3, 200), (1, 7)], 2, 64, 16, BF, seed=10)
    q = cb.tokens(6)
    within(sv.paged_attention(q, *cb.eight(), scale=scale, **cb.scales()), *attention(cb, q, scale, 0))


def test_rows_that_see_nothing_and_rows_behind_the_last():
    cb = EightBatch([(6, 6), (5, 300)], 1, 64, 16, BF, seed=11, extra_tokens=3)
    cb.kv_len[0] = 2                          # of six new tokens, four lie before slot 0
    q = cb.tokens(4)
    out = torch.full_like(q, 7.0)
    sv.paged_attention(q, *cb.eight(), out=out, **cb.scales())
    cb.seqs[0] = (6, 2)
    want, tol = attention(cb, q, default_scale(64), 0)
    assert bool((out[:4] == 0).all()) and bool((out[-3:] == 7).all())
    within(out[:-3], want[:-3], tol[:-3])


def test_a_pass_as_it_is_used():
    """Prompt, round and single token through an 8-bit cache with norms: what is
    attended to is what was written, and what is read back."""
    d, f = 64, freqs(64)
    cb = EightBatch([(40, 40), (70, 70)], 2, d, 16, BF, fill=False, seed=12)
    w = [torch.linspace(0.8, 1.2, d, device="cuda").to(BF) for _ in range(2)]
    lens = [40, 70]
    for new in (None, (6, 6), (1, 1)):
        if new:
            lens = [x + n for x, n in zip(lens, new)]
            cb.seqs = list(zip(new, lens))
            cb.starts = [0, new[0], new[0] + new[1]]
            cb.N = sum(new)
            cb.q_start = torch.tensor(cb.starts, dtype=torch.int32, device="cuda")
            cb.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
            wide = -(-max(lens) // 16)
            table = torch.arange(2 * wide, dtype=torch.int32).view(2, wide)
            table[:, :cb.table.shape[1]] = cb.table if wide >= cb.table.shape[1] else cb.table[:, :wide]
            # pages that no sequence has yet
            free = [p for p in range(cb.k8.shape[0]) if p not in cb.table[cb.table >= 0].tolist()]
            for b, (_, t) in enumerate(cb.seqs):
                for i in range(-(-t // 16)):
                    if i >= -(-(t - new[b]) // 16):
                        table[b, i] = free.pop()
            cb.table, cb.pages = table, table.cuda()
        k, v, q = cb.tokens(2, 2.0), cb.tokens(2), cb.tokens(8)
        q = sv.append_kv(k, v, *cb.eight(), inv_freq=f, q=q, q_norm=w[0], k_norm=w[1], **cb.scales())
        out = sv.paged_attention(q, *cb.eight(), **cb.scales())
        cb.refresh()
        within(out, *attention(cb, q, default_scale(d), 0))
        kr, vr = sv.read_kv(*cb.eight(), rows=cb.N, **cb.scales())
        for b, (n, t) in enumerate(cb.seqs):
            rows = slice(cb.starts[b], cb.starts[b + 1])
            assert torch.equal(kr[rows].cpu().double(), cb.sequence(cb.k, b)[t - n:])
            assert torch.equal(vr[rows].cpu().double(), cb.sequence(cb.v, b)[t - n:])
