"""warp_sample against its 64-bit definition: the kept set and the token are
equal, the probabilities good to fp32 rounding."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_08_gb300 as sv
from cache_refs import warp_row

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
# one exp2 good to 2^-22, the reciprocal of the mass and two products rounded
PROB_TOL = 2.0 ** -22 + 4 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sv.build()
    return sv.load()


def check(z, u, T=None, k=None, p=None, m=None, ws=None):
    """One call, every row against the definition."""
    R, V = z.shape
    dev = lambda x, t: None if x is None else torch.as_tensor(np.asarray(x), dtype=t).cuda()  # noqa: E731
    ws = ws or sv.CacheWorkspace()
    tok, probs = sv.warp_sample(z, dev(u, torch.float64), temperature=dev(T, torch.float32),
                                top_k=dev(k, torch.int32), top_p=dev(p, torch.float32),
                                min_p=dev(m, torch.float32), probs=True, ws=ws)
    only, none = sv.warp_sample(z, dev(u, torch.float64), temperature=dev(T, torch.float32),
                                top_k=dev(k, torch.int32), top_p=dev(p, torch.float32),
                                min_p=dev(m, torch.float32), ws=ws)
    assert none is None and torch.equal(tok, only)
    rows, none = sv.warp_sample(z, temperature=dev(T, torch.float32), top_k=dev(k, torch.int32),
                                top_p=dev(p, torch.float32), min_p=dev(m, torch.float32),
                                probs=True, ws=ws)[::-1]
    assert none is None and torch.equal(rows, probs)
    assert ws.status() == 0
    zc, tok, probs = z.float().cpu().numpy(), tok.cpu().numpy(), probs.cpu().numpy()
    f32 = lambda x, r, d: d if x is None else float(np.float32(np.asarray(x)[r]))  # noqa: E731
    for r in range(R):
        want, kept, t = warp_row(zc[r], f32(T, r, 1.0), 0 if k is None else int(k[r]),
                                 f32(p, r, 1.0), f32(m, r, 0.0), float(np.asarray(u)[r]))
        assert tok[r] == t, (r, tok[r], t)
        assert np.array_equal(probs[r] > 0, kept & (want > 1e-29)), r
        assert np.all(np.abs(probs[r] - want) <= PROB_TOL * want + 1e-29), r


def logits(R, V, dt, spread=3.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(R, V, generator=g) * spread).to(TYPES[dt]).cuda()


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 32000, 50257])
def test_every_filter_on_every_size(dt, V):
    R = 16
    rng = np.random.RandomState(V)
    z = logits(R, V, dt, seed=V)
    u, T = rng.rand(R), rng.uniform(0.5, 1.5, R)
    k, p, m = rng.randint(1, 300, R), rng.uniform(0.3, 0.999, R), rng.uniform(1e-4, 0.2, R)
    check(z, u)
    check(z, u, T)
    check(z, u, T, k=k)
    check(z, u, T, p=p)
    check(z, u, T, m=m)
    check(z, u, T, k, p)
    check(z, u, T, k, p, m)
    check(z, u, T, None, p, m)


@pytest.mark.parametrize("dt,V,R", [("f32", 128256, 6), ("bf16", 128256, 6), ("f32", 262144, 3),
                                    ("f16", 151937, 4), ("f32", 500009, 2)])
def test_large_vocabularies(dt, V, R):
    rng = np.random.RandomState(V)
    z = logits(R, V, dt, 2.0, seed=V)
    u = rng.rand(R)
    check(z, u)
    check(z, u, rng.uniform(0.5, 1.5, R), rng.randint(1, V, R), rng.uniform(0.8, 0.9999, R))
    check(z, u, None, None, rng.uniform(0.8, 0.9999, R), rng.uniform(1e-7, 0.01, R))


def test_filter_values_at_their_ends():
    z = logits(12, 3000, "f32", seed=1)
    u = np.linspace(0, 1 - 2.0 ** -53, 12)
    k = [0, -3, 1, 2999, 3000, 5000, 1, 2, 0, 0, 7, 7]
    p = [1.0, 2.0, 1.0, 0.999999, 0.5, 1.0, 0.0, -1.0, 1e-9, np.nan, 0.9, 1.0]
    m = [0.0, -1.0, 0.0, 0.0, 0.0, 1e-30, 0.5, 0.0, 0.0, np.nan, 1.0, 3.0]
    kk, pp, mm = np.array(k), np.array(p, np.float32), np.array(m, np.float32)
    ref = [(int(a), 1.0 if np.isnan(b) else float(b), 0.0 if np.isnan(c) else float(c))
           for a, b, c in zip(kk, pp, mm)]
    tok, probs = sv.warp_sample(z, torch.as_tensor(u).cuda(), top_k=torch.as_tensor(kk, dtype=torch.int32).cuda(),
                                top_p=torch.as_tensor(pp).cuda(), min_p=torch.as_tensor(mm).cuda(), probs=True)
    for r in range(12):
        want, kept, t = warp_row(z[r].cpu().numpy(), 1.0, *ref[r], u=float(u[r]))
        assert int(tok[r]) == t, r
        assert np.all(np.abs(probs[r].cpu().numpy() - want) <= PROB_TOL * want + 1e-29), r


@pytest.mark.parametrize("V", [5, 2000, 40000])
def test_equal_logits_are_taken_lowest_index_first(V):
    """Rows of one value, of two, and of a few."""
    rows = [np.zeros(V), np.full(V, -3.5), np.where(np.arange(V) % 3 == 0, 1.0, 0.5),
            np.round(np.random.RandomState(V).randn(V) * 2) / 2, -0.0 * np.ones(V)]
    z = torch.as_tensor(np.stack(rows), dtype=torch.float32).cuda()
    R = len(rows)
    u = np.random.RandomState(1).rand(R)
    for k in (None, np.full(R, min(V, 3)), np.full(R, V // 2 + 1)):
        for p in (None, np.full(R, 0.37), np.full(R, 0.8)):
            check(z, u, None, k, p)
    check(z.to(torch.bfloat16), u, np.full(R, 0.7), np.full(R, V // 3 + 1), np.full(R, 0.5),
          np.full(R, 0.9))


def test_masked_logits_and_a_single_survivor():
    V = 5000
    z = logits(6, V, "f32", seed=2)
    z[:, ::2] = float("-inf")
    z[1] = float("-inf")
    z[1, 4321] = -7.0
    z[2] = float("-inf")
    z[2, [7, 9]] = torch.tensor([-1e30, -1e30], device="cuda")
    z[3, 1::2] = torch.finfo(torch.float32).min
    z[4, 100] = 3e38
    u = np.array([0.3, 0.999, 0.5, 0.7, 0.5, 0.0])
    check(z, u)
    check(z, u, None, np.full(6, 4000), np.full(6, 0.9))
    check(z, u, np.full(6, 2.0), None, None, np.full(6, 0.05))


@pytest.mark.parametrize("dt", list(TYPES))
def test_rows_in_rising_order(dt):
    """Without filters the maximum is found on the way: rows that rise, that
    jump late, and whose first parts are masked."""
    V = 70001
    up = torch.linspace(-60.0, 25.0, V)
    late = torch.full((V,), -3.0)
    late[-5] = 40.0
    masked = torch.linspace(-1.0, 1.0, V)
    masked[: V * 3 // 4] = float("-inf")
    saw = (torch.arange(V) % 977).float() / 100 + torch.arange(V).float() / 3000
    z = torch.stack([up, late, masked, saw, up.flip(0)]).to(TYPES[dt]).cuda()
    zc = z.float().cpu().numpy()
    for T in (np.ones(5), np.array([0.3, 1.0, 5.0, 2.0, 0.7])):
        temp = torch.as_tensor(T, dtype=torch.float32).cuda()
        for u in (0.0, 0.3, 0.77, 1 - 2.0 ** -53):
            tok, probs = sv.warp_sample(z, torch.full((5,), u, dtype=torch.float64, device="cuda"),
                                        temperature=temp, probs=True)
            for r in range(5):
                # (what lies more than 85 T below the maximum weighs nothing)
                low = zc[r] - zc[r].max() < np.float32(-85) * np.float32(T[r])
                want, _, t = warp_row(np.where(low, -np.inf, zc[r]), float(temp[r]), u=u)
                # masses are good to 1e-10: that far from a border either side may be drawn
                # (the falling row's last e^-23 lie within it of the row's end)
                got, c = int(tok[r]), np.cumsum(want)
                assert want[got] > 0 and c[got] - want[got] <= u + 1e-10 and c[got] >= u - 1e-10, (r, u)
                assert got == t or abs(c[min(got, t)] - u) <= 1e-10, (r, u)
                assert np.all(np.abs(probs[r].cpu().numpy() - want) <= PROB_TOL * want + 1e-29), (r, u)


@pytest.mark.parametrize("R,V,dt", [(3, 262144, "f32"), (2, 262145, "bf16"), (40, 9001, "f16"), (300, 700, "f32")])
def test_plain_rows_without_answers(R, V, dt):
    z = logits(R, V, dt, seed=R)
    z[0, V // 2:] = float("-inf")
    z[1] = float("-inf")
    u = torch.rand(R, dtype=torch.float64, generator=torch.Generator().manual_seed(R)).cuda()
    ws = sv.CacheWorkspace()
    tok, probs = sv.warp_sample(z, u, probs=True, ws=ws)
    assert ws.status() == sv.STATUS_ZERO_MASS
    assert int(tok[1]) == -1 and not bool(probs[1].any())
    for r in (0, R - 1):
        if r != 1:
            want, _, t = warp_row(z[r].float().cpu().numpy(), u=float(u[r]))
            assert int(tok[r]) == t
            assert np.all(np.abs(probs[r].cpu().numpy() - want) <= PROB_TOL * want + 1e-29)
    for bad in (float("nan"), float("inf")):
        y = z.clone()
        y[0, V - 1] = bad
        ws = sv.CacheWorkspace()
        tok, probs = sv.warp_sample(y, u, probs=True, ws=ws)
        assert ws.status() == sv.STATUS_ZERO_MASS | sv.STATUS_BAD_VALUE
        assert int(tok[0]) == -1 and not bool(probs[0].any())


def test_rows_without_an_answer():
    V = 3000
    z = logits(6, V, "bf16", seed=3)
    z[0] = float("-inf")
    z[2, 17] = float("nan")
    z[3, 2999] = float("inf")
    T = torch.tensor([1.0, 1.0, 1.0, 1.0, 0.0, 1.0], device="cuda")
    u = torch.full((6,), 0.4, dtype=torch.float64, device="cuda")
    ws = sv.CacheWorkspace()
    tok, probs = sv.warp_sample(z, u, temperature=T, probs=True, ws=ws)
    assert ws.status() == sv.STATUS_ZERO_MASS | sv.STATUS_BAD_VALUE
    tok = tok.tolist()
    assert [t == -1 for t in tok] == [True, False, True, True, True, False]
    for r in (0, 2, 3, 4):
        assert not bool(probs[r].any())
    for r in (1, 5):
        assert tok[r] == warp_row(z[r].float().cpu().numpy(), u=0.4)[2]
        assert abs(float(probs[r].double().sum()) - 1) < 1e-5


def test_strided_rows_shapes_and_outputs():
    B, K1, V = 3, 4, 1001
    wide = torch.randn(B, K1, V + 7, generator=torch.Generator().manual_seed(4)).cuda()
    z = wide[..., 3:V + 3]                              # not 16-byte aligned
    u = torch.rand(B, K1, dtype=torch.float64, generator=torch.Generator().manual_seed(5)).cuda()
    tok, probs = sv.warp_sample(z, u, probs=True)
    assert tok.shape == (B, K1) and probs.shape == (B, K1, V)
    for b in range(B):
        for i in range(K1):
            want, _, t = warp_row(z[b, i].cpu().numpy(), u=float(u[b, i]))
            assert int(tok[b, i]) == t
            assert np.all(np.abs(probs[b, i].cpu().numpy() - want) <= PROB_TOL * want)
    t1, _ = sv.warp_sample(z[0, 0], u[0, 0])
    assert int(t1) == int(tok[0, 0])
    out, tout = torch.empty(B, K1, V, device="cuda"), torch.empty(B, K1, dtype=torch.int32, device="cuda")
    a, b = sv.warp_sample(z, u, probs_out=out, token_out=tout)
    assert a is tout and b is out and torch.equal(out, probs) and torch.equal(tout, tok)
    e, _ = sv.warp_sample(torch.empty(0, V, device="cuda"), torch.empty(0, dtype=torch.float64, device="cuda"))
    assert e.shape == (0,)


def test_a_draw_that_needs_every_digit():
    """Goals set a hair on either side of a boundary between two tokens: the
    64-bit order decides."""
    V = 20000
    z = logits(1, V, "f32", 1.0, seed=6)
    w = np.exp(z[0].double().cpu().numpy() - float(z.max()))
    c = np.cumsum(w) / w.sum()
    at = [10, 777, 5000, 12345, 19990]
    rel = 1e-9
    u = np.array([c[i] * (1 + s * rel) for i in at for s in (-1, 1)])
    tok, _ = sv.warp_sample(z.expand(len(u), V).contiguous(), torch.as_tensor(u).cuda())
    assert tok.tolist() == [i + (s > 0) for i in at for s in (-1, 1)]


def test_a_nucleus_that_needs_every_digit():
    V = 4096
    z = logits(1, V, "f32", 1.0, seed=7)
    zc = z[0].cpu().numpy().astype(np.float64)
    order = np.argsort(-zc, kind="stable")
    w = np.exp(zc[order] - zc.max())
    c = np.cumsum(w) / w.sum()
    ps = np.array([np.float32(c[i]) for i in (3, 100, 1000, 3000)], dtype=np.float32)
    ps = np.concatenate([ps, np.nextafter(ps, np.float32(0)), np.nextafter(ps, np.float32(1))])
    check(z.expand(len(ps), V).contiguous(), np.full(len(ps), 0.5), None, None, ps)


@pytest.mark.parametrize("step", [0.01, 0.02, 0.05, 0.1, 0.25, 1.0])
def test_borders_of_many_equal_logits(step):
    """Logits on a grid: a border holds from a few dozen to thousands of equal
    values, ranked by one warp, by a CTA, by the cluster, or bisected."""
    V, R = 50000, 6
    g = torch.Generator().manual_seed(int(step * 1000))
    z = (torch.round(torch.randn(R, V, generator=g) * 3 / step) * step).cuda()
    rng = np.random.RandomState(9)
    u, k, p = rng.rand(R), rng.randint(1, V, R), rng.uniform(0.3, 0.999, R)
    check(z, u, None, k)
    check(z, u, None, None, p)
    check(z, u, np.full(R, 0.8), k, p, np.full(R, 1e-4))


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("V", [40, 310, 1913, 30011])
def test_a_nucleus_that_reaches_the_smallest_logits(dt, V):
    """Flat rows and top-p near one: the border lies among the smallest logits,
    below what the histogram's scale was taken from."""
    R = 8
    z = logits(R, V, dt, 3.0, seed=V + 1)
    T = np.array([1.0, 7.5, 17.0, 23.0, 42.0, 45.0, 70.0, 1000.0])
    u = np.linspace(0.01, 0.99, R)
    for p in (0.98, 0.999, 0.99999):
        check(z, u, T, None, np.full(R, p))
        check(z, u, T, None, np.full(R, p), np.full(R, 1e-7))


def test_rows_larger_than_shared_memory():
    V = 2_000_003
    z = logits(2, V, "f32", 2.0, seed=9)
    u = np.array([0.25, 0.9])
    check(z, u)
    check(z, u, None, np.array([50, V - 3]), np.array([0.9, 0.999]))
    check(z, u, None, None, np.array([0.5, 0.95]), np.array([1e-4, 0.0]))


def test_a_border_far_below_the_maximum():
    """Top-k keeps elements that lie beyond the histogram's reach."""
    V = 6000
    z = logits(3, V, "f32", 1.0, seed=10)
    z[:, :3000] -= 200.0
    u, k = np.array([0.1, 0.5, 0.9]), np.array([3001, 4000, V - 1])
    zc = z.cpu().numpy()
    tok, probs = sv.warp_sample(z, torch.as_tensor(u).cuda(), top_k=torch.as_tensor(k, dtype=torch.int32).cuda(), probs=True)
    for r in range(3):
        want, _, t = warp_row(zc[r], 1.0, int(k[r]), u=float(u[r]))
        assert int(tok[r]) == t
        assert np.all(np.abs(probs[r].cpu().numpy() - want) <= PROB_TOL * want + 1e-29)
    check(z, u, np.full(3, 30.0), k, np.array([0.999, 1.0, 0.5]))


@pytest.mark.parametrize("filters", [False, True])
def test_temperatures_at_their_limits(filters):
    V = 4000
    z = logits(6, V, "f32", seed=11)
    T = torch.tensor([1e-36, 1e36, 0.9e-36, 1.1e36, float("nan"), -1.0], device="cuda")
    u = torch.full((6,), 0.6, dtype=torch.float64, device="cuda")
    p = torch.full((6,), 0.9, device="cuda") if filters else None
    ws = sv.CacheWorkspace()
    tok, probs = sv.warp_sample(z, u, temperature=T, top_p=p, probs=True, ws=ws)
    assert ws.status() == sv.STATUS_BAD_VALUE
    assert tok[2:].tolist() == [-1] * 4 and not bool(probs[2:].any())
    assert int(tok[0]) == int(z[0].argmax()) and float(probs[0].max()) == 1.0
    want, kept, t = warp_row(z[1].cpu().numpy(), float(T[1]), 0, float(p[1]) if filters else 1.0, 0.0, 0.6)
    assert int(tok[1]) == t and np.array_equal(probs[1].cpu().numpy() > 0, kept)
    assert np.all(np.abs(probs[1].cpu().numpy() - want) <= PROB_TOL * want)


def test_bindings_refuse_what_does_not_fit():
    z = logits(2, 100, "f32")
    u = torch.rand(2, dtype=torch.float64, device="cuda")
    E = sv.SpecVerifyError
    for bad in (lambda: sv.warp_sample(z), lambda: sv.warp_sample(z.cpu(), u),
                lambda: sv.warp_sample(z.double(), u), lambda: sv.warp_sample(z, u.float()),
                lambda: sv.warp_sample(z, u[:1]), lambda: sv.warp_sample(z.t(), u),
                lambda: sv.warp_sample(z, u, temperature=u),
                lambda: sv.warp_sample(z, u, top_k=torch.ones(2, device="cuda")),
                lambda: sv.warp_sample(z, token_out=torch.zeros(2, dtype=torch.int32, device="cuda")),
                lambda: sv.warp_sample(z, u, probs_out=torch.zeros(2, 99, device="cuda"))):
        with pytest.raises(E):
            bad()
