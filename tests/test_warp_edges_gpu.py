"""warp_sample at exact ties and at the smallest temperatures, against its
64-bit definition."""
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


def check(z, u, T=1.0, p=1.0, m=0.0, filtered=True):
    """Every row of z under one setting of the filters against the definition."""
    R = z.shape[0]
    full = lambda x: torch.full((R,), x, dtype=torch.float32, device="cuda")  # noqa: E731
    ws = sv.CacheWorkspace()
    kw = dict(top_p=full(p), min_p=full(m)) if filtered else {}
    tok, probs = sv.warp_sample(z, torch.as_tensor(u, dtype=torch.float64).cuda(), temperature=full(T),
                                probs=True, ws=ws, **kw)
    assert ws.status() == 0
    zc, f32 = z.float().cpu().numpy(), lambda x: float(np.float32(x))  # noqa: E731
    for r in range(R):
        want, kept, t = warp_row(zc[r], f32(T), 0, f32(p), f32(m), float(u[r]))
        got = probs[r].cpu().numpy()
        assert np.array_equal(got > 0, kept & (want > 1e-29)), (r, int((got > 0).sum()), int(kept.sum()))
        assert int(tok[r]) == t, (r, int(tok[r]), t)
        assert np.all(np.abs(got - want) <= PROB_TOL * want + 1e-29), r


@pytest.mark.parametrize("dt", list(TYPES))
@pytest.mark.parametrize("value", [-3.5, 0.0, 2.75, 5.1, -41.3])
@pytest.mark.parametrize("V", [2, 100, 128, 160, 4096, 40000])
def test_goals_that_fall_on_a_border_between_equal_logits(dt, value, V):
    """Rows of one value (alone, beside masked logits, beside ones too small to
    count): every mass is a whole number, and goals u V and p V fall exactly on a
    border."""
    rows = torch.full((6, V), value)
    rows[1, 1::2] = float("-inf")                     # V / 2 are left
    rows[2, ::2] = float("-inf")
    rows[3, 1::2] = value - 200.0
    u = np.array([0.5, 0.5, 0.25, 0.5, 0.0, 0.75])
    for T in (1.0, 0.7, 1.9):
        if abs(rows[0, 0].to(TYPES[dt]).float()) > 60 * T:
            continue
        z = rows.to(TYPES[dt]).cuda()
        check(z, u, T, filtered=False)
        for p in (0.5, 0.25, 0.75, 1.0):
            check(z, u, T, p)
        check(z, u, T, 0.5, 0.3)


@pytest.mark.parametrize("T", [1e-32, 1e-33, 1e-34, 1e-35, 1.1e-36])
def test_a_nucleus_at_the_smallest_temperatures(T):
    """Logits as close together as the temperature is small."""
    R, V = 24, 3000
    T = float(np.float32(T))
    z = (torch.randn(R, V, generator=torch.Generator().manual_seed(31), dtype=torch.float64) * (3 * T)).float().cuda()
    u = np.linspace(0.02, 0.98, R)
    for p in (0.3, 0.7, 0.95):
        check(z, u, T, p)


def test_rows_are_not_written_over_their_logits():
    wide = torch.randn(5, 40, device="cuda")
    u = torch.rand(4, dtype=torch.float64, device="cuda")
    for z, out in ((wide[:4], wide[:4]), (wide[:4], wide[1:]), (wide[1:], wide[:4]), (wide[::3], wide[2:4])):
        with pytest.raises(sv.SpecVerifyError, match="overlap"):
            sv.warp_sample(z, u[:z.shape[0]], probs_out=out)
    out = torch.empty(9, 40, device="cuda")
    out[5:] = wide[:4]                                # side by side, in one block of memory
    token, rows = sv.warp_sample(out[5:], u, probs_out=out[1:5])
    same = sv.warp_sample(wide[:4], u, probs=True)
    assert torch.equal(token, same[0]) and torch.equal(rows, same[1])


def test_leading_axes_that_make_no_rows_are_refused():
    z, u = torch.randn(3, 4, 50, device="cuda"), torch.rand(12, dtype=torch.float64, device="cuda")
    for bad in (z.transpose(0, 1), z[:, :3].expand(3, 3, 50), torch.empty(2, 3, 0, device="cuda")):
        with pytest.raises(sv.SpecVerifyError):
            sv.warp_sample(bad, u[:bad.shape[0] * bad.shape[1]])
    token, _ = sv.warp_sample(z[:, :1], u[:3])        # an axis of length one is no axis
    assert token.shape == (3, 1) and torch.equal(token[:, 0], sv.warp_sample(z[:, 0], u[:3])[0])
