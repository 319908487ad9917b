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
