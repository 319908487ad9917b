"""Host-side refusals of the calls on 8-bit caches and with norms (no GPU needed:
every call fails its checks, or is a no-op, before any CUDA work)."""
import ctypes
import struct

import pytest
import torch

import speculative_decoding_verification_08_gb300 as sv
from speculative_decoding_verification_08_gb300.paged import PagedCache

S2 = struct.pack("@2q", 128, 64)
WS, BIG = 1 << 20, 1 << 30
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    sv.build()
    return sv.load()


def flat(a):
    return [x for v in a.values() for x in (v if isinstance(v, tuple) else (v,))]


def cache(**kw):
    a = dict(k=1 << 20, v=1 << 21, k_stride=(64 * 8, 64, 64 * 16), v_stride=(64 * 8, 64, 64 * 16),
             num_pages=4, page_size=16, kv_heads=2, head_dim=64, dtype=3, B=2, tokens=3, max_pages=2,
             pages=4096, pages_stride=2, q_start=4096, kv_len=4096)
    a.update(kw)
    return struct.pack("@QQ3q3q8iQqQQ", *flat(a))      # sv_paged_cache


def scales(**kw):
    a = dict(k=1 << 22, v=1 << 23, k_stride=(32, 2, 1), v_stride=(32, 2, 1))
    a.update(kw)
    return struct.pack("@QQ3q3q", *flat(a))            # sv_cache_scales


def attend(lib, c, s=scales(), dt=1, q=4096, o=8192, heads=4, scale=0.125, window=0, ws=WS, n=BIG):
    return lib.sv_paged_attention_scaled(c, s, dt, q, S2, o, S2, heads, ctypes.c_float(scale), window, None, 0, ws, n,
                                         None)


def append(lib, c, s=scales(), dt=1, k=4096, v=4096, q=4096, o=4096, heads=4, qn=4096, kn=4096, nt=0, eps=1e-6,
           f=4096, rot=64, ws=WS, n=BIG):
    return lib.sv_append_kv_normed(c, s, dt, k, S2, v, S2, q, S2, o, S2, heads, qn, kn, nt, ctypes.c_float(eps), f, rot,
                                   0, None, ws, n, None)


def read(lib, c, s=scales(), dt=1, k=4096, v=4096, ks=S2, ws=WS, n=BIG):
    return lib.sv_read_kv(c, s, dt, k, ks, v, S2, ws, n, None)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(tokens=-1), dict(kv_heads=0), dict(head_dim=8), dict(head_dim=24), dict(head_dim=144),
    dict(page_size=0), dict(page_size=12), dict(num_pages=0), dict(max_pages=0), dict(dtype=0), dict(dtype=1),
    dict(dtype=4), dict(max_pages=1 << 28), dict(k=0), dict(v=0), dict(pages=0), dict(q_start=0), dict(kv_len=0),
    dict(pages_stride=1), dict(k=(1 << 20) + 8), dict(k_stride=(8, 64, 64)), dict(v_stride=(64, -64, 64))])
def test_bad_caches_are_refused(lib, kw):
    for call in (attend, append, read):
        assert call(lib, cache(**kw)) == sv.SV_EINVAL, call


@pytest.mark.parametrize("kw", [dict(k=0), dict(v=0), dict(k_stride=(-32, 2, 1)), dict(v_stride=(32, -2, 1))])
def test_bad_scales_are_refused(lib, kw):
    for call in (attend, append, read):
        assert call(lib, cache(), scales(**kw)) == sv.SV_EINVAL, call


def test_scales_that_vectors_share_are_not_written(lib):
    assert append(lib, cache(), scales(k_stride=(32, 2, 0))) == sv.SV_EINVAL
    assert append(lib, cache(), scales(v_stride=(0, 2, 1))) == sv.SV_EINVAL


def test_bad_calls_are_refused(lib):
    for dt in (0, 3, 4, -1):
        for call in (attend, append, read):
            assert call(lib, cache(), dt=dt) == sv.SV_EINVAL
    for call in (attend, append, read):
        assert call(lib, None) == sv.SV_EINVAL
        for kw in (dict(ws=None), dict(ws=WS + 8), dict(n=255)):
            assert call(lib, cache(), **kw) == sv.SV_EWORKSPACE, (call, kw)
    assert attend(lib, cache(), None) == sv.SV_EINVAL
    for kw in (dict(heads=0), dict(heads=3), dict(scale=NAN), dict(scale=INF), dict(window=-1), dict(q=None),
               dict(o=None), dict(q=4104)):
        assert attend(lib, cache(), **kw) == sv.SV_EINVAL, kw
    for kw in (dict(rot=-4), dict(rot=68), dict(rot=6), dict(f=None), dict(heads=-1), dict(q=None), dict(heads=0),
               dict(nt=2), dict(nt=3), dict(eps=NAN), dict(eps=-1e-6), dict(eps=INF), dict(k=None), dict(o=None),
               dict(v=4100)):
        assert append(lib, cache(), **kw) == sv.SV_EINVAL, kw
    # a norm of queries that there are none of
    assert append(lib, cache(), q=None, heads=0) == sv.SV_EINVAL
    for kw in (dict(k=None), dict(v=None), dict(ks=struct.pack("@2q", 127, 64)), dict(k=4104)):
        assert read(lib, cache(), **kw) == sv.SV_EINVAL, kw


def test_sixteen_bit_caches_take_tokens_of_their_type(lib):
    for call in (append, read):
        assert call(lib, cache(dtype=1), None, dt=2) == sv.SV_EINVAL
        assert call(lib, cache(dtype=2), None, dt=2, ws=None) == sv.SV_EWORKSPACE
        assert call(lib, cache(), None) == sv.SV_EINVAL


def test_empty_batches_do_nothing(lib):
    for kw in (dict(B=0), dict(tokens=0)):
        c = cache(**kw)
        assert attend(lib, c, q=None, o=None, ws=None, n=0) == 0
        assert append(lib, c, k=None, v=None, ws=None, n=0) == 0
        assert read(lib, c, k=None, v=None, ws=None, n=0) == 0
        assert lib.sv_paged_attention_scratch_size(c, 4) == 0


def test_scratch_sizes(lib):
    def size(heads=4, **kw):
        return lib.sv_paged_attention_scratch_size(cache(**kw), heads)
    # 2 query heads to a kv head: up to 128 rows of a sequence go without
    assert size(B=2, tokens=128) == 0 and size(B=2, tokens=129) > 0
    assert size(heads=2, B=2, tokens=256) == 0 and size(heads=2, B=2, tokens=257) > 0
    slots = 2 * 2 * 16
    assert size(B=2, tokens=1000) >= 2 * slots * 2 * 64 * 2 + 4 * 4 and size(B=2, tokens=1000) % 256 == 0
    assert size(B=2, tokens=1000, max_pages=1 << 24) == 0          # more than a GPU should be asked for
    assert size(heads=3, B=2, tokens=1000) == 0 and size(heads=0, B=2, tokens=1000) == 0


def test_bindings_refuse_without_a_gpu(lib):
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(2, 8, 1, 64, dtype=torch.float8_e4m3fn), torch.zeros(2, 8, 1, dtype=torch.uint8)
    s, i = s.view(torch.float8_e8m0fnu), torch.zeros(1, 1, dtype=torch.int32)
    for bad in (lambda: sv.append_kv(x, x, c, c, i, i, i, k_scale=s, v_scale=s),
                lambda: sv.append_kv(x, x, x, x, i, i, i, k_norm=x),
                lambda: sv.paged_attention(x, c, c, i, i, i, k_scale=s, v_scale=s),
                lambda: sv.read_kv(c, c, i, i, i, rows=1, k_scale=s, v_scale=s),
                lambda: sv.read_kv(c, c, i, i, i, rows=1, dtype=torch.float32, k_scale=s, v_scale=s),
                lambda: sv._native().append_kv_normed(x, x, c, c, i, i, i, *[None] * 4, False, None, None, 1e-6, s, s,
                                                      0, 0, 0),
                lambda: sv._native().read_kv(c, c, i, i, i, 1, 1, s, s, None, None, 0, 0, 0),
                lambda: sv._native().read_kv(c, c, i, i, i, -1, 1, s, s, None, None, 0, 0, 0),
                lambda: sv._native().paged_attention_scaled(x, c, c, i, i, i, None, 0, None, s, s, 0, 0, 0),
                lambda: sv._native().read_kv(c)):
        with pytest.raises(sv.SpecVerifyError):
            bad()


def test_a_paged_cache_of_eight_bits_has_scales():
    c = PagedCache(2, 6, 8, 3, 16, dtype=torch.float8_e4m3fn, device="cpu")
    assert c.k.dtype == torch.float8_e4m3fn and c.k_scale.dtype == torch.float8_e8m0fnu
    assert tuple(c.k_scale[0].shape) == tuple(c.k[0].shape[:3]) == (6, 8, 3)
    assert set(c._scales(1)) == {"k_scale", "v_scale"}
    assert PagedCache(2, 6, 8, 3, 16, device="cpu")._scales(0) == {}
    with pytest.raises(ValueError):
        c.read(0, ["nobody"])


@pytest.mark.parametrize("dt,parts,exact", [(torch.bfloat16, 3, 23), (torch.float16, 4, 20)])
def test_queries_are_sums_of_e5m2_numbers(dt, parts, exact):
    """What the attention's split of queries relies on: every value is the sum of so
    many e5m2 numbers, exactly down to 2^-exact of the largest, to 2^-31 of it below."""
    x = torch.arange(0, 1 << 16, dtype=torch.int32).to(torch.int16).view(dt).float()
    x = x[torch.isfinite(x)]
    for top in (1.0, 1.75, 1.7578125, 1.99, 3.0, 57344.0):
        top = torch.tensor(top).to(dt).float()
        m, e = torch.frexp(top)
        unit = 2.0 ** (int(e) - 16 + (1 if float(m) > 0.875 else 0))   # brings it to 57344 or less
        y = (x[x.abs() <= top] / unit).double()
        rest = y.clone()
        for _ in range(parts):
            rest = rest - rest.float().to(torch.float8_e5m2).double()
        largest = float(top) / unit
        assert 28672 < largest <= 57344
        assert bool((rest[y.abs() >= largest * 2.0 ** -exact] == 0).all())
        assert float(rest.abs().max()) <= largest * 2.0 ** -31
