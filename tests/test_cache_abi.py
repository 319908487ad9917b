"""Host-side refusals of the paged-cache and warp calls (no GPU needed: every
call fails its checks, or is a no-op, before any CUDA work)."""
import ctypes
import struct

import pytest

import speculative_decoding_verification_08_gb300 as sv


@pytest.fixture(scope="module")
def lib():
    sv.build()
    return sv.load()


def cache(**kw):
    a = dict(k=1 << 20, v=1 << 21, k_stride=(64 * 8, 64, 64 * 16), v_stride=(64 * 8, 64, 64 * 16),
             num_pages=4, page_size=16, kv_heads=2, head_dim=64, dtype=1, B=2, tokens=3, max_pages=2,
             pages=4096, pages_stride=2, q_start=4096, kv_len=4096)
    a.update(kw)
    flat = []
    for x in a.values():
        flat.extend(x if isinstance(x, tuple) else (x,))
    return struct.pack("@QQ3q3q8iQqQQ", *flat)         # sv_paged_cache


S2 = struct.pack("@2q", 128, 64)
WS, BIG = 1 << 20, 1 << 30


def attend(lib, c, q=4096, qs=S2, o=8192, os=S2, heads=4, scale=0.125, window=0, ws=WS, n=BIG):
    return lib.sv_paged_attention(c, q, qs, o, os, heads, ctypes.c_float(scale), window, ws, n, None)


def append(lib, c, k=4096, ks=S2, v=4096, vs=S2, q=4096, qs=S2, o=4096, os=S2, heads=4, f=4096,
           rot=64, ws=WS, n=BIG):
    return lib.sv_append_kv(c, k, ks, v, vs, q, qs, o, os, heads, f, rot, 0, None, ws, n, None)


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(tokens=-1), dict(kv_heads=0), dict(head_dim=0), dict(head_dim=12),
    dict(head_dim=136), dict(page_size=0), dict(page_size=12), dict(num_pages=0), dict(max_pages=0),
    dict(dtype=0), dict(dtype=3), dict(max_pages=1 << 28), dict(k=0), dict(v=0), dict(pages=0),
    dict(q_start=0), dict(kv_len=0), dict(pages_stride=1), dict(k=(1 << 20) + 8),
    dict(k_stride=(1, 64, 64)), dict(v_stride=(64, -64, 64))])
def test_bad_caches_are_refused(lib, kw):
    assert attend(lib, cache(**kw)) == sv.SV_EINVAL
    assert append(lib, cache(**kw)) == sv.SV_EINVAL


def test_bad_calls_are_refused(lib):
    assert attend(lib, None) == sv.SV_EINVAL and append(lib, None) == sv.SV_EINVAL
    for kw in (dict(heads=0), dict(heads=3), dict(scale=float("nan")), dict(scale=float("inf")),
               dict(window=-1)):
        assert attend(lib, cache(), **kw) == sv.SV_EINVAL, kw
    for kw in (dict(rot=-4), dict(rot=68), dict(rot=6), dict(f=None), dict(heads=-1), dict(q=None),
               dict(heads=0)):
        assert append(lib, cache(), **kw) == sv.SV_EINVAL, kw
    for kw in (dict(ws=None), dict(ws=WS + 8), dict(n=255)):
        assert attend(lib, cache(), **kw) == sv.SV_EWORKSPACE, kw
        assert append(lib, cache(), **kw) == sv.SV_EWORKSPACE, kw


def test_empty_batches_do_nothing(lib):
    for kw in (dict(B=0), dict(tokens=0)):
        c = cache(**kw)
        assert attend(lib, c, q=None, o=None, ws=None, n=0) == 0
        assert append(lib, c, k=None, v=None, ws=None, n=0) == 0


def test_warp_refusals(lib):
    def warp(z=4096, zs=100, dt=0, R=2, V=100, u=4096, tok=4096, probs=4096, ps=100, ws=WS, n=BIG):
        return lib.sv_warp_sample(z, zs, dt, R, V, None, None, None, None, u, tok, probs, ps, ws, n,
                                  None)
    for kw in (dict(z=None), dict(zs=99), dict(dt=3), dict(dt=-1), dict(R=-1), dict(V=0),
               dict(V=1 << 31), dict(u=None), dict(tok=None, probs=None), dict(ps=99)):
        assert warp(**kw) == sv.SV_EINVAL, kw
    for kw in (dict(ws=None), dict(ws=WS + 16), dict(n=128)):
        assert warp(**kw) == sv.SV_EWORKSPACE, kw
    assert warp(R=0, z=None, ws=None) == 0


def test_status_words(lib):
    assert "page" in sv.status_string(sv.STATUS_BAD_PAGE)
    assert "length" in sv.status_string(sv.STATUS_BAD_LENGTH)
    assert lib.sv_cache_workspace_size() % 256 == 0


def test_bindings_refuse_without_a_gpu(lib):
    """What is no CUDA tensor is refused before any CUDA work."""
    import torch
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    c = torch.zeros(2, 8, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    for bad in (lambda: sv.append_kv(x, x, c, c, i, i, i), lambda: sv.paged_attention(x, c, c, i, i, i),
                lambda: sv.warp_sample(torch.zeros(2, 8)),
                lambda: sv._native().append_kv(x, x, c, c, i, i, i, *[None] * 4, False, 0, 0, 0),
                lambda: sv._native().paged_attention(x, c, c, i, i, i, None, 0, None, 0, 0, 0),
                lambda: sv._native().warp_sample(*[None] * 12), lambda: sv._native().append_kv(x)):
        with pytest.raises(sv.SpecVerifyError):
            bad()
