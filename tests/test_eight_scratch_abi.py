"""Sizes of the room that sequences of an 8-bit cache are read back to (no GPU needed)."""
import ctypes

import pytest

import speculative_decoding_verification_08_gb300 as sv
from test_eight_abi import S2, cache, scales


@pytest.fixture(scope="module")
def lib():
    sv.build()
    return sv.load()


def batch(**kw):
    kw = {**dict(B=2, tokens=1000), **kw}
    return cache(pages_stride=kw.get("max_pages", 2), **kw)


def size(lib, heads=4, **kw):
    return lib.sv_paged_attention_scratch_size(batch(**kw), heads)


def test_no_more_than_the_cache_in_sixteen_bits(lib):
    # 2 kv heads of 64, pages of 16 slots, two caches, two bytes a value
    page = 2 * 64 * 16 * 2 * 2
    for wide in (3, 50, 100000):
        assert size(lib, num_pages=4, max_pages=wide) == 4 * page
    # a table of fewer entries than the cache has pages: as many, and a table of their own
    for pool in (5, 1 << 30):
        assert 4 * page < size(lib, num_pages=pool) <= 4 * page + 256


def test_tables_that_reading_back_does_not_look_through(lib):
    # 16 GiB in 16 bits: 2^34 / 512 bytes a slot, 16 slots a page, 2 sequences
    assert size(lib, max_pages=1 << 20) > 0 and size(lib, max_pages=(1 << 20) + 1) == 0
    big = dict(max_pages=1 << 20, page_size=1 << 10, B=1 << 30, tokens=(1 << 31) - 1024)
    assert size(lib, heads=1 << 10, kv_heads=1 << 10, head_dim=128, **big) == 0      # (past 64 bits)
    assert size(lib, heads=2 << 16, kv_heads=1 << 16, max_pages=1) > 0
    assert size(lib, heads=2 << 17, kv_heads=1 << 17, max_pages=1) == 0


def test_scratch_is_refused_where_its_size_is_none(lib):
    def call(scratch, **kw):
        return lib.sv_paged_attention_scaled(batch(**kw), scales(), 1, 4096, S2, 8192, S2, kw.get("kv_heads", 2),
                                             ctypes.c_float(1), 0, scratch, 1 << 40, None, 0, None)
    for scratch in (None, 1 << 20):
        assert call(scratch) == sv.SV_EWORKSPACE        # (looked at after these)
        for kw in (dict(kv_heads=1 << 17, max_pages=1), dict(max_pages=(1 << 20) + 1)):
            assert call(scratch, **kw) == (sv.SV_EINVAL if scratch else sv.SV_EWORKSPACE)
