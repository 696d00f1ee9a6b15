"""The largest calls of the paged attention that its list of tiles can count (CPU only: fake
pointers, never dereferenced)."""

import ctypes

import pytest
import torch

P = 0x30000
UNSUPPORTED = 2


@pytest.fixture(scope="module")
def lib():
    from kv_cached_decode_gb300 import build, load_library

    build.build()
    return load_library()


def call(lib, batch, n_tokens, hk, hq, width, page=65536):
    from kv_cached_decode_gb300 import PagedCache, TokenRows

    c = PagedCache(P, P, page * 64 * hk, page * 64, 64, 1000, hk, 64, page, P, width, width, batch)
    q = TokenRows(P, hq * 64, 64, 0x50000, hq)
    return lib.kvd_paged_attn(0, ctypes.byref(c), n_tokens, n_tokens, ctypes.byref(q), P, P, 0.125,
                              0x100000, 1 << 40, 0, None, None)


# units of a row: tokens * (query heads per KV head) / 128 and one more, for each KV head; at their
# longest width * page / 128 tiles of weight 5, and 20 for the unit; below 4e9 in all
@pytest.mark.skipif(torch.cuda.is_available(), reason="the calls that pass would be launched")
@pytest.mark.parametrize("batch,n_tokens,hk,hq,width,fits", [
    (90, 1, 1, 1, 16384, True), (100, 1, 1, 1, 16384, False),
    (1000, 8000, 8, 64, 1024, False), (1000, 8000, 8, 64, 16, True),
    (1, 1 << 20, 1, 128, 16, False), (1, 1 << 16, 1, 128, 16, True),
    (1 << 20, 1 << 20, 1, 1, 1, True), (1 << 20, 1 << 20, 2, 2, 1, False)])
def test_calls_that_the_list_can_count(lib, batch, n_tokens, hk, hq, width, fits):
    got = call(lib, batch, n_tokens, hk, hq, width)
    assert (got != UNSUPPORTED) == fits, got
