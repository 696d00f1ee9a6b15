"""Host checks of the scaled rotation, paged cache and token log probability calls (CPU only: fake
aligned pointers, never dereferenced), and pins of the tests' 64-bit forms."""

import ctypes
import math

import numpy as np
import pytest
import torch

import ref64_serving as ref

P = 0x30000
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from kv_cached_decode_gb300 import build, load_library

    build.build()
    return load_library()


def spec(**kw):
    from kv_cached_decode_gb300 import RopeSpec

    c = dict(base=1e4, rot_dim=64, interleaved=0, scaling=0, factor=1.0, low=1.0, high=4.0,
             original_len=100, magnitude=1.0)
    c.update(kw)
    return ctypes.byref(RopeSpec(**c))


BAD_SPECS = [dict(base=0.0), dict(base=-1.0), dict(base=NAN), dict(base=INF), dict(magnitude=NAN),
             dict(magnitude=INF), dict(interleaved=2), dict(interleaved=-1), dict(scaling=4),
             dict(scaling=-1), dict(scaling=1, factor=0.0), dict(scaling=1, factor=NAN),
             dict(scaling=2, factor=INF), dict(scaling=2, low=0.0), dict(scaling=2, high=1.0),
             dict(scaling=3, high=NAN), dict(scaling=3, high=INF), dict(scaling=3, low=NAN),
             dict(scaling=2, original_len=0), dict(scaling=3, base=1.0)]


def rows(**kw):
    from kv_cached_decode_gb300 import HeadRows

    c = dict(x=P, stride_b=640, stride_h=64, stride_t=640, weight=0, out=0x50000, n_heads=10)
    c.update(kw)
    return ctypes.byref(HeadRows(**c))


def test_rope_scaled_refusals(lib):
    def call(q=None, k=None, dtype=0, batch=1, n=4, pos0=None, positions=None, s=None):
        return lib.kvd_rope_scaled(dtype, batch, n, rows() if q is None else q, k, pos0, positions,
                                   spec() if s is None else s, 0, None, None)

    for kw in (dict(x=0), dict(out=0), dict(n_heads=0), dict(x=P + 8), dict(out=P + 2),
               dict(weight=P), dict(stride_t=60), dict(stride_h=-64), dict(stride_b=4),
               dict(out=P)):
        assert call(rows(**kw)) == 1, kw
        assert call(k=rows(**kw)) == 1, kw
    for kw in (dict(dtype=2), dict(batch=-1), dict(n=-1), dict(pos0=P, positions=P)):
        assert call(**kw) == 1, kw
    for kw in BAD_SPECS:
        assert call(s=spec(**kw), batch=0) == 1, kw
    for rot in (0, 8, 24, 80, -16):
        assert call(s=spec(rot_dim=rot), batch=0) == 2
    assert lib.kvd_rope_scaled(0, 0, 4, rows(), None, None, None, None, 0, None, None) == 1
    for good in (dict(), dict(rot_dim=16, interleaved=1), dict(scaling=1, factor=3.0),
                 dict(scaling=2), dict(scaling=3, high=32.0), dict(factor=NAN, low=NAN)):
        assert call(s=spec(**good), batch=0) == 0 and call(s=spec(**good), n=0) == 0
    assert lib.kvd_rope_scaled(0, 1, 4, None, None, None, None, spec(), 0, None, None) == 0
    assert call(batch=1 << 30, n=1 << 30) == 2


def cache(**kw):
    from kv_cached_decode_gb300 import PagedCache

    c = dict(k=0x10000, v=0x20000, stride_p=8 * 16 * 64, stride_h=16 * 64, stride_t=64, n_pages=50,
             n_kv_heads=8, head_dim=64, page_size=16, table=0x8004, table_stride=20, table_width=20,
             batch=3)
    c.update(kw)
    return ctypes.byref(PagedCache(**c))


def token_rows(**kw):
    from kv_cached_decode_gb300 import TokenRows

    c = dict(x=P, stride_t=640, stride_h=64, out=0, n_heads=8)
    c.update(kw)
    return ctypes.byref(TokenRows(**c))


BAD_CACHES = [dict(k=0), dict(v=0), dict(table=0), dict(k=0x10008), dict(v=0x20002),
              dict(table=0x8002), dict(n_pages=0), dict(n_kv_heads=0), dict(batch=0),
              dict(table_width=0), dict(table_stride=19), dict(stride_p=0), dict(stride_h=63),
              dict(stride_t=32), dict(stride_p=8 * 16 * 64 + 4), dict(stride_h=-64),
              dict(page_size=0), dict(page_size=-16)]
ODD_CACHES = [dict(head_dim=128), dict(page_size=4), dict(page_size=24), dict(page_size=1 << 17),
              dict(table_width=1 << 27, table_stride=1 << 27), dict(stride_p=1 << 40)]
BAD_ROWS = [dict(x=0), dict(x=P + 8), dict(n_heads=0), dict(stride_t=-640), dict(stride_h=4)]


def test_paged_append_refusals(lib):
    def call(c=None, dtype=0, n=4, k=None, v=None, q=None, starts=P, lens=P, lens_out=None, s=None):
        return lib.kvd_paged_append(dtype, c or cache(), n, k or token_rows(), v or token_rows(), q,
                                    starts, lens, lens_out, s, 0, None, None)

    for kw in BAD_CACHES:
        assert call(cache(**kw)) == 1, kw
    for kw in ODD_CACHES:
        assert call(cache(**kw)) == 2, kw
    for kw in BAD_ROWS + [dict(n_heads=7), dict(out=0x50000)]:
        assert call(k=token_rows(**kw)) == 1 and call(v=token_rows(**kw)) == 1, kw
    for kw in BAD_ROWS + [dict(out=0), dict(out=0x50008), dict(out=P)]:
        assert call(q=token_rows(**{"out": 0x50000, **kw})) == 1, kw
    for kw in (dict(dtype=2), dict(n=-1), dict(starts=None), dict(lens=None),
               dict(lens=P, lens_out=P), dict(s=spec(base=0.0))):
        assert call(**kw) == 1, kw
    assert call(s=spec(rot_dim=8)) == 2
    assert lib.kvd_paged_append(0, None, 4, token_rows(), token_rows(), None, P, P, None, None, 0,
                                None, None) == 1
    assert lib.kvd_paged_append(0, cache(), 4, token_rows(), None, None, P, P, None, None, 0, None,
                                None) == 1


def test_paged_attn_refusals(lib):
    from kv_cached_decode_gb300 import KVD_OP_PAGED_ATTN, kvd_workspace_size

    def call(c=None, dtype=0, n=4, most=4, q=None, starts=P, lens=P, scale=0.125, ws=0x100000,
             size=1 << 30):
        return lib.kvd_paged_attn(dtype, c or cache(), n, most,
                                  q or token_rows(out=0x50000, n_heads=16), starts, lens, scale, ws,
                                  size, 0, None, None)

    for kw in BAD_CACHES:
        assert call(cache(**kw)) == 1, kw
    for kw in ODD_CACHES:
        assert call(cache(**kw)) == 2, kw
    for kw in BAD_ROWS + [dict(out=0), dict(out=0x50008), dict(out=P), dict(n_heads=9)]:
        assert call(q=token_rows(**{"out": 0x50000, **kw})) == 1, kw
    for kw in (dict(dtype=2), dict(n=-1), dict(most=0), dict(starts=None), dict(lens=None),
               dict(scale=NAN), dict(scale=INF), dict(scale=-INF)):
        assert call(**kw) == 1, kw
    assert call(q=token_rows(out=0x50000, n_heads=8 * 129)) == 2
    assert call(n=0) == 0
    need = kvd_workspace_size(KVD_OP_PAGED_ATTN, 3, 16, 8, 1, 4)
    for kw in (dict(ws=None), dict(ws=0x100010), dict(size=need - 1)):
        assert call(**kw) == 3, kw
    sizes = [kvd_workspace_size(KVD_OP_PAGED_ATTN, 1, 16, 8, 1, n) for n in (1, 2, 7, 64, 65, 9999)]
    assert sizes == sorted(sizes) and sizes[3] == sizes[5] > sizes[2] > 65536
    for bad in (dict(n_q_heads=9, n_kv_heads=8), dict(n_q_heads=129), dict(n_q_heads=0),
                dict(qlen=0)):
        assert kvd_workspace_size(KVD_OP_PAGED_ATTN, 1, **bad) == 0, bad


def test_token_logprobs_refusals(lib):
    def call(dtype=2, x=P, stride=1000, rows=2, vocab=1000, tokens=P, given=1, top=5):
        return lib.kvd_token_logprobs(dtype, x, stride, rows, vocab, None, tokens, given, P, P, P,
                                      P, top, P, P, 0, None, None)

    for kw in (dict(dtype=3), dict(dtype=-1), dict(x=0), dict(x=P + 2), dict(dtype=0, x=P + 1),
               dict(stride=999), dict(vocab=0), dict(rows=-1), dict(tokens=None), dict(given=-1),
               dict(top=-1)):
        assert call(**kw) == 1, kw
    for kw in (dict(given=17), dict(top=33), dict(vocab=524289, stride=524289), dict(rows=1 << 28)):
        assert call(**kw) == 2, kw
    assert call(rows=0) == 0


def test_other_calls_refuse_32_bit_types(lib):
    from kv_cached_decode_gb300 import Cache

    c = Cache(k=0x10000, v=0x20000, stride_b=8 * 512 * 64, stride_h=512 * 64, stride_t=64, batch=2,
              n_kv_heads=8, head_dim=64, capacity=512)
    assert lib.kvd_kv_append(2, ctypes.byref(c), 1, 1, P, P, P, None, 0, None, None) == 1
    assert lib.kvd_decode_attn(2, 1, 8, P, ctypes.byref(c), None, 100, None, 1, 0.125, 0x60000,
                               None, 0, 0, None, None) == 1


def test_binding_refuses_host_and_misshapen_tensors():
    import kv_cached_decode_gb300 as kvd

    x = torch.zeros(2, 3, 4, 64, dtype=torch.float16)
    t = torch.zeros(5, 3, 64, dtype=torch.float16)
    for f in (lambda: kvd.kvd_rope_scaled(x, q_out=x, rope=kvd.make_rope()),
              lambda: kvd.kvd_rope_scaled(rope=kvd.make_rope()),
              lambda: kvd.make_rope(scaling="other"),
              lambda: kvd.make_paged_cache(x, x, torch.zeros(1, 1, dtype=torch.int32)),
              lambda: kvd.make_paged_cache(x, x[:1], torch.zeros(1, 1, dtype=torch.int32)),
              lambda: kvd.make_paged_cache(x, x, torch.zeros(3, dtype=torch.int32)),
              lambda: kvd.kvd_paged_attn(t, None, t, None, None, None),
              lambda: kvd.kvd_token_logprobs(torch.zeros(2, 5)),
              lambda: kvd.kvd_token_logprobs(torch.zeros(5))):
        with pytest.raises((ValueError, AttributeError)):
            f()
    with pytest.raises(TypeError):
        kvd.make_paged_cache(x, x, torch.zeros(1, 1))
    with pytest.raises(TypeError):
        kvd.kvd_token_logprobs(torch.zeros(2, 5, dtype=torch.int32))


def test_frequencies():
    plain = ref.theta()
    assert np.allclose(plain, 1e4 ** (-np.arange(32) / 32))
    kw = dict(base=1e4, factor=8.0, original_len=4096, low=1.0, high=4.0)
    for scaling in ("bands", "ramp"):
        t = ref.theta(scaling=scaling, **kw)
        turns = 4096 * plain / (2 * math.pi)
        ratio = plain / t
        assert np.all((ratio >= 1 - 1e-12) & (ratio <= 8 + 1e-12)) and np.all(np.diff(ratio) > -1e-9)
        assert np.allclose(ratio[turns > 16], 1) and np.allclose(ratio[turns < 0.25], 8)
    assert np.allclose(ref.theta(scaling="linear", factor=4.0), plain / 4)


def test_rotation_by_hand():
    x = np.arange(64.0)
    y, _ = ref.rotate(x, np.array(3), dict(rot_dim=16, interleaved=True, base=100.0))
    a = 3 * 100.0 ** (-2 * 5 / 16)
    assert np.isclose(y[10], 10 * math.cos(a) - 11 * math.sin(a))
    assert np.isclose(y[11], 11 * math.cos(a) + 10 * math.sin(a)) and np.array_equal(y[16:], x[16:])
    y, _ = ref.rotate(x, np.array(3), dict(rot_dim=16, base=100.0))
    assert np.isclose(y[5], 5 * math.cos(a) - 13 * math.sin(a))


def test_logprobs_by_hand():
    lp, rank, ent, lse, ids, tlp = ref.logprobs([0.0, 1.0, 1.0, -np.inf], [2, 3, -1], 1.0, 4)
    z = math.log(1 + 2 * math.e)
    assert np.allclose(lp, [1 - z, -np.inf, 0]) and rank == [1, 3, -1] and ids == [1, 2, 0, -1]
    p = np.exp(np.array([0, 1, 1]) - z)
    assert np.isclose(ent, -(p * np.log(p)).sum()) and np.isclose(lse, z)
    assert np.allclose(tlp, [1 - z, 1 - z, -z, -np.inf])


def test_chunk_attention_by_hand():
    q, k = torch.zeros(2, 1, 64, dtype=torch.float64), torch.zeros(1, 3, 64, dtype=torch.float64)
    v = torch.arange(3.0, dtype=torch.float64)[None, :, None].expand(1, 3, 64)
    out = ref.chunk_attention(q, k, v, 0.125)[0]
    assert torch.allclose(out[0], torch.full((1, 64), 0.5, dtype=torch.float64))
    assert torch.allclose(out[1], torch.ones(1, 64, dtype=torch.float64))
