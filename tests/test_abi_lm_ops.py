"""Host checks of the head norm, windowed attention, 4-bit cache and filtered sampling calls
(CPU only: fake aligned pointers, never dereferenced), and pins of the tests' 64-bit forms."""

import ctypes

import numpy as np
import pytest
import torch

import ref64

P = 0x30000
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from kv_cached_decode_gb300 import build, load_library

    build.build()
    return load_library()


def _rows(**kw):
    from kv_cached_decode_gb300 import HeadRows

    c = dict(x=P, stride_b=640, stride_h=64, stride_t=640, weight=0, out=0x50000, n_heads=10)
    c.update(kw)
    return ctypes.byref(HeadRows(**c))


def test_qk_norm_rope_refusals(lib):
    f = lib.kvd_qk_norm_rope

    def call(q=None, k=None, dtype=0, batch=1, n=4, eps=1e-6, base=1e4):
        return f(dtype, batch, n, _rows() if q is None else q, k, None, eps, base, 0, None, None)

    for kw in (dict(x=0), dict(out=0), dict(n_heads=0), dict(x=P + 8), dict(out=P + 2),
               dict(weight=P + 4), dict(stride_t=60), dict(stride_h=-64), dict(stride_b=4),
               dict(out=P)):  # in place, but not the output's layout
        assert call(_rows(**kw)) == 1, kw
        assert call(k=_rows(**kw)) == 1, kw
    for kw in (dict(dtype=2), dict(batch=-1), dict(n=-1), dict(eps=-1.0), dict(eps=NAN),
               dict(eps=INF), dict(base=-1.0), dict(base=NAN), dict(base=INF)):
        assert call(**kw) == 1, kw
    assert call(batch=0) == 0 and call(n=0) == 0
    assert f(0, 1, 4, None, None, None, 1e-6, 1e4, 0, None, None) == 0
    assert call(batch=1 << 30, n=1 << 30) == 2  # more warps than a grid holds


def _cache(**kw):
    from kv_cached_decode_gb300 import Cache

    c = dict(k=0x10000, v=0x20000, stride_b=8 * 512 * 64, stride_h=512 * 64, stride_t=64, batch=2,
             n_kv_heads=8, head_dim=64, capacity=512)
    c.update(kw)
    return Cache(**c)


def test_window_attn_refusals(lib):
    from kv_cached_decode_gb300 import NewTokens

    def call(c=None, dtype=0, batch=2, hq=8, qlen=1, q=P, lens=None, fixed=100, app=None, window=64,
             sinks=4, scale=0.125, out=0x60000):
        return lib.kvd_window_attn(dtype, batch, hq, qlen, q, ctypes.byref(c or _cache()), lens,
                                   fixed, app, window, sinks, scale, out, None, 0, 0, None, None)

    for kw in (dict(window=0), dict(window=-5), dict(sinks=-1), dict(hq=9), dict(fixed=513),
               dict(fixed=-1), dict(q=0), dict(out=0), dict(q=P + 8), dict(out=P), dict(dtype=5),
               dict(scale=NAN), dict(batch=3), dict(c=_cache(k=0)),
               dict(app=ctypes.byref(NewTokens(P, P, None)))):  # appended without lengths
        assert call(**kw) == 1, kw
    for qlen in (0, -1, 17):
        assert call(qlen=qlen) == 2
    assert call(c=_cache(head_dim=128)) == 2
    assert call(batch=0) == 0

    def pre(c=None, batch=2, hq=8, n=16, q=P, plens=0x40000, lens_in=None, lens_out=None, window=64,
            sinks=4, rope=0.0, scale=0.125):
        return lib.kvd_prefill_window_attn(0, batch, hq, n, q, ctypes.byref(c or _cache()), P, P,
                                           lens_in, plens, lens_out, window, sinks, scale, rope, P,
                                           0, None, None)

    for kw in (dict(window=0), dict(sinks=-1), dict(hq=9), dict(plens=None), dict(q=P + 8),
               dict(lens_in=P, lens_out=P), dict(rope=-1.0), dict(scale=NAN), dict(n=-1)):
        assert pre(**kw) == 1, kw
    assert pre(batch=0) == 0 and pre(n=0) == 0


def _q4(**kw):
    from kv_cached_decode_gb300 import Q4Cache

    c = dict(k=0x10000, v=0x20000, params=0x8008, stride_b=8 * 512, stride_h=512, batch=2,
             n_kv_heads=8, head_dim=64, capacity=512)
    c.update(kw)
    return Q4Cache(**c)


def test_q4_refusals(lib):
    def append(c=None, dtype=0, batch=2, q=4, k=P, v=P, lens=0x40000, counts=None, lens_out=None):
        return lib.kvd_q4_append(dtype, ctypes.byref(c or _q4()), batch, q, k, v, lens, counts,
                                 lens_out, 0, None, None)

    def dequant(c=None, dtype=0, batch=2, n=4, k=P, v=P):
        return lib.kvd_q4_dequant(dtype, ctypes.byref(c or _q4()), batch, n, k, v, None, 0, None,
                                  None)

    def attn(c=None, dtype=0, batch=2, hq=8, qlen=1, q=P, lens=None, fixed=100, causal=1, window=0,
             sinks=0, scale=0.125, out=0x60000):
        return lib.kvd_q4_attn(dtype, batch, hq, qlen, q, ctypes.byref(c or _q4()), lens, fixed,
                               causal, window, sinks, scale, out, None, 0, 0, None, None)

    for call in (append, dequant, attn):
        for kw in (dict(k=0), dict(v=0), dict(params=0), dict(k=0x10008), dict(v=0x10001),
                   dict(params=0x8004), dict(batch=0), dict(n_kv_heads=0), dict(capacity=0),
                   dict(stride_h=511), dict(stride_b=100), dict(stride_b=-1)):
            assert call(_q4(**kw)) == 1, kw
        assert call(_q4(head_dim=128)) == 2
        assert call(_q4(capacity=(1 << 30) + 1, stride_h=1 << 31, stride_b=1 << 35)) == 2
        assert call(dtype=2) == 1 and call(batch=3) == 1 and call(batch=-1) == 1
        assert call(batch=0) == 0
    for kw in (dict(q=-1), dict(k=0), dict(v=P + 8), dict(lens=P, lens_out=P),
               dict(counts=P, lens_out=P)):
        assert append(**kw) == 1, kw
    assert append(q=0) == 0
    assert dequant(n=-1) == 1 and dequant(k=P + 8) == 1
    assert dequant(n=0) == 0 and dequant(k=0, v=0) == 0
    for kw in (dict(hq=9), dict(q=0), dict(out=0), dict(q=P + 8), dict(out=P), dict(fixed=513),
               dict(fixed=-1), dict(window=-1), dict(sinks=-1), dict(window=3, causal=0),
               dict(scale=NAN), dict(scale=INF)):
        assert attn(**kw) == 1, kw
    for qlen in (0, 17):
        assert attn(qlen=qlen) == 2


def test_sample_filtered_refusals(lib):
    def call(x=P, stride=1000, batch=2, vocab=1000, u=P, token=P):
        return lib.kvd_sample_filtered(x, stride, batch, vocab, None, None, None, None, u, token,
                                       None, None, 0, None, None)

    for kw in (dict(x=0), dict(u=0), dict(token=0), dict(stride=999), dict(vocab=0),
               dict(batch=-1)):
        assert call(**kw) == 1, kw
    assert call(vocab=524289, stride=524289) == 2 and call(batch=65536) == 2
    assert call(batch=0) == 0


def test_workspace_sizes(lib):
    from kv_cached_decode_gb300 import (KVD_OP_Q4_ATTN, KVD_OP_VERIFY_ATTN, KVD_OP_WINDOW_ATTN,
                                        KVD_WS_COUNTER_BYTES, kvd_workspace_size)

    for a in ((1, 20, 20, 1, 5, 448), (1, 1, 1, 1, 1, 65536), (2, 8, 2, 1, 16, 32768)):
        assert kvd_workspace_size(KVD_OP_WINDOW_ATTN, *a) == kvd_workspace_size(
            KVD_OP_VERIFY_ATTN, *a)
    assert kvd_workspace_size(KVD_OP_Q4_ATTN, 1, 32, 8, 1, 1, 8192) == KVD_WS_COUNTER_BYTES
    big = kvd_workspace_size(KVD_OP_Q4_ATTN, 16, 32, 8, 1, 1, 32768)
    # two partials (64 values, a maximum and a sum) per CTA and query vector, 152 SMs x 2 CTAs
    assert big >= KVD_WS_COUNTER_BYTES + 2 * 304 * 4 * 66 * 4
    for bad in ((0, 8, 8, 1, 1, 10), (1, 9, 8, 1, 1, 10), (1, 8, 8, 1, 17, 10), (1, 8, 8, 1, 0, 10),
                (1, 8, 8, 1, 1, -1)):
        assert kvd_workspace_size(KVD_OP_Q4_ATTN, *bad) == 0


def test_the_binding_refuses_before_the_library_is_called(lib):
    import kv_cached_decode_gb300 as kvd

    h = torch.zeros(1, 2, 3, 64, dtype=torch.float16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        kvd.kvd_qk_norm_rope(h, None, h)
    with pytest.raises(ValueError, match="q or k is needed"):
        kvd.kvd_qk_norm_rope()
    with pytest.raises(ValueError, match=r"\[batch, heads, n, 64\]"):
        kvd.kvd_qk_norm_rope(h[0], None, h)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        kvd.kvd_window_attn(h, None, h, None, 5)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        kvd.kvd_prefill_window_attn(h, None, h, h, i, h, 5)
    with pytest.raises(ValueError, match="k_new must be a CUDA tensor"):
        kvd.kvd_q4_append(None, h, h)
    with pytest.raises(ValueError, match="k_out must be a CUDA tensor"):
        kvd.kvd_q4_dequant(None, h, h)
    with pytest.raises(ValueError, match="is needed"):
        kvd.kvd_q4_dequant(None)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        kvd.kvd_q4_attn(h, None, h)
    with pytest.raises(ValueError, match="logits must be a CUDA tensor"):
        kvd.kvd_sample_filtered(torch.zeros(1, 5), torch.zeros(1), i)
    with pytest.raises(TypeError, match="logits must be torch.float32"):
        kvd.kvd_sample_filtered(torch.zeros(1, 5).half(), torch.zeros(1), i)
    u8 = torch.zeros(1, 2, 5, 32, dtype=torch.uint8)
    par = torch.zeros(1, 2, 5, 4, dtype=torch.int16)
    with pytest.raises(ValueError, match="CUDA tensors"):
        kvd.make_q4_cache(u8, u8, par)
    with pytest.raises(TypeError, match="uint8"):
        kvd.make_q4_cache(u8.int(), u8, par)
    with pytest.raises(ValueError, match="params"):
        kvd.make_q4_cache(u8, u8, par[:, :, :4])


# ------------------------------------------------------------------ the 64-bit forms ---
def test_norm_rope_form_is_a_complex_product_of_unit_rows():
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((2, 3, 4, 64)), rng.standard_normal(64)
    pos = np.array([[5], [70000]]) + np.arange(4)
    got, _ = ref64.norm_rope(x, w, pos, 1e-6, 10000.0)
    y = x / np.sqrt((x ** 2).sum(-1, keepdims=True) / 64 + 1e-6) * w
    a = pos[:, None, :, None] * 10000.0 ** (-np.arange(32) / 32)
    z = (y[..., :32] + 1j * y[..., 32:]) * np.exp(1j * a)
    assert np.abs(got - np.concatenate([z.real, z.imag], -1)).max() < 1e-10
    flat, _ = ref64.norm_rope(x, None, pos, 0.0, 0)
    assert np.allclose((flat ** 2).mean(-1), 1)


def test_attention_form_against_torch():
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(*s, 64, generator=g, dtype=torch.float64)
               for s in ((4, 5), (2, 30), (2, 30)))
    see = ref64.visible(30, 5, True, 7, 2)
    out, mag, smax = ref64.attention(q, k, v, see, 0.3)
    mask = torch.from_numpy(see)
    want = torch.nn.functional.scaled_dot_product_attention(
        q, k.repeat_interleave(2, 0), v.repeat_interleave(2, 0), attn_mask=mask, scale=0.3)
    assert (out - want).abs().max() < 1e-12 and (mag >= out.abs() - 1e-12).all()
    # the mask, counted by hand: position 25 + i sees itself, 6 before it, and 0, 1
    assert see.sum(1).tolist() == [9] * 5 and see[0, 19] and not see[0, 18] and see[0, 1]
    assert ref64.visible(3, 5).sum(1).tolist() == [0, 0, 1, 2, 3]


def test_q4_form_on_rows_worked_by_hand():
    x = np.zeros((3, 64), np.float32)
    x[0, :16] = np.arange(16)                    # 0..15: step 1, zero point 0, exact
    x[1] = -3.0                                  # equal values: 15 steps of bf16(0.2)
    x[2, 0], x[2, 1] = -1.5, 6.0                 # range 7.5: step 0.5, zero point 3
    n, step, z = ref64.q4_quantise(x)
    assert step[0] == 1 and z[0] == 0 and np.array_equal(n[0, :16], np.arange(16))
    assert step[1] == np.float32(0.2001953125) and z[1] == 15 and (n[1] == 0).all()
    assert step[2] == 0.5 and z[2] == 3 and n[2, 0] == 0 and n[2, 1] == 15 and n[2, 2] == 3
    val = ref64.q4_values(ref64.q4_pack(n), ref64.q4_params(step, z))
    assert np.array_equal(val[0], x[0]) and np.allclose(val[1], -3.0, rtol=2 ** -9)
    assert np.array_equal(val[2], x[2])
    assert ref64.bf16_round(np.float32(1 + 2 ** -8)) == 1 and ref64.bf16_round(
        np.float32(1 + 3 * 2 ** -8)) == np.float32(1 + 2 ** -6)  # ties to even


def test_sample_form_on_small_rows():
    x = np.log([0.1, 0.4, 0.2, 0.3])
    assert [ref64.sample(x, u)[0] for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.99)] == \
        [0, 0, 1, 1, 2, 2, 3, 3]
    assert ref64.sample(x, 0.5, top_k=2)[::2] == (1, 2) and ref64.sample(x, 0.6, top_k=2)[0] == 3
    assert ref64.sample(x, 0.0, top_p=0.39)[2] == 1 and ref64.sample(x, 0.0, top_p=0.41)[2] == 2
    assert ref64.sample(x, 0.0, min_p=0.6)[2] == 2     # 0.3 / 0.4 = 0.75, 0.2 / 0.4 = 0.5
    assert ref64.sample(x, 0.7, T=0)[::2] == (1, 1)
    assert ref64.sample([1.0, 1.0, 1.0, 0.0], 0.99, top_k=2)[::2] == (1, 2)  # ties: lower ids
    assert ref64.sample([-np.inf, np.nan], 0.5) == (-1, -np.inf, 0)
    tok, lp, n = ref64.sample(x, 0.99, top_k=3, top_p=0.9)
    assert tok == 3 and n == 3 and abs(lp - np.log(0.3 / 0.9)) < 1e-12


@pytest.mark.parametrize("Hq,H,n", [(1, 1, 1), (2, 2, 1), (8, 1, 5), (20, 4, 1), (17, 1, 4)])
def test_workspace_of_a_capacity_covers_every_window(lib, Hq, H, n):
    """A call plans over what its window leaves of the capacity, and a shorter range can be cut
    into more splits than a longer one: blocks take tiles in rounds of two, one round each up to
    128 rounds and two each from 129 on. The reported size grows with the capacity and holds
    the partials (64 values, a maximum and a sum) of every shorter range that is worth cutting."""
    from kv_cached_decode_gb300 import (KVD_OP_DECODE_ATTN, KVD_OP_VERIFY_ATTN, KVD_OP_WINDOW_ATTN,
                                        KVD_WS_COUNTER_BYTES, kvd_workspace_size)

    M = Hq // H * n
    nsub = -(-M // 16)
    msub, units = -(-M // nsub), H * nsub

    def need(L):
        tiles = -(-L // 64)
        rounds = -(-tiles // 2)
        per = 2 * -(-rounds // min(rounds, 128))
        if units > 8 or 2 * -(-rounds // 16) - per <= 12:
            return KVD_WS_COUNTER_BYTES
        slots = units * -(-tiles // per) * msub
        return KVD_WS_COUNTER_BYTES + -(-slots * 64 * 4 // 256) * 256 + slots * 2 * 4

    ops = [KVD_OP_WINDOW_ATTN, KVD_OP_VERIFY_ATTN] + [KVD_OP_DECODE_ATTN] * (n == 1)
    most = 0
    for L in range(64, 100000, 64):
        most = max(most, need(L))
        for op in ops:
            assert kvd_workspace_size(op, 1, Hq, H, 1, n, L) >= most, L
    # 16512 positions: 65 splits of four tiles; a window of 15000: 118 of two
    assert need(15104) > need(16512) or units > 8


def test_q4_workspace_of_a_loose_bound(lib):
    """max_len may be any upper bound of the length: a looser one never gives less."""
    from kv_cached_decode_gb300 import KVD_OP_Q4_ATTN, kvd_workspace_size

    for B, Hq, H, n in ((1, 8, 8, 1), (16, 32, 8, 1), (64, 32, 8, 1), (80, 8, 8, 5), (81, 8, 8, 1)):
        last = 0
        for e in range(5, 31):
            for L in (1 << e, (1 << e) + (1 << e - 1)):
                size = kvd_workspace_size(KVD_OP_Q4_ATTN, B, Hq, H, 1, n, L)
                assert size >= last, (B, L)
                last = size


def test_a_cache_split_over_two_devices_is_refused():
    """One address of the two would be another device's."""
    from types import SimpleNamespace

    import kv_cached_decode_gb300 as kvd

    def fake(dev):
        return SimpleNamespace(shape=torch.Size((1, 2, 5, 64)), stride=lambda: (640, 320, 64, 1),
                               dtype=torch.float16, is_cuda=True, get_device=lambda: dev,
                               data_ptr=lambda: P)

    assert kvd.make_cache(fake(0), fake(0)).capacity == 5
    with pytest.raises(ValueError, match="one device"):
        kvd.make_cache(fake(0), fake(1))
