"""The 4-bit cache on the GPU: append and read-back bit by bit against the format's
definition, attention against 64 bits over the stored values."""

import numpy as np
import pytest
import torch

import ref64
from gpu_util import new_err, require_gpu

pytestmark = pytest.mark.gpu
DT = [torch.float16, torch.bfloat16]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _i32(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _host(cache):
    return [t.cpu().numpy() for t in cache._tensors]


def _cases(dtype):
    """Rows where the format can go wrong: ties, constants, zeros, extremes of the type."""
    g = torch.Generator().manual_seed(5)
    big = torch.finfo(dtype).max
    rows = [torch.randn(64, generator=g), torch.zeros(64), -torch.zeros(64), torch.full((64,), 3.0),
            torch.full((64,), -0.7), torch.arange(64) - 31.5, torch.arange(64) % 16,
            torch.linspace(-big, big, 64, dtype=torch.float64).float(), torch.full((64,), big), torch.full((64,), -big),
            torch.full((64,), torch.finfo(dtype).tiny), torch.randn(64, generator=g) * 1e-7,
            1000 + torch.randn(64, generator=g), torch.randn(64, generator=g) * 1e4,
            torch.where(torch.arange(64) == 7, 100.0, 0.01),
            torch.linspace(-1, 1, 64) * torch.finfo(dtype).smallest_normal]
    return torch.stack(rows).to(dtype)


@pytest.mark.parametrize("dtype", DT)
def test_append_bits_follow_the_definition(dtype):
    import kv_cached_decode_gb300 as kvd

    x = _cases(dtype).cuda().reshape(2, 2, 4, 64)
    y = torch.randn(2, 2, 4, 64, device="cuda").to(dtype)
    c = kvd.new_q4_cache(2, 2, 9)
    err = new_err()
    out = _i32(0, 0)
    kvd.kvd_q4_append(c, x, y, _i32(0, 5), lens_out=out, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 0 and out.tolist() == [4, 9]
    k, v, par = _host(c)
    for t, (data, at) in ((x, (k, 0)), (y, (v, 2))):
        n, step, z = ref64.q4_quantise(t.float().cpu().numpy())
        want = np.zeros_like(data)
        wpar = np.zeros((2, 2, 9, 2), np.int16)
        for b, p in ((0, 0), (1, 5)):
            want[b, :, p:p + 4] = ref64.q4_pack(n[b])
            wpar[b, :, p:p + 4] = ref64.q4_params(step[b], z[b])
        assert np.array_equal(data, want)
        assert np.array_equal(par[..., at:at + 2], wpar)
        # and the values are near: half a step and what the grid's rounding moved
        val = ref64.q4_values(data, par[..., at:at + 2])
        for b, p in ((0, 0), (1, 5)):
            d = np.abs(val[b, :, p:p + 4] - t[b].double().cpu().numpy())
            s, zz = step[b].astype(float), np.abs(z[b].astype(float))
            assert (d <= s * (0.5 + 15 * 2.0 ** -8 + zz * 2.0 ** -10)).all()


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n", [64, 1100])
def test_append_bits_of_random_rows(dtype, n):
    """Rows of every magnitude and offset: the quotients round as the definition's divisions."""
    import kv_cached_decode_gb300 as kvd

    g = torch.Generator().manual_seed(n)
    H = 8
    low, high = (-120, 120) if dtype == torch.bfloat16 else (-20, 13)
    x = []
    for _ in "kv":
        e = torch.randint(low, high, (1, H, n, 1), generator=g).double()
        off = torch.randn(1, H, n, 1, generator=g) * (torch.rand(1, H, n, 1, generator=g) < 0.5)
        x.append(((torch.randn(1, H, n, 64, generator=g).double() + 4 * off) * 2 ** e).to(dtype))
    c = kvd.new_q4_cache(1, H, n)
    err = new_err()
    kvd.kvd_q4_append(c, x[0].cuda(), x[1].cuda(), dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    k, v, par = _host(c)
    for t, data, at in ((x[0], k, 0), (x[1], v, 2)):
        want, step, z = ref64.q4_quantise(t.float().numpy())
        assert np.array_equal(par[..., at:at + 2], ref64.q4_params(step, z))
        assert np.array_equal(data, ref64.q4_pack(want))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,H,n,cap", [(1, 1, 1, 1), (3, 5, 33, 97), (2, 8, 700, 1001)])
def test_append_counts_and_read_back(dtype, B, H, n, cap):
    import kv_cached_decode_gb300 as kvd

    g = torch.Generator(device="cuda").manual_seed(n)
    k = torch.randn(B, H, n, 64, generator=g, device="cuda").to(dtype)
    v = torch.randn(B, H, n, 64, generator=g, device="cuda").to(dtype)
    c = kvd.new_q4_cache(B, H, cap)
    for t in c._tensors:
        t.fill_(17)
    counts = torch.randint(0, n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    counts[0] = n
    pos = torch.randint(0, cap - n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens, err = torch.full_like(pos, -1), new_err()
    kvd.kvd_q4_append(c, k, v, pos, lens_out=lens, counts=counts, dev_err=err)
    assert torch.equal(lens, pos + counts) and int(err) == 0
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    kvd.kvd_q4_dequant(c, kb, vb, pos0=pos, dev_err=err)
    only = torch.empty_like(v)
    kvd.kvd_q4_dequant(c, v_out=only, pos0=pos)
    torch.cuda.synchronize()
    assert int(err) == 0 and torch.equal(only, vb)
    data = _host(c)
    for b in range(B):
        p, m = int(pos[b]), int(counts[b])
        for t in data:  # rows outside were left as they were
            assert (t[b, :, :p] == 17).all() and (t[b, :, p + m:] == 17).all()
        for x, back in ((k, kb), (v, vb)):
            q, step, z = ref64.q4_quantise(x[b, :, :m].float().cpu().numpy())
            want = torch.from_numpy((q - z.astype(np.float32)).astype(np.float32) * step).to(dtype)
            assert torch.equal(back[b, :, :m].cpu(), want)


def test_append_errors_on_the_device():
    import kv_cached_decode_gb300 as kvd

    x = torch.randn(4, 2, 3, 64, device="cuda", dtype=torch.float16)
    c = kvd.new_q4_cache(4, 2, 10)
    err, out = new_err(), _i32(9, 9, 9, 9)
    kvd.kvd_q4_append(c, x, x, _i32(8, -1, 7, 0), lens_out=out, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 16 and out.tolist() == [8, -1, 10, 3]
    assert not c._tensors[0][:2].any() and c._tensors[0][2, :, 7:].any()
    err.zero_()
    kvd.kvd_q4_append(c, x, x, counts=_i32(4, -1, 0, 1), lens_out=out, dev_err=err)
    assert int(err) == 16 and out.tolist() == [0, 0, 0, 1]
    err.zero_()
    y = torch.full_like(x, 7.0)
    kvd.kvd_q4_dequant(c, y, pos0=_i32(8, -1, 7, 2 ** 31 - 1), dev_err=err)
    assert int(err) == 16 and (y[[0, 1, 3]] == 7).all() and not (y[2] == 7).all()
    # an infinity or a NaN: its row reads back as NaN, the others are not touched by it
    err.zero_()
    x[1, 1, 2, 3] = float("inf")
    x[2, 0, 0, 63] = float("nan")
    kvd.kvd_q4_append(c, x, torch.zeros_like(x), dev_err=err)
    kvd.kvd_q4_dequant(c, y)
    assert int(err) == 19
    nan = torch.isnan(y).all(-1)
    assert nan[1, 1, 2] and nan[2, 0, 0] and int(torch.isnan(y).sum()) == 128


# ------------------------------------------------------------------ attention --------
def _filled(B, H, cap, g, spread=1.0, offset=0.5):
    """A cache of random rows, written by its definition, every position filled."""
    import kv_cached_decode_gb300 as kvd

    c = kvd.new_q4_cache(B, H, cap)
    for t, at in ((0, 0), (1, 2)):
        x = torch.randn(B, H, cap, 64, generator=g) * spread + offset * torch.randn(
            1, H, 1, 64, generator=g)
        n, step, z = ref64.q4_quantise(x.numpy())
        c._tensors[t].copy_(torch.from_numpy(ref64.q4_pack(n)))
        c._tensors[2][..., at:at + 2].copy_(torch.from_numpy(ref64.q4_params(step, z)))
    return c


def _attend(c, q, lens, want_rows=None, scale=0.125, **kw):
    """Run the kernel and compare every row with 64 bits. lens: a list."""
    import kv_cached_decode_gb300 as kvd

    B, Hq, n, _ = q.shape
    H, cap = c.n_kv_heads, c.capacity
    out = torch.full_like(q, 123.0)
    ws = kvd.new_workspace(kvd.kvd_workspace_size(kvd.KVD_OP_Q4_ATTN, B, Hq, H, 1, n, cap))
    err = new_err()
    kvd.kvd_q4_attn(q, c, out, ws, lens=_i32(*lens), scale=scale, dev_err=err, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0 and not ws[:kvd.KVD_WS_COUNTER_BYTES].any()
    kd, vd, par = _host(c)
    for b in range(B):
        L = lens[b]
        k = torch.from_numpy(ref64.q4_values(kd[b, :, :L], par[b, :, :L, 0:2]))
        v = torch.from_numpy(ref64.q4_values(vd[b, :, :L], par[b, :, :L, 2:4]))
        see = ref64.visible(L, n, kw.get("causal", True), kw.get("window", 0),
                            kw.get("n_sinks", 0))
        # scores are sums over n and over the zero point, apart
        kmag = torch.from_numpy(ref64.q4_values(kd[b, :, :L], par[b, :, :L, 0:2], size=True))
        want, mag, smax = ref64.attention(q[b].double().cpu(), k, v, see, scale, kmag)
        # a weight below binary16's normal range is off by 2^-25 of the largest step's power
        # of two, times |n - z|: at most 4 times the largest value for these rows
        vmax = float(v.abs().max()) if L else 0.0
        floor = L * 2.0 ** -25 * vmax * 4
        tol = ref64.attention_bound(want, mag, smax, q.dtype, torch.float16, floor)
        bad = (out[b].double().cpu() - want).abs() > tol
        assert not bad.any(), (b, L, int(bad.sum()), bad.nonzero()[0].tolist())
    return out


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("B,Hq,H,n,cap,lens", [
    (1, 1, 1, 1, 1, [1]),
    (3, 2, 2, 1, 40, [0, 1, 40]),
    (2, 8, 2, 1, 333, [333, 31]),
    (4, 5, 1, 1, 1025, [1025, 32, 33, 700]),
    (2, 3, 3, 5, 100, [100, 5]),
    (1, 8, 2, 5, 777, [777]),
    (2, 16, 1, 1, 130, [129, 64]),
    (1, 20, 1, 3, 65, [65]),
    (1, 4, 1, 16, 520, [519]),
    (2, 2, 2, 4, 64, [2, 0]),           # fewer positions than queries: rows that see nothing
])
def test_attention_shapes(dtype, B, Hq, H, n, cap, lens):
    g = torch.Generator().manual_seed(cap * 7 + n)
    c = _filled(B, H, cap, g)
    q = torch.randn(B, Hq, n, 64, generator=g).to(dtype).cuda()
    out = _attend(c, q, lens)
    for b, L in enumerate(lens):
        assert not out[b, :, :max(0, n - L)].any()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (17, 0), (33, 40), (64, 1), (100, 64),
                                          (500, 5), (5000, 2), (7, 5000), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("n", [1, 5])
def test_attention_windows(window, sinks, n):
    g = torch.Generator().manual_seed(window % 1000 + sinks % 1000 + n)
    c = _filled(3, 2, 641, g)
    q = torch.randn(3, 6, n, 64, generator=g).half().cuda()
    _attend(c, q, [641, 200, n], window=window, n_sinks=sinks)


def test_attention_cross_and_scales():
    g = torch.Generator().manual_seed(3)
    c = _filled(2, 2, 300, g)
    q = torch.randn(2, 4, 3, 64, generator=g).half().cuda()
    _attend(c, q, [300, 7], causal=False)
    _attend(c, q, [300, 2], causal=False)
    for scale in (0.0, -0.125, 1.0):
        _attend(c, q, [300, 7], scale=scale)


@pytest.mark.parametrize("dtype", DT)
def test_attention_small_and_large_magnitudes(dtype):
    """Powers of two of q and of the rows that leave binary16's range without the scaling."""
    import kv_cached_decode_gb300 as kvd

    g = torch.Generator().manual_seed(8)
    for up in ((-12, 12) if dtype == torch.float16 else (-100, 100)):
        c = _filled(1, 2, 200, g)
        q = (torch.randn(1, 4, 2, 64, generator=g) * 2.0 ** up).to(dtype).cuda()
        if dtype == torch.float16 and up > 0:
            q.clamp_(-60000, 60000)
        _attend(c, q, [200], scale=2.0 ** -up * 0.1)
    # V's steps far above and below binary16, changing along the cache
    c = _filled(1, 1, 256, g)
    step = c._tensors[2][..., 2:3].contiguous().view(torch.bfloat16)
    e = torch.linspace(-40, 3, 256, device="cuda")[None, None, :, None]
    c._tensors[2][..., 2:3] = (step.float() * torch.exp2(e)).bfloat16().view(torch.int16)
    q = torch.randn(1, 2, 1, 64, generator=g).to(dtype).cuda()
    out = torch.empty_like(q)
    for L in (1, 30, 100, 256):
        _attend(c, q, [L])
    assert kvd.kvd_version() and out.shape == q.shape


def test_one_long_row():
    g = torch.Generator().manual_seed(4)
    c = _filled(1, 1, 40001, g)
    q = torch.randn(1, 4, 1, 64, generator=g).half().cuda()
    _attend(c, q, [40001])
    _attend(c, q, [513])
    _attend(c, q, [0])


@pytest.mark.parametrize("Hq,n,dtype,window", [(8, 1, torch.float16, 0), (8, 1, torch.bfloat16, 0),
                                               (24, 2, torch.float16, 0), (8, 5, torch.float16, 0),
                                               (8, 2, torch.float16, 8160)])
def test_many_tiles_stream_through_the_workspace(Hq, n, dtype, window):
    """Work enough for the launches whose CTAs take stretches of one list of tiles: ragged rows,
    rows that are empty or hold a tile, units cut by many CTAs, lists cut at the ends of units."""
    import kv_cached_decode_gb300 as kvd

    g = torch.Generator(device="cuda").manual_seed(Hq + n)
    B, H, cap = 20, 8, 8201
    c = kvd.new_q4_cache(B, H, cap)
    kvd.kvd_q4_append(c, *(torch.randn(B, H, cap, 64, generator=g, device="cuda").half()
                           for _ in "kv"))
    q = torch.randn(B, Hq, n, 64, generator=g, device="cuda").to(dtype)
    kw = dict(window=window, n_sinks=40) if window else {}
    full = _attend(c, q, [cap] * B, **kw)
    few = [0, 1, 17, 3000, 0, 33, 2, 500, 64, 0, 900]
    _attend(c, q, [cap] + few + [31, 32, 0, 1500, 700, 8200, 8000, 300], **kw)
    _attend(c, q, few + [1] * 8 + [cap], **kw)
    for L in (40, 250, 700):
        _attend(c, q, [L] * B, **kw)
    _attend(c, q, [cap * (b + 1) // B for b in range(B)], **kw)
    _attend(c, q, [0] * B, **kw)
    _attend(c, q, [0, 0, 0, 5] + [0] * 16, **kw)
    # a length out of range leaves its row
    ws = kvd.new_workspace(kvd.kvd_workspace_size(kvd.KVD_OP_Q4_ATTN, B, Hq, H, 1, n, cap))
    out, err = torch.full_like(q, 9.0), new_err()
    kvd.kvd_q4_attn(q, c, out, ws, lens=_i32(cap, -1, cap, cap, cap + 1, *[cap] * 15), dev_err=err,
                    **kw)
    torch.cuda.synchronize()
    assert int(err) == 16 and (out[[1, 4]] == 9).all()
    keep = [0, 2, 3] + list(range(5, B))
    assert torch.allclose(out[keep].float(), full[keep].float(), rtol=2 ** -7, atol=2 ** -10)
    for w in (None, ws[:4096 * 16]):
        with pytest.raises(kvd.KvdError) as e:
            kvd.kvd_q4_attn(q, c, out, w, lens=_i32(*[cap] * B), **kw)
        assert e.value.status == 3
    # the same bits on every run
    again = torch.empty_like(q)
    for _ in range(5):
        kvd.kvd_q4_attn(q, c, again, ws, lens=_i32(*[cap] * B), **kw)
        assert torch.equal(again, full)


def test_rows_that_do_not_see_infinities():
    """A NaN row (a token stored from an infinity) outside a query's window, behind its
    position or past the length does not reach it."""
    import kv_cached_decode_gb300 as kvd

    g = torch.Generator().manual_seed(6)
    c = _filled(1, 1, 200, g)
    q = torch.randn(1, 2, 4, 64, generator=g).half().cuda()
    clean = torch.empty_like(q)
    kw = dict(window=50, n_sinks=2)
    kvd.kvd_q4_attn(q, c, clean, lens=_i32(150), **kw)
    nan = c._tensors[2]
    for t in (5, 90, 97, 149, 150, 160):
        nan[0, 0, t, 0] = nan[0, 0, t, 2] = 0x7FC0
    nan[0, 0, 98, 2] = 0x7F80            # an infinite step
    nan[0, 0, 99, 3] = 0x7C00            # an infinite zero point
    out = torch.empty_like(q)
    kvd.kvd_q4_attn(q, c, out, lens=_i32(150), **kw)
    torch.cuda.synchronize()
    # positions 146..149 see t > p - 50: 97.., 98.., 99.., 100..; 149 only the last query
    assert torch.isnan(out[0, :, 0]).all()
    assert not torch.isfinite(out[0, :, 1]).any() and not torch.isfinite(out[0, :, 2]).any()
    assert torch.isnan(out[0, :, 3]).all()
    for t in (97, 98, 99, 149):
        nan[0, 0, t, 0] = 0x3F80
        nan[0, 0, t, 2] = 0x3F80
        nan[0, 0, t, 3] = 0
    kvd.kvd_q4_attn(q, c, out, lens=_i32(150), **kw)
    assert torch.isfinite(out).all()
    # a NaN that only the first query sees leaves the others' bits as they are
    kvd.kvd_q4_attn(q, c, clean, lens=_i32(150), **kw)
    nan[0, 0, 97, 2] = 0x7FC0
    kvd.kvd_q4_attn(q, c, out, lens=_i32(150), **kw)
    assert torch.equal(out[0, :, 1:], clean[0, :, 1:]) and torch.isnan(out[0, :, 0]).all()
    # a NaN in one query stays in its row
    q[0, 0, 2, 9] = float("nan")
    nan[0, 0, 97, 2] = 0x3F80
    kvd.kvd_q4_attn(q, c, out, lens=_i32(150), **kw)
    assert torch.isnan(out[0, 0, 2]).all() and int(torch.isnan(out).sum()) == 64


def test_bad_lengths_streams_graphs_and_strided_caches():
    import kv_cached_decode_gb300 as kvd

    g = torch.Generator().manual_seed(7)
    c = _filled(3, 2, 300, g)
    q = torch.randn(3, 4, 1, 64, generator=g).half().cuda()
    want = torch.full_like(q, 5.0)
    kvd.kvd_q4_attn(q, c, want, lens=_i32(300, 100, 300))
    out, err = torch.full_like(q, 5.0), new_err()
    kvd.kvd_q4_attn(q, c, out, lens=_i32(300, 301, -1), dev_err=err)
    assert int(err) == 16 and torch.equal(out[0], want[0]) and (out[1:] == 5).all()
    # the same rows in a larger buffer, heads and rows apart
    big = [torch.zeros(4, 3, 320, t.shape[3], dtype=t.dtype, device="cuda") for t in c._tensors]
    for x, t in zip(big, c._tensors):
        x[:3, 1:, :300] = t
    view = kvd.make_q4_cache(*[x[:3, 1:, :300] for x in big])
    kvd.kvd_q4_attn(q, view, out, lens=_i32(300, 100, 300))
    assert torch.equal(out, want)
    # another stream, and two graphs
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    lens = _i32(300, 100, 300)
    o1, o2 = torch.zeros_like(q), torch.zeros_like(q)
    kvd.kvd_q4_attn(q, c, o1, lens=lens, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvd.kvd_q4_attn(q, c, o2, lens=lens, flags=kvd.KVD_FLAG_PDL)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o1, want) and torch.equal(o2, want)
    # fixed_len instead of lens
    kvd.kvd_q4_attn(q, c, out, fixed_len=300)
    assert torch.equal(out[0], want[0])


def test_offsets_past_32_bits():
    """The last row of a cache of more than 2^32 bytes."""
    import kv_cached_decode_gb300 as kvd

    H, cap = 16, 1 << 23                 # 2^32 bytes of K, as many of V
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GiB")
    c = kvd.new_q4_cache(1, H, cap)
    x = torch.randn(1, H, 40, 64, device="cuda").half()
    y = torch.randn(1, H, 40, 64, device="cuda").half()
    kvd.kvd_q4_append(c, x, y, _i32(cap - 40))
    q = torch.randn(1, H, 1, 64, device="cuda").half()
    out, small = torch.empty_like(q), torch.empty_like(q)
    kvd.kvd_q4_attn(q, c, out, lens=_i32(cap), window=40)
    d = kvd.new_q4_cache(1, H, 40)
    kvd.kvd_q4_append(d, x, y)
    kvd.kvd_q4_attn(q, d, small, lens=_i32(40))
    torch.cuda.synchronize()
    assert torch.allclose(out.float(), small.float(), rtol=2 ** -10, atol=2 ** -12)
