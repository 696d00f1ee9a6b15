"""Sliding window with sinks over the 16-bit cache (kvd_window_attn, kvd_prefill_window_attn)
against 64 bits: lengths from nothing to past the window, odd windows, sinks that end inside
a tile or meet the window, the fused append, and what lies outside the window."""

import numpy as np
import pytest
import torch

import ref64
from gpu_util import new_err, require_gpu

pytestmark = pytest.mark.gpu
DT = [torch.float16, torch.bfloat16]
WINDOWS = [(1, 0), (1, 3), (16, 0), (17, 5), (64, 64), (65, 1), (100, 130), (513, 4), (4000, 2),
           (7, 5000), (2 ** 31 - 1, 2 ** 31 - 1)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _i32(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _inputs(dtype, B, Hq, H, n, cap, seed):
    g = torch.Generator().manual_seed(seed)
    k = torch.randn(B, H, cap, 64, generator=g).to(dtype)
    v = torch.randn(B, H, cap, 64, generator=g).to(dtype)
    q = torch.randn(B, Hq, n, 64, generator=g).to(dtype)
    return q, k, v


def _compare(out, q, k, v, lens, window, sinks, scale=0.125):
    n = q.shape[2]
    for b, L in enumerate(lens):
        see = ref64.visible(L, n, True, window, sinks)
        want, mag, smax = ref64.attention(q[b].double(), k[b, :, :L].double(),
                                          v[b, :, :L].double(), see, scale)
        tol = ref64.attention_bound(want, mag, smax, q.dtype)
        bad = (out[b].double().cpu() - want).abs() > tol
        assert not bad.any(), (b, L, int(bad.sum()), bad.nonzero()[0].tolist())


def _run(q, k, v, lens, window, sinks, append=False, rope=0.0, flags=0, poison=True):
    """The kernel on a cache where every tile-neighbour no query sees holds NaN."""
    import kv_cached_decode_gb300 as kvd

    B, Hq, n, _ = q.shape
    H, cap = k.shape[1:3]
    kd, vd = k.clone(), v.clone()
    if poison:
        for b, L in enumerate(lens):
            seen = np.zeros(cap, bool)
            seen[:L] = ref64.visible(L, n, True, window, sinks).any(0)
            kd[b, :, ~seen] = float("nan")
            vd[b, :, ~seen] = float("inf")
    lens_in = list(lens)
    app = lo = None
    if append:
        lens_in = [L - n for L in lens]
        new = [torch.stack([x[b, :, L - n:L] for b, L in enumerate(lens)]).cuda()
               for x in (k, v)]
        for b, L in enumerate(lens):
            kd[b, :, L - n:L] = vd[b, :, L - n:L] = float("nan")
        lo = torch.full((B,), -1, dtype=torch.int32, device="cuda")
        app = (new[0], new[1], lo) + ((rope,) if rope else ())
    kd, vd = kd.cuda(), vd.cuda()
    out, err = torch.full_like(q.cuda(), 99.0), new_err()
    ws = kvd.new_workspace(kvd.kvd_workspace_size(kvd.KVD_OP_WINDOW_ATTN, B, Hq, H, 1, n, cap))
    kvd.kvd_window_attn(q.cuda(), kvd.make_cache(kd, vd), out, ws, window, sinks,
                        lens=_i32(*lens_in), dev_err=err, append=app, flags=flags)
    torch.cuda.synchronize()
    assert int(err) == 0 and not ws[:kvd.KVD_WS_COUNTER_BYTES].any()
    if append:
        assert lo.tolist() == list(lens)
        for b, L in enumerate(lens):  # the new rows are in the cache
            assert rope or torch.equal(kd[b, :, L - n:L].cpu(), k[b, :, L - n:L])
            assert torch.equal(vd[b, :, L - n:L].cpu(), v[b, :, L - n:L])
    return out


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_one_token(dtype, window, sinks):
    for (B, Hq, H, lens, cap) in ((3, 2, 2, [700, 64, 0], 701), (2, 10, 2, [1, 333], 400),
                                  (1, 1, 1, [1], 1)):
        q, k, v = _inputs(dtype, B, Hq, H, 1, cap, window % 97 + cap)
        out = _run(q, k, v, lens, window, sinks)
        _compare(out, q, k, v, lens, window, sinks)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n", [2, 5, 16])
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_blocks(dtype, window, sinks, n):
    for (B, Hq, H, lens, cap) in ((2, 2, 2, [600, n], 640), (2, 8, 2, [131, n - 1], 131 + n)):
        q, k, v = _inputs(dtype, B, Hq, H, n, cap, window % 89 + cap + n)
        out = _run(q, k, v, lens, window, sinks)
        _compare(out, q, k, v, lens, window, sinks)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("Hq,H,n", [(17, 1, 1), (8, 2, 5), (2, 1, 16), (12, 2, 11), (36, 1, 3)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (17, 5), (100, 130), (2000, 4)])
def test_more_query_vectors_than_sixteen(dtype, Hq, H, n, window, sinks):
    """Query blocks of up to 32 (17, 20, 32, 2 x 33, 4 x 27), rows empty or shorter than n."""
    for B, lens, cap in ((5, [2900, 0, n, 64, 129], 2900), (1, [n - 1], 40)):
        q, k, v = _inputs(dtype, B, Hq, H, n, cap, window + cap + n)
        out = _run(q, k, v, lens, window, sinks)
        _compare(out, q, k, v, lens, window, sinks)
        lens = [max(L, n) for L in lens]
        out = _run(q, k, v, lens, window, sinks, append=True)
        _compare(out, q, k, v, lens, window, sinks)


@pytest.mark.parametrize("n", [1, 5])
@pytest.mark.parametrize("window,sinks", [(1, 0), (30, 3), (64, 64), (1000, 1)])
def test_fused_append(window, sinks, n):
    lens = [600, n, 64, 65]
    q, k, v = _inputs(torch.float16, 4, 6, 3, n, 600, n + window)
    out = _run(q, k, v, lens, window, sinks, append=True)
    _compare(out, q, k, v, lens, window, sinks)
    plain = _run(q, k, v, lens, window, sinks)
    assert torch.equal(out, plain)


@pytest.mark.parametrize("n", [1, 4])
def test_fused_append_with_rotation_equals_rope_first(n):
    import kv_cached_decode_gb300 as kvd

    lens = [300, 64 + n]
    q, k, v = _inputs(torch.float16, 2, 4, 2, n, 320, 11)
    out = _run(q, k, v, lens, 70, 3, append=True, rope=10000.0)
    qr, kr = q.cuda().clone(), k.clone()
    pos = _i32(*[L - n for L in lens])
    new = torch.stack([k[b, :, L - n:L] for b, L in enumerate(lens)]).cuda()
    kvd.kvd_rope(qr, new, pos)
    for b, L in enumerate(lens):
        kr[b, :, L - n:L] = new[b].cpu()
    want = _run(qr.cpu(), kr, v, lens, 70, 3)
    assert torch.equal(out, want)


def test_values_some_queries_do_not_see():
    """Infinities and NaN in V rows that only some queries of a block see reach those."""
    import kv_cached_decode_gb300 as kvd

    for dtype in DT:
        q, k, v = _inputs(dtype, 1, 4, 1, 5, 300, 2)
        clean = _run(q, k, v, [250], 60, 2, poison=False)
        # queries at 245..249 see t > p - 60: from 186, 187, 188, 189, 190 on
        v2 = v.clone()
        v2[0, 0, 186, 7] = float("inf")
        v2[0, 0, 187, 63] = float("nan")
        v2[0, 0, 249, 0] = float("-inf")
        out = _run(q, k, v2, [250], 60, 2, poison=False).cpu()
        clean = clean.cpu()
        keep = torch.ones(5, 64, dtype=torch.bool)
        keep[0, 7] = keep[0, 63] = keep[1, 63] = keep[4, 0] = False
        assert torch.equal(out[0][:, keep], clean[0][:, keep])
        assert (out[0, :, 0, 7] == float("inf")).all() and torch.isnan(out[0, :, :2, 63]).all()
        assert (out[0, :, 4, 0] == float("-inf")).all()
    assert kvd.kvd_version()


def test_a_window_as_long_as_the_cache_is_the_plain_call():
    import kv_cached_decode_gb300 as kvd

    for n in (1, 5):
        q, k, v = _inputs(torch.float16, 2, 8, 2, n, 900, 21)
        lens = [900, 450]
        out = _run(q, k, v, lens, 900, 0)
        want = torch.empty_like(out)
        ws = kvd.new_workspace(1 << 20)
        cache = kvd.make_cache(k.cuda(), v.cuda())
        if n == 1:
            kvd.kvd_decode_attn(q.cuda(), cache, want, ws, lens=_i32(*lens))
        else:
            kvd.kvd_verify_attn(q.cuda(), cache, want, ws, lens=_i32(*lens))
        assert torch.allclose(out.float(), want.float(), rtol=2 ** -9, atol=2 ** -12)


def test_long_windows_through_the_workspace_and_pdl_chain():
    import kv_cached_decode_gb300 as kvd

    q, k, v = _inputs(torch.float16, 1, 2, 1, 1, 30000, 31)
    for L in (30000, 20011, 64):
        out = _run(q, k, v, [L], 20000, 100)
        _compare(out, q, k, v, [L], 20000, 100)
    # steps in a captured chain: append through the call, then read what it wrote
    n = 1
    kd, vd = k[:, :, :300].cuda(), v[:, :, :300].cuda()
    cache = kvd.make_cache(kd, vd)
    lens = [_i32(100)] + [_i32(0) for _ in range(3)]
    qs = [torch.randn(1, 2, n, 64, device="cuda").half() for _ in range(3)]
    new = [torch.randn(2, 1, 1, n, 64, device="cuda").half() for _ in range(3)]
    outs = [torch.zeros_like(x) for x in qs]
    ws = kvd.new_workspace(1 << 20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for i in range(3):
            kvd.kvd_window_attn(qs[i], cache, outs[i], ws, 40, 2, lens=lens[i],
                                append=(new[i][0], new[i][1], lens[i + 1]),
                                flags=kvd.KVD_FLAG_PDL)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert lens[3].tolist() == [103]
    for i in range(3):
        _compare(outs[i], qs[i].cpu(), kd.cpu(), vd.cpu(), [101 + i], 40, 2)


def test_bad_lengths_leave_rows_alone():
    import kv_cached_decode_gb300 as kvd

    for n in (1, 3):
        q, k, v = _inputs(torch.float16, 3, 2, 2, n, 100, 41)
        out, err = torch.full_like(q.cuda(), 7.0), new_err()
        kvd.kvd_window_attn(q.cuda(), kvd.make_cache(k.cuda(), v.cuda()), out,
                            kvd.new_workspace(1 << 16), 10, 1, lens=_i32(100, 101, -1),
                            dev_err=err)
        torch.cuda.synchronize()
        assert int(err) == 16 and (out[1:] == 7).all()
        _compare(out, q, k, v, [100], 10, 1)


# ------------------------------------------------------------------ prefill ----------
def _prefill(dtype, B, Hq, H, n, cap, plens, start, window, sinks, seed, rope=0.0):
    import kv_cached_decode_gb300 as kvd

    q, k, v = _inputs(dtype, B, Hq, H, n, cap, seed)
    kn, vn = (torch.randn(B, H, n, 64, generator=torch.Generator().manual_seed(seed + i)).to(dtype)
              for i in (1, 2))
    kd, vd = k.clone(), v.clone()
    for b in range(B):
        L = start[b] + plens[b]
        k[b, :, start[b]:L] = kn[b, :, :plens[b]]
        v[b, :, start[b]:L] = vn[b, :, :plens[b]]
        seen = np.zeros(cap, bool)
        if plens[b]:
            seen[:L] = ref64.visible(L, plens[b], True, window, sinks).any(0)
        kd[b, :, ~seen] = float("nan")
        vd[b, :, ~seen] = float("nan")
    kd, vd = kd.cuda(), vd.cuda()
    out, err = torch.full_like(q.cuda(), 55.0), new_err()
    lo = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    kvd.kvd_prefill_window_attn(q.cuda(), kvd.make_cache(kd, vd), kn.cuda(), vn.cuda(),
                                _i32(*plens), out, window, sinks, lens_in=_i32(*start),
                                lens_out=lo, rope_base=rope, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 0 and lo.tolist() == [s + p for s, p in zip(start, plens)]
    out = out.cpu()
    for b in range(B):
        m, L = plens[b], start[b] + plens[b]
        assert not out[b, :, m:].any()
        if rope:
            continue
        assert torch.equal(kd[b, :, start[b]:L].cpu(), k[b, :, start[b]:L])
        see = ref64.visible(L, m, True, window, sinks)
        want, mag, smax = ref64.attention(q[b, :, :m].double(), k[b, :, :L].double(),
                                          v[b, :, :L].double(), see, 0.125)
        tol = ref64.attention_bound(want, mag, smax, dtype)
        bad = (out[b, :, :m].double() - want).abs() > tol
        assert not bad.any(), (b, int(bad.sum()), bad.nonzero()[0].tolist())
    return out, q, kn, vn


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 2), (50, 0), (64, 64), (129, 4), (200, 70),
                                          (1000, 3), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_prefill(window, sinks):
    dtype = DT[window % 2]
    _prefill(dtype, 2, 2, 1, 300, 300, [300, 129], [0, 0], window, sinks, 51)
    _prefill(dtype, 2, 1, 1, 150, 700, [150, 1], [431, 640], window, sinks, 52)
    _prefill(dtype, 2, 3, 3, 1, 40, [1, 0], [39, 3], window, sinks, 53)


def test_prefill_rotation_and_agreement_with_the_token_by_token_call():
    import kv_cached_decode_gb300 as kvd

    out, q, kn, vn = _prefill(torch.float16, 1, 2, 1, 200, 300, [200], [60], 33, 2, 61,
                              rope=10000.0)
    # the same prompt a token at a time; the prefix is NaN where nothing sees it
    g = torch.Generator().manual_seed(61)
    k = torch.randn(1, 1, 300, 64, generator=g).half().cuda()
    v = torch.randn(1, 1, 300, 64, generator=g).half().cuda()
    cache = kvd.make_cache(k, v)
    ws = kvd.new_workspace(1 << 16)
    for j in range(200):
        o = torch.empty(1, 2, 1, 64, dtype=torch.float16, device="cuda")
        new = [x[:, :, j:j + 1].contiguous().cuda() for x in (q, kn, vn)]
        kvd.kvd_window_attn(new[0], cache, o, ws, 33, 2, lens=_i32(60 + j),
                            append=(new[1], new[2], None, 10000.0))
        assert torch.allclose(o.cpu().float(), out[:, :, j:j + 1].float(), rtol=2 ** -8,
                              atol=2 ** -9), j


@pytest.mark.parametrize("Hq,H,n", [(8, 2, 5), (4, 4, 1), (16, 16, 12)])
def test_a_wait_that_runs_out_is_reported(Hq, H, n):
    """The first stage of every unit's last split never completes (KVD_FLAG_TEST_STALL): the
    blocks of 32, 8 and 16 query vectors give up, write nothing, and the next call is right."""
    import kv_cached_decode_gb300 as kvd

    L = 1500
    q, k, v = _inputs(torch.float16, 1, Hq, H, n, L, n)
    cache = kvd.make_cache(k.cuda(), v.cuda())
    ws = kvd.new_workspace(kvd.kvd_workspace_size(kvd.KVD_OP_WINDOW_ATTN, 1, Hq, H, 1, n, L))
    qd = q.cuda()
    out, err = torch.full_like(qd, 3.0), new_err()
    kvd.kvd_window_attn(qd, cache, out, ws, L, fixed_len=L, flags=kvd.KVD_FLAG_TEST_STALL,
                        dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 20 and (out == 3.0).all()
    err.zero_()
    kvd.kvd_window_attn(qd, cache, out, ws, L, fixed_len=L, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    _compare(out.cpu(), q, k, v, [L], L, 0)


@pytest.mark.parametrize("Hq,H,n,cap,window", [(1, 1, 1, 16512, 15000), (2, 2, 1, 16512, 15000),
                                               (8, 1, 5, 33000, 16200), (1, 1, 4, 70000, 15500)])
def test_a_long_window_with_the_workspace_of_its_capacity(Hq, H, n, cap, window):
    """Windows that are cut into more splits than the whole capacity would be, with a workspace of
    exactly the reported size."""
    lens = [cap]
    q, k, v = _inputs(torch.float16, 1, Hq, H, n, cap, cap + n)
    out = _run(q, k, v, lens, window, 3)
    _compare(out, q, k, v, lens, window, 3)
