"""kvd_qk_norm_rope against its 64-bit form: strides, head counts, far and negative
positions, in place, one and many tokens."""

import numpy as np
import pytest
import torch

import ref64
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _check(got, x, w, pos, eps, base):
    want, mag = ref64.norm_rope(x.double().cpu().numpy(),
                                None if w is None else w.double().cpu().numpy(),
                                pos, eps, base)
    want, mag = torch.from_numpy(want), torch.from_numpy(mag)
    # the output's rounding, and 64 roundings of 2^-24 in the sum of squares (half of it
    # after the root), the products and the angle
    err = mag * 2.0 ** -18
    tol = err + ref64.HALF[got.dtype] * (want.abs() + err) + 2.0 ** -24
    bad = (got.double().cpu() - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("B,n,hq,hk", [(1, 1, 1, 1), (8, 1, 32, 8), (3, 5, 9, 3), (2, 300, 20, 4),
                                       (1, 2500, 15, 5), (5, 1, 8, 1)])
def test_fused_projection(dtype, B, n, hq, hk):
    import kv_cached_decode_gb300 as kvd

    g = torch.Generator(device="cuda").manual_seed(B * 1000 + n)
    qkv = (torch.randn(B, n, hq + 2 * hk, 64, generator=g, device="cuda") * 3).to(dtype)
    wq, wk = ((1 + 0.3 * torch.randn(64, generator=g, device="cuda")).to(dtype) for _ in "qk")
    pos0 = torch.randint(0, 131072, (B,), generator=g, device="cuda", dtype=torch.int32)
    heads = qkv.transpose(1, 2)
    q, k = heads[:, :hq], heads[:, hq:hq + hk]
    qo = torch.full((B, hq, n, 64), float("nan"), dtype=dtype, device="cuda")
    ko = torch.full((B, hk, n, 64), float("nan"), dtype=dtype, device="cuda")
    before = qkv.clone()
    kvd.kvd_qk_norm_rope(q, k, qo, ko, q_weight=wq, k_weight=wk, pos0=pos0)
    torch.cuda.synchronize()
    assert torch.equal(qkv, before)
    pos = pos0.cpu().numpy()[:, None].astype(np.int64) + np.arange(n)
    _check(qo, q, wq, pos, 1e-6, 10000.0)
    _check(ko, k, wk, pos, 1e-6, 10000.0)


@pytest.mark.parametrize("base", [0.0, 500000.0, 0.5])
def test_one_tensor_in_place_and_positions(base):
    import kv_cached_decode_gb300 as kvd

    B, H, n = 4, 6, 3
    x = torch.randn(B, H, n, 64, device="cuda", dtype=torch.float16)
    pos0 = torch.tensor([0, -7, 2 ** 31 - 2, 1 << 20], dtype=torch.int32, device="cuda")
    pos = pos0.cpu().numpy()[:, None].astype(np.int64) + np.arange(n)
    if base == 0.5:
        # theta above 1: 2^31 of its turns are known to 2^31 * 2^-52 in 64 bits here
        pos0[2] = 12345
        pos[2] = 12345 + np.arange(n)
    y = x.clone()
    kvd.kvd_qk_norm_rope(k=y, k_out=y, pos0=pos0, eps=1e-5, base=base)
    torch.cuda.synchronize()
    _check(y, x, None, pos, 1e-5, base)
    z = torch.empty_like(x)
    kvd.kvd_qk_norm_rope(q=x, q_out=z, pos0=pos0, eps=1e-5, base=base)
    assert torch.equal(y, z)


def test_extreme_values_rows():
    import kv_cached_decode_gb300 as kvd

    x = torch.zeros(1, 4, 1, 64, device="cuda", dtype=torch.bfloat16)
    x[0, 1] = 1e-6                      # eps dominates
    x[0, 2, 0, 5] = float("inf")
    x[0, 3] = torch.randn(64, device="cuda").bfloat16()
    y = torch.empty_like(x)
    kvd.kvd_qk_norm_rope(q=x, q_out=y, eps=1e-6)
    want, _ = ref64.norm_rope(x[:, [0, 1, 3]].double().cpu().numpy(), None,
                              np.zeros((1, 1), np.int64), 1e-6, 10000.0)
    got = y[:, [0, 1, 3]].double().cpu().numpy()
    assert (got[0, 0] == 0).all()
    assert np.abs(got - want).max() <= 2.0 ** -8 * np.abs(want).max() * 1.01
    assert torch.isnan(y[0, 2, 0, 5])   # inf / inf, as the formula has it


def test_padded_strides_and_size_one_axes():
    import kv_cached_decode_gb300 as kvd

    big = torch.randn(3, 7, 11, 72, device="cuda", dtype=torch.float16)
    x = big[:, 1:6, 2:9, :64]
    y = torch.empty(3, 5, 7, 64, device="cuda", dtype=torch.float16)
    kvd.kvd_qk_norm_rope(q=x, q_out=y)
    _check(y, x, None, np.arange(7)[None].repeat(3, 0), 1e-6, 10000.0)
    one = torch.randn(64 + 3, device="cuda", dtype=torch.float16)[:64].as_strided(
        (1, 1, 1, 64), (3, 5, 1, 1))
    y = torch.empty(1, 1, 1, 64, device="cuda", dtype=torch.float16)
    kvd.kvd_qk_norm_rope(q=one, q_out=y)
    _check(y, one, None, np.zeros((1, 1), np.int64), 1e-6, 10000.0)
    with pytest.raises(kvd.KvdError):    # rows that start off a 16-byte boundary
        bad = torch.randn(4, 5, 66, device="cuda", dtype=torch.float16)[None, :, :, :64]
        kvd.kvd_qk_norm_rope(q=bad, q_out=torch.empty(1, 4, 5, 64, device="cuda",
                                                      dtype=torch.float16))
    with pytest.raises(kvd.KvdError):    # in place needs the output's layout
        t = torch.randn(2, 5, 3, 64, device="cuda", dtype=torch.float16)
        v = t.transpose(1, 2)
        out = torch.as_strided(t, (2, 3, 5, 64), (960, 320, 64, 1))
        kvd.kvd_qk_norm_rope(q=v, q_out=out)


def test_empty_calls_and_streams():
    import kv_cached_decode_gb300 as kvd

    e = torch.empty(0, 4, 1, 64, device="cuda", dtype=torch.float16)
    kvd.kvd_qk_norm_rope(q=e, q_out=torch.empty_like(e))
    e = torch.empty(2, 4, 0, 64, device="cuda", dtype=torch.float16)
    kvd.kvd_qk_norm_rope(q=e, q_out=torch.empty_like(e))
    x = torch.randn(2, 4, 3, 64, device="cuda", dtype=torch.float16)
    y, z = torch.empty_like(x), torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    kvd.kvd_qk_norm_rope(q=x, q_out=y, stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kvd.kvd_qk_norm_rope(q=x, q_out=z, flags=kvd.KVD_FLAG_PDL)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, z)
