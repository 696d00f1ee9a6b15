"""kvd_rope_scaled against its 64-bit form: layouts, parts of the head, scalings, strides, far and
negative positions, in place."""

import numpy as np
import pytest
import torch

import ref64_serving as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

SPECS = [dict(),
         dict(rot_dim=32, interleaved=True, base=500.0),
         dict(rot_dim=16),
         dict(rot_dim=48, magnitude=1.25),
         dict(rot_dim=48, interleaved=True),
         dict(interleaved=True, scaling="linear", factor=4.0),
         dict(base=500000.0, scaling="bands", factor=8.0, original_len=8192, low=1.0, high=4.0),
         dict(scaling="ramp", factor=16.0, original_len=4096, low=1.0, high=32.0,
              magnitude=1.2772588),
         dict(rot_dim=32, scaling="ramp", factor=2.0, original_len=100, low=0.5, high=90.0)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def check(got, x, pos, spec):
    want, size = ref.rotate(x.double().cpu().numpy(), pos, spec)
    tol = ref.rotation_bound(want, size, got.dtype, np.abs(pos).max())
    rot = spec.get("rot_dim", 64)
    assert torch.equal(got[..., rot:], x[..., rot:])
    bad = np.abs(got.double().cpu().numpy() - want) > tol
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[0].tolist())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("spec", SPECS, ids=range(len(SPECS)))
def test_layouts_and_scalings(dtype, spec):
    import kv_cached_decode_gb300 as kvd

    g = torch.Generator(device="cuda").manual_seed(1)
    B, n, hq, hk = 3, 7, 9, 2
    qkv = (torch.randn(B, n, hq + 2 * hk, 64, generator=g, device="cuda") * 2).to(dtype)
    pos0 = torch.tensor([0, 100000, -50], dtype=torch.int32, device="cuda")
    heads = qkv.transpose(1, 2)
    q, k = heads[:, :hq], heads[:, hq:hq + hk]
    qo = torch.full((B, hq, n, 64), float("nan"), dtype=dtype, device="cuda")
    ko = torch.full((B, hk, n, 64), float("nan"), dtype=dtype, device="cuda")
    before = qkv.clone()
    kvd.kvd_rope_scaled(q, k, qo, ko, rope=kvd.make_rope(**spec), pos0=pos0)
    torch.cuda.synchronize()
    assert torch.equal(qkv, before)
    pos = (pos0.cpu().numpy()[:, None].astype(np.int64) + np.arange(n))[:, None]
    check(qo, q, pos, spec)
    check(ko, k, pos, spec)


@pytest.mark.parametrize("B,n,hq,hk", [(1, 1, 1, 1), (8, 1, 32, 8), (2, 300, 20, 4),
                                       (1, 2500, 15, 5), (70, 40, 17, 0)])
def test_sizes(B, n, hq, hk):
    import kv_cached_decode_gb300 as kvd

    g = torch.Generator(device="cuda").manual_seed(B + n)
    q = torch.randn(B, hq, n, 64, generator=g, device="cuda").half()
    k = torch.randn(B, hk, n, 64, generator=g, device="cuda").half() if hk else None
    qo, ko = torch.empty_like(q), None if k is None else torch.empty_like(k)
    spec = dict(rot_dim=32)
    kvd.kvd_rope_scaled(q, k, qo, ko, rope=kvd.make_rope(**spec))
    torch.cuda.synchronize()
    pos = np.arange(n)[None, None]
    check(qo, q, pos, spec)
    if hk:
        check(ko, k, pos, spec)


def test_positions_in_place_and_back():
    import kv_cached_decode_gb300 as kvd

    B, H, n = 2, 5, 11
    x = torch.randn(B, H, n, 64, device="cuda", dtype=torch.bfloat16)
    at = torch.randint(-2000, 1 << 20, (B, n), dtype=torch.int32, device="cuda")
    spec = dict(interleaved=True, base=1000.0)
    rope = kvd.make_rope(**spec)
    y = x.clone()
    kvd.kvd_rope_scaled(k=y, k_out=y, rope=rope, positions=at)
    torch.cuda.synchronize()
    check(y, x, at.cpu().numpy().astype(np.int64)[:, None], spec)
    z = torch.empty_like(x)
    kvd.kvd_rope_scaled(y, q_out=z, rope=rope, positions=-at)
    # turned back: two roundings of a 16-bit pair
    torch.cuda.synchronize()
    err = (z.double() - x.double()).abs().max()
    assert err <= 2 * 2.0 ** -8 * 2 * x.double().abs().max()


def test_plain_form_is_the_norm_calls_rotation():
    """Halves, the whole head, no scaling: kvd_qk_norm_rope's angles, after a norm that divides
    by 1 (rows of mean square 1)."""
    import kv_cached_decode_gb300 as kvd

    x = (torch.randint(0, 2, (4, 3, 9, 64), device="cuda") * 2 - 1).half()
    pos0 = torch.tensor([0, 5, 77777, 131071], dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(x), torch.empty_like(x)
    kvd.kvd_qk_norm_rope(x, q_out=a, pos0=pos0, eps=0.0)
    kvd.kvd_rope_scaled(x, q_out=b, pos0=pos0, rope=kvd.make_rope())
    torch.cuda.synchronize()
    # fp32 roundings apart (rsqrt: 2 ulp; different products): at most one 16-bit step
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -10 * 1.5


def test_untouched_dims_keep_infinities_and_nan():
    import kv_cached_decode_gb300 as kvd

    x = torch.randn(1, 2, 3, 64, device="cuda", dtype=torch.float16)
    x[..., 40] = float("inf")
    x[..., 63] = float("nan")
    y = torch.empty_like(x)
    kvd.kvd_rope_scaled(x, q_out=y, rope=kvd.make_rope(rot_dim=32))
    torch.cuda.synchronize()
    assert torch.equal(y[..., 32:].view(torch.int16), x[..., 32:].view(torch.int16))
    assert torch.isfinite(y[..., :32]).all()


def test_many_specs_from_one_thread():
    import kv_cached_decode_gb300 as kvd

    x = torch.randn(2, 2, 5, 64, device="cuda", dtype=torch.float16)
    pos = np.arange(5)[None, None]
    for _ in range(2):
        for spec in SPECS:
            y = torch.empty_like(x)
            kvd.kvd_rope_scaled(x, q_out=y, rope=kvd.make_rope(**spec))
            torch.cuda.synchronize()
            check(y, x, pos, spec)
