"""kvd_token_logprobs where the largest logit seen so far, times log2 e / T, is far from 0 or past
fp32: masks of any size in a part of a row or all of it, temperatures close to 0."""

import pytest
import torch

import ref64_serving as ref
from gpu_util import require_gpu
from test_gpu_token_logprobs import TYPES, check, run, tokens_for

pytestmark = pytest.mark.gpu
V = 20000  # several rounds of a block


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def check_far(out, x, tokens, top, T):
    """As check, for outputs that may be past fp32: from -2^128 (1 - 2^-25) on, the middle between
    its lowest value and what would be the next, the rounding to fp32 is -inf. There the output is
    held to that, and check gets the value in 64 bits in its place."""
    lowest = -2.0 ** 128 * (1 - 2.0 ** -25)
    out = {k: v.double() if v.dtype == torch.float32 else v for k, v in out.items()}
    for r in range(x.shape[0]):
        lp, _, _, lse, _, tlp = ref.logprobs(x[r].double().cpu().numpy(), tokens[r].tolist(),
                                             float(T[r]), top)
        for name, want in (("lse", lse), ("logprob", lp), ("top_logprob", tlp)):
            want = torch.tensor(want, dtype=torch.float64, device=x.device)
            past = (want <= lowest) & want.isfinite()
            assert (out[name][r][past] == -float("inf")).all(), (r, name)
            out[name][r] = torch.where(past, want, out[name][r])
    check(out, x, tokens, top, T)


def temperatures(n, lo=0.4, hi=2.0):
    """n of them, so that rounding goes either way in the products with them."""
    return torch.linspace(lo, hi, n, device="cuda")


@pytest.mark.parametrize("fill", [-1e4, -1e9, -3e9, -1e10, -7e10, -1e20, -1e30, -1e37, -3.3e38,
                                  1e10, 1e30])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R", [24, 700])  # rows of a cluster, rows of one block
def test_rows_with_a_mask(fill, dtype, R):
    """All of a row; its first 9000 ids; all but one id; every other id."""
    x = torch.randn(R, V, device="cuda") * 3
    x[0::4] = fill
    x[1::4, :9000] = fill
    x[2::4, :4096] = fill
    x[2::4, 4097:] = fill
    x[3::4, ::2] = fill
    x = x.to(TYPES[dtype])
    T = temperatures(R)
    t = tokens_for(R, 2, V, 1)
    some = slice(0, 24)  # the 64-bit form takes a while
    out = run(x, t, 5, T)
    check_far({k: v[some] for k, v in out.items()}, x[some], t[some], 5, T[some])
    assert torch.isfinite(out["entropy"]).all() and not out["logprob"].isnan().any()


@pytest.mark.parametrize("big", [-3e9, -1e10, -3e10, 5e9, 1e10])
def test_neighbours_that_still_weigh(big):
    """Logits some steps of fp32 apart, under a temperature that leaves them weights."""
    R = 16
    x = torch.full((R, V), big, device="cuda")
    low = torch.nextafter(x, torch.full_like(x, -float("inf")))
    x[:, 1::3] = low[:, 1::3]
    x[:, 2::3] = torch.nextafter(low, torch.full_like(x, -float("inf")))[:, 2::3]
    for T in (temperatures(R), temperatures(R, 150.0, 900.0)):
        t = tokens_for(R, 2, V, 2)
        check(run(x, t, 3, T), x, t, 3, T)


@pytest.mark.parametrize("top", [0, 1, 4])
def test_the_lowest_values_of_fp32(top):
    """Logits below 0 whose product with log2 e / T is past fp32, not all of them equal."""
    x = torch.full((6, V), torch.finfo(torch.float32).min, device="cuda")
    x[0, 5] = -3e38
    x[1, 9000:9100] = -3.2e38
    x[2, V - 1] = -2.9e38
    x[3] = torch.linspace(-3.4e38, -2.5e38, V, device="cuda")
    x[4] = torch.linspace(-2.5e38, -3.4e38, V, device="cuda")
    t = tokens_for(6, 2, V, 3)
    for R in (slice(0, 1), slice(0, 6)):
        check(run(x[R], t[R], top), x[R], t[R], top)


@pytest.mark.parametrize("dtype", TYPES)
def test_temperatures_close_to_0(dtype):
    R = 8
    x = (-5 - torch.rand(R, V, device="cuda")).to(TYPES[dtype])
    T = torch.tensor([2e-38, 2.1e-38, 2.4e-38, 3e-38, 1e-37, 1e-36, 1e-30, 1e-20], device="cuda")
    t = tokens_for(R, 2, V, 4)
    out = run(x, t, 3, T)
    check(out, x, t, 3, T)
    best = (x == x.amax(1, keepdim=True)).sum(1).double().log()
    assert ((out["entropy"].double() - best).abs() < 1e-5).all()
