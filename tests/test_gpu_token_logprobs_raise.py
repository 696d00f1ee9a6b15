"""kvd_token_logprobs where the largest logit grows along the row, far from 0: what was summed up
relative to one reference is carried over to the next, whose product with log2 e / T is rounded."""

import pytest
import torch

from gpu_util import require_gpu
from test_gpu_token_logprobs import TYPES, check, run, tokens_for

pytestmark = pytest.mark.gpu
V = 20000  # several rounds of a block


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("offset", [0.0, 100.0, -1000.0, 3e4, -2e5, 1e6, -5e6])
@pytest.mark.parametrize("kind", ["ascending", "late", "steps"])
@pytest.mark.parametrize("R", [16, 700])  # rows of a cluster, rows of one block
def test_a_reference_that_moves(offset, kind, R):
    g = torch.Generator(device="cuda").manual_seed(5)
    if kind == "ascending":
        x = (torch.randn(R, V, generator=g, device="cuda") * 2).sort(1).values
    elif kind == "late":  # one id behind the first round weighs a little more than all before it
        x = torch.randn(R, V, generator=g, device="cuda")
        x[:, 15000] = torch.linspace(5.0, 12.0, R, device="cuda")
    else:  # each round a step above the one before
        x = torch.floor(torch.arange(V, device="cuda") / 4096.0).repeat(R, 1) * 0.5
    x = x + offset
    T = torch.linspace(0.4, 2.0, R, device="cuda")
    t = tokens_for(R, 2, V, 6)
    out = run(x, t, 3, T)
    some = slice(0, R, R // 16)
    check({k: v[some] for k, v in out.items()}, x[some], t[some], 3, T[some])


@pytest.mark.parametrize("dtype", TYPES)
def test_each_type(dtype):
    x = (torch.randn(12, V, device="cuda") * 40 - 1000).to(TYPES[dtype])
    x = x.sort(1).values
    T = torch.linspace(5.0, 40.0, 12, device="cuda")
    t = tokens_for(12, 2, V, 7)
    check(run(x, t, 3, T), x, t, 3, T)
