"""kvd_token_logprobs against its 64-bit form: sizes and alignments, ties, infinities and NaN,
orders that grow the list of alternatives, precision near probability 1."""

import numpy as np
import pytest
import torch

import ref64_serving as ref
from gpu_util import new_err, require_gpu

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def run(x, tokens=None, top=0, T=None, **kw):
    import kv_cached_decode_gb300 as kvd

    R = x.shape[0]
    f, i = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    out = dict(entropy=torch.full((R,), 9.0, **f), lse=torch.full((R,), 9.0, **f))
    if tokens is not None:
        out.update(logprob=torch.full(tokens.shape, 9.0, **f),
                   rank=torch.full(tokens.shape, -9, **i))
    if top:
        out.update(top_id=torch.full((R, top), -9, **i),
                   top_logprob=torch.full((R, top), 9.0, **f))
    kvd.kvd_token_logprobs(x, tokens, temperature=T, **out, **kw)
    torch.cuda.synchronize()
    return out


def check(out, x, tokens=None, top=0, T=None, skip=()):
    """fp32 sums: a weight's exponent is off by 2^-24 of its size three times (distance, product,
    ex2: 2^-22), and 2^-24 for each level of the sums, 40 at most; all relative to sums of numbers
    of one sign. The exponent's size: up to 100 bits matter (less weighs nothing)."""
    rel = 2.0 ** -22 * 4 + 40 * 2.0 ** -24 + 100 * 3 * 2.0 ** -24
    X = x.double().cpu().numpy()
    for r in range(x.shape[0]):
        if r in skip:
            continue
        t = [] if tokens is None else tokens[r].tolist()
        temp = 1.0 if T is None else float(T[r])
        lp, rank, ent, lse, ids, tlp = ref.logprobs(X[r], t, temp, top)
        near = lambda got, want: (got == want) or (  # noqa: E731
            abs(got - want) <= rel * abs(want) + 2.0 ** -120)
        got = {k: v[r].tolist() for k, v in out.items()}
        assert near(got["lse"], lse) or abs(got["lse"] - lse) <= rel * (
            abs(X[r].max() / temp) + 15), (r, got["lse"], lse)
        assert near(got["entropy"], ent), (r, got["entropy"], ent)
        if t:
            assert got["rank"] == rank, (r, got["rank"], rank)
            assert all(near(a, b) for a, b in zip(got["logprob"], lp)), (r, got["logprob"], lp)
        if top:
            assert got["top_id"] == ids, (r, got["top_id"], ids)
            assert all(near(a, b) for a, b in zip(got["top_logprob"], tlp)), (
                r, got["top_logprob"], tlp)


def tokens_for(R, m, V, seed=0):
    g = np.random.default_rng(seed)
    t = g.integers(0, V, (R, m)).astype(np.int32)
    t[g.random((R, m)) < 0.1] = -1
    return torch.from_numpy(t).cuda()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4096, 4097, 8191, 51865, 128000])
def test_sizes(dtype, V):
    for R, off, pad in ((1, 0, 0), (3, 1, 5)):
        buf = torch.randn(R * (V + pad) + off + 8, device="cuda").mul(3).to(TYPES[dtype])
        x = buf[off:off + R * (V + pad)].view(R, V + pad)[:, :V]
        t = tokens_for(R, 3, V, V)
        check(run(x, t, min(20, V)), x, t, min(20, V))


@pytest.mark.parametrize("R", [1, 2, 14, 15, 60, 300])
def test_row_counts(R):
    x = torch.randn(R, 30011, device="cuda") * 2
    t = tokens_for(R, 1, 30011, R)
    T = torch.rand(R, device="cuda") * 2 + 0.1
    check(run(x, t, 5, T), x, t, 5, T)


@pytest.mark.parametrize("m", [1, 2, 16])
@pytest.mark.parametrize("top", [0, 1, 2, 31, 32])
def test_given_and_alternatives(m, top):
    x = torch.randn(4, 20000, device="cuda").to(torch.bfloat16)  # many ties
    t = tokens_for(4, m, 20000, m)
    check(run(x, t, top), x, t, top)


@pytest.mark.parametrize("kind", ["ascending", "descending", "equal", "two", "steps", "peaks"])
@pytest.mark.parametrize("V", [3000, 100003, 400001])
def test_orders_of_the_row(kind, V):
    i = torch.arange(V, device="cuda", dtype=torch.float32)
    x = {"ascending": i / V * 20, "descending": -i / V * 20, "equal": torch.zeros(V, device="cuda"),
         "two": (i % 2) * 1.0, "steps": torch.floor(i / 4096), "peaks": (i % 64 == 5) * 30.0 + i % 3
         }[kind]
    x = x[None].repeat(20, 1)  # rows of one block each, and of clusters
    for rows in (x[:1], x):
        t = tokens_for(rows.shape[0], 2, V, 3)
        check(run(rows, t, 32), rows, t, 32)


@pytest.mark.parametrize("dtype", TYPES)
def test_infinities_and_nan(dtype):
    V = 9001
    x = torch.randn(9, V, device="cuda").to(TYPES[dtype])
    inf = float("inf")
    x[1, :] = -inf
    x[2, 5:] = -inf                 # fewer ids than alternatives
    x[3, 100], x[3, 8000] = inf, inf
    x[4, ::2] = -inf
    x[5, 4097:] = -inf
    x[6, :4097] = -inf
    x[7, 77] = inf
    x[8, 0], x[8, 1] = -0.0, 0.0    # equal
    x[8, 2:] = -5.0
    t = torch.tensor([[5, 9000, -1, 77]] * 9, dtype=torch.int32, device="cuda")
    t[3] = torch.tensor([8000, 100, 4, -1])
    t[8] = torch.tensor([0, 1, 2, 9000])
    err = new_err()
    check(run(x, t, 20, dev_err=err), x, t, 20)
    assert int(err) == 0
    for at in (0, 4000, V - 1):
        y = x.clone()
        y[:, at] = float("nan")
        err = new_err()
        check(run(y, t, 20, dev_err=err), y, t, 20)
        assert int(err) == 19


def test_near_probability_one_and_far_ids():
    x = torch.full((3, 50000), -30.0, device="cuda")
    x[0, 123] = 10.0
    x[1, 123], x[1, 49999] = 10.0, -8.0
    x[2, 123] = 100.0               # the others weigh 2^-187: nothing is lost but that
    t = torch.tensor([[123, 7]] * 3, dtype=torch.int32, device="cuda")
    check(run(x[:2], t[:2], 3), x[:2], t[:2], 3)
    out = run(x, t, 3)
    assert out["logprob"][2].tolist() == [-0.0, -130.0]
    small = torch.tensor([0.01, 1.0, 1e-30], device="cuda")
    got = run(x, t, 3, small)
    check(got, x, t, 3, small, skip=(0, 2))
    assert got["logprob"][2, 0] == 0 and got["top_id"][2, 0] == 123
    large = torch.full((3,), 1e30, device="cuda")
    check(run(x, t, 3, large), x, t, 3, large)


def test_bad_tokens_and_temperatures():
    x = torch.randn(4, 5000, device="cuda")
    t = torch.tensor([[1], [-2], [5000], [4999]], dtype=torch.int32, device="cuda")
    err = new_err()
    out = run(x, t, 4, dev_err=err)
    assert int(err) == 18
    assert out["rank"][1] == -1 and out["logprob"][2] == 0
    check(out, x, t, 4, skip=(1, 2))
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        T = torch.ones(4, device="cuda")
        T[2] = bad
        t = tokens_for(4, 1, 5000)
        err = new_err()
        out = run(x, t, 4, T, dev_err=err)
        assert int(err) == 21
        check(out, x, t, 4, T, skip=(2,))
        assert out["entropy"][2] == 9 and out["rank"][2] == -9 and (out["top_id"][2] == -9).all()


def test_any_subset_of_outputs():
    import kv_cached_decode_gb300 as kvd

    x = torch.randn(2, 7000, device="cuda")
    t = tokens_for(2, 3, 7000)
    full = run(x, t, 6)
    for names in (["entropy"], ["lse"], ["logprob"], ["rank"], ["top_id"], ["top_logprob"],
                  ["rank", "top_logprob"]):
        out = {n: torch.empty_like(full[n]) for n in names}
        kvd.kvd_token_logprobs(x, t if {"logprob", "rank"} & set(names) else None, **out)
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], full[n]) for n in names)


def test_the_same_bits_on_every_run_and_captured():
    x = torch.randn(3, 128000, device="cuda").to(torch.bfloat16)
    t = tokens_for(3, 1, 128000)
    first = run(x, t, 20)
    for _ in range(4):
        again = run(x, t, 20)
        assert all(torch.equal(first[k], again[k]) for k in first)
    import kv_cached_decode_gb300 as kvd

    out = {k: torch.empty_like(v) for k, v in first.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvd.kvd_token_logprobs(x, t, **out)
    for _ in range(2):
        for v in out.values():
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(first[k], out[k]) for k in first)
