"""kvd_sample_filtered against its 64-bit form: token and number of kept ids are equal,
log-probabilities within fp32 rounding."""

import numpy as np
import pytest
import torch

import ref64
from gpu_util import new_err, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _draw(x, u, T=None, k=None, p=None, m=None, flags=0):
    import kv_cached_decode_gb300 as kvd

    B = x.shape[0]
    f = lambda v, t=torch.float32: None if v is None else torch.tensor(  # noqa: E731
        np.broadcast_to(np.asarray(v), (B,)).copy(), dtype=t, device="cuda")
    tok = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((B,), 7.0, device="cuda")
    n = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    err = new_err()
    kvd.kvd_sample_filtered(x, f(u), tok, temperature=f(T), top_k=f(k, torch.int32), top_p=f(p),
                            min_p=f(m), logprob=lp, n_kept=n, dev_err=err, flags=flags)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), lp.cpu().numpy(), n.cpu().numpy(), int(err)


def _check(x, u, T=None, k=None, p=None, m=None, want_err=0):
    tok, lp, n, err = _draw(x, u, T, k, p, m)
    assert err == want_err
    B = x.shape[0]
    xs = x.cpu().numpy()
    at = lambda v, b, d: d if v is None else np.broadcast_to(np.asarray(v), (B,))[b]  # noqa: E731
    f = lambda v: float(np.float32(v))  # noqa: E731
    for b in range(B):
        w = ref64.sample(xs[b], f(at(u, b, 0)), f(at(T, b, 1.0)), int(at(k, b, 0)),
                         f(at(p, b, 1.0)), f(at(m, b, 0.0)))
        assert tok[b] == w[0] and n[b] == w[2], (b, (tok[b], n[b]), w)
        # the log of a quotient rounded to fp32, itself within 2 units; weights 2^-31 each
        if np.isfinite(w[1]):
            assert abs(lp[b] - w[1]) <= 2.0 ** -21 * abs(w[1]) + 2.0 ** -30, (b, lp[b], w[1])
            if w[1] < -0.7:
                assert abs(lp[b] - w[1]) <= 2.0 ** -22 * (1 + abs(w[1]))
        else:
            assert lp[b] == w[1]
    return tok


PARAMS = [dict(), dict(T=0.7), dict(k=50), dict(p=0.9), dict(m=0.05), dict(T=0.8, k=50, p=0.9),
          dict(T=1.3, k=40, p=0.95, m=0.02), dict(T=0.0, k=5), dict(k=1), dict(p=0.0), dict(p=1e-6),
          dict(T=3.0, p=0.99), dict(T=0.01, k=100, p=0.999), dict(k=10 ** 6), dict(m=1.0),
          dict(m=1e-20), dict(T=100.0, p=0.5)]


@pytest.mark.parametrize("V", [1, 2, 33, 512, 1000, 8191, 8193, 16385, 51865, 131072])
def test_vocabularies_and_parameters(V):
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(len(PARAMS), V, generator=g, device="cuda") * 3
    u = torch.rand(len(PARAMS), generator=g, device="cuda").cpu().numpy()
    d = dict(T=1.0, k=0, p=1.0, m=0.0)
    rows = {n: [q.get(n, d[n]) for q in PARAMS] for n in d}
    _check(x, u, **rows)
    _check(torch.randn(3, V, generator=g, device="cuda"), [0.0, 0.5, 1 - 2.0 ** -24])


def test_the_largest_vocabulary_and_a_large_batch():
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(4, 524288, generator=g, device="cuda") * 2.5
    _check(x, [0.1, 0.9, 0.5, 0.3], T=[1, 0.7, 2.0, 1], k=[0, 1000, 0, 30000],
           p=[0.95, 1, 0.8, 0.9], m=[0, 0, 0, 1e-3])
    x = torch.randn(300, 5003, generator=g, device="cuda") * 2.5
    _check(x, np.linspace(0, 0.999, 300), T=np.linspace(0.2, 2, 300),
           k=np.arange(300) * 3, p=np.linspace(0.3, 1, 300))


@pytest.mark.parametrize("V", [700, 20000, 100000])
def test_ties(V):
    """Logits rounded to 8 bits, constants, two values: cuts among equal logits fall by id."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(8, V, generator=g, device="cuda") * 2
    x[:4] = x[:4].bfloat16().float()
    x[4] = 1.25
    x[5] = torch.where(torch.rand(V, generator=g, device="cuda") < 0.5, 0.0, -0.0)
    x[6] = torch.where(torch.rand(V, generator=g, device="cuda") < 0.3, 2.0, 1.0)
    x[7] = (torch.arange(V, device="cuda") % 7).float()
    u = np.array([0.1, 0.99, 0.5, 0.7, 0.25, 0.25, 0.6, 0.9])
    _check(x, u, k=[50, 200, V // 2, 0, V // 3, 177, V // 2, 129])
    _check(x, u, p=[0.5, 0.9, 0.99, 0.3, 0.5, 0.25, 0.75, 0.9])
    _check(x, u, k=[50, 200, V // 2, 600, V // 3, 177, V // 2, 500],
           p=[0.5, 0.9, 0.99, 0.3, 0.5, 0.25, 0.75, 0.9])
    _check(x, u, m=0.5)


def test_masked_logits():
    """Rows of -inf, of the type's lowest value, +inf, NaN."""
    g = torch.Generator(device="cuda").manual_seed(4)
    V = 30000
    x = torch.randn(10, V, generator=g, device="cuda")
    keep = torch.rand(V, generator=g, device="cuda") < 0.001
    x[0, ~keep] = float("-inf")
    x[1] = float("-inf")
    x[2, ~keep] = torch.finfo(torch.float32).min
    x[3] = torch.finfo(torch.float32).min
    x[4, 777] = x[4, 20001] = float("inf")
    x[5] = float("-inf")
    x[5, V - 1] = -3e38
    x[6, 5:] = float("-inf")
    x[7] *= 1e37
    x[8] *= 1e-37
    u = np.linspace(0.05, 0.95, 10)
    for kw in (dict(), dict(k=3), dict(p=0.7), dict(k=1000, p=0.99, m=0.01), dict(T=0.0),
               dict(T=1e-30), dict(T=1e30)):
        _check(x, u, **kw)
    x[9, 4] = float("nan")
    x[9, 100] = float("nan")
    _check(x, u, k=20, want_err=19)
    x[9] = float("nan")
    _check(x, u, want_err=19)


def test_parameters_out_of_range_leave_the_row():
    x = torch.randn(8, 1000, device="cuda")
    nan, inf = float("nan"), float("inf")
    tok, lp, n, err = _draw(x, [0.5, 0.5, 0.5, 0.5, 0.5, nan, 0.5, 0.5],
                            T=[-1, nan, inf, 1, 1, 1, 1, 0], p=[1, 1, 1, nan, 1, 1, 1, 0.5],
                            m=[0, 0, 0, 0, nan, 0, 0, 0])
    assert err == 21
    assert (tok[:6] == -7).all() and (lp[:6] == 7).all() and (n[:6] == -7).all()
    assert (tok[6:] >= 0).all() and tok[7] == int(x[7].argmax())


def test_strided_rows_streams_graphs_and_repeats():
    import kv_cached_decode_gb300 as kvd

    g = torch.Generator(device="cuda").manual_seed(9)
    big = torch.randn(6, 40007, generator=g, device="cuda") * 3
    x = big[:, 3:40000]
    u = np.linspace(0.1, 0.9, 6)
    want = _check(x, u, k=100, p=0.9)
    _check(big[::2, 1:], u[::2], T=0.9, p=0.9)
    tok = torch.zeros(6, dtype=torch.int32, device="cuda")
    ud = torch.tensor(u, dtype=torch.float32, device="cuda")
    k = torch.full((6,), 100, dtype=torch.int32, device="cuda")
    p = torch.full((6,), 0.9, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        kvd.kvd_sample_filtered(x, ud, tok, top_k=k, top_p=p, stream=side)
        side.synchronize()
        assert (tok.cpu().numpy() == want).all()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvd.kvd_sample_filtered(x, ud, tok, top_k=k, top_p=p, flags=kvd.KVD_FLAG_PDL)
    tok.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert (tok.cpu().numpy() == want).all()


def test_frequencies():
    """20000 evenly spaced uniforms draw the kept distribution."""
    V, N = 50, 20000
    x = torch.linspace(2, -3, V, device="cuda")[None].repeat(N, 1).contiguous()
    u = (np.arange(N) + 0.5) / N
    tok, _, n, _ = _draw(x, u, k=20, p=0.9)
    w = np.exp(np.linspace(2, -3, V))[:n[0]]
    freq = np.bincount(tok, minlength=V)[:n[0]] / N
    # evenly spaced uniforms: every frequency within 2 draws of its probability
    assert np.abs(freq - w / w.sum()).max() <= 2.0 / N and tok.max() < n[0]


@pytest.mark.parametrize("V", [700, 40000])
@pytest.mark.parametrize("logm", [0.01, 6.4, 6.6, 7.9, 8.1, 12.0, 14.4, 14.6, 15.1, 15.9, 16.1, 24.0,
                                  39.9, 40.1])
def test_min_p_where_its_forms_change(V, logm):
    """min_p = 2^-logm: what it drops is only added up below 2^-14.5, listed or weighed above."""
    g = torch.Generator(device="cuda").manual_seed(int(10 * logm))
    x = torch.randn(6, V, generator=g, device="cuda") * 3.0
    u = torch.rand(6, generator=g, device="cuda").cpu().numpy()
    for p in (0.3, 0.9, 0.999, 1.0):
        _check(x, u, m=2.0 ** -logm, p=p)
        _check(x, u, m=2.0 ** -logm, p=p, k=300, T=0.9)


@pytest.mark.parametrize("V", [5, 700, 40000])
def test_min_p_above_one_keeps_one_id(V):
    """No weight is above 1, so nothing passes and the one id that is always kept is the first of
    the order: the lowest of those tied for the largest logit. At 1 all of these stay."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(5, V, generator=g, device="cuda").clamp(max=1.0)
    first = torch.tensor([0, 1, V // 3, V - 3, 2], device="cuda")
    for b in range(5):
        x[b, first[b]:first[b] + 3] = 1.5
    x[4, 2:5] = float("inf")
    u = [0.0, 0.3, 0.6, 0.999, 0.5]
    for m in (np.nextafter(np.float32(1), np.float32(2)), 1.5, 1e30, np.inf):
        for kw in (dict(), dict(p=0.9), dict(k=3), dict(k=2, p=0.5), dict(T=0.3)):
            tok, lp, n, err = _draw(x, u, m=m, **kw)
            assert err == 0 and (n == 1).all() and (lp == 0).all()
            assert (tok == first.cpu().numpy()).all(), (m, kw)
    _, lp, n, _ = _draw(x, u, m=1.0)
    ties = (x == x.max(1, keepdim=True).values).sum(1).cpu().numpy()
    assert (ties >= 3).all() and (n == ties).all() and np.allclose(lp, -np.log(ties))


@pytest.mark.parametrize("V", [600, 30000])
@pytest.mark.parametrize("T", [0.3, 1.0, 7.0])
def test_the_logprob_of_a_drawn_id_of_little_weight(V, T):
    """u = 0 draws the first kept id, whatever its weight (2^-16 down to 2^-44 of the largest)."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(24, V, generator=g, device="cuda") * T
    x[:, V // 2] = x.max() + 3 * T
    x[:, 0] = x[:, V // 2] - T * torch.linspace(11.2, 30.4, 24, device="cuda")
    for kw in (dict(), dict(k=min(V - 1, 20000)), dict(k=100) if V == 600 else dict(p=1.0)):
        _check(x, np.zeros(24), T=T, **kw)
    few = torch.full((24, V), float("-inf"), device="cuda")
    few[:, 0], few[:, 5:9] = x[:, 0], x[:, V // 2:V // 2 + 1]
    _check(few, np.zeros(24), T=T, k=4)
    _check(few, np.zeros(24), T=T, k=5)
    _check(few, np.zeros(24), T=T)


@pytest.mark.parametrize("min_p", [1e-30, 1e-13, 2.0 ** -40, 1e-9, 1e-6, 2.0 ** -14 * 0.99, 2.0 ** -14,
                                   0.02])
@pytest.mark.parametrize("T", [0.3, 1.0, 40.0])
def test_how_many_ids_pass_min_p(min_p, T):
    """Thousands of logits within 1e-4 of the border, a few units of fp32 apart: the count is that
    of 64 bits."""
    V = 20000
    g = torch.Generator(device="cuda").manual_seed(3)
    m = torch.tensor([0.0, 3.75, -700.0], dtype=torch.float64, device="cuda")[:, None]
    edge = T * float(np.log(np.float64(np.float32(min_p))))
    at = edge * (1 + 1e-4 * (2 * torch.rand(3, V, generator=g, device="cuda",
                                            dtype=torch.float64) - 1))
    x = (m + at).float()
    x[:, 77] = m[:, 0].float()
    u = np.array([0.01, 0.5, 0.9])
    T = float(np.float32(T))
    for kw in (dict(), dict(k=V - 5), dict(p=0.9999999), dict(k=100)):
        _check(x, u, T=T, m=min_p, **kw)
    few = torch.full((3, V), float("-inf"), device="cuda")
    few[:, 50:150] = x[:, 50:150]
    _check(few, u, T=T, m=min_p, k=99)
    _check(few, u, T=T, m=min_p)
