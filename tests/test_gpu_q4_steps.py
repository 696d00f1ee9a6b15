"""4-bit attention where the rows' steps differ by many powers of two: what a query does not see
changes no bit of its output, and rows of little weight, or of zeros, cost the others no
precision. Compared with 64 bits over the stored values."""

import numpy as np
import pytest
import torch

import ref64
from gpu_util import new_err, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _i32(*a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _cache(k, v):
    """A one-row cache of k and v [H, cap, 64] (fp32 on the CPU), by the format's definition."""
    import kv_cached_decode_gb300 as kvd

    c = kvd.new_q4_cache(1, *k.shape[:2])
    for i, x in enumerate((k, v)):
        n, step, z = ref64.q4_quantise(x.numpy())
        c._tensors[i][0].copy_(torch.from_numpy(ref64.q4_pack(n)))
        c._tensors[2][0, ..., 2 * i:2 * i + 2].copy_(torch.from_numpy(ref64.q4_params(step, z)))
    return c


def _run(c, q, L, **kw):
    import kv_cached_decode_gb300 as kvd

    B, Hq, n, _ = q.shape
    ws = kvd.new_workspace(kvd.kvd_workspace_size(kvd.KVD_OP_Q4_ATTN, B, Hq, c.n_kv_heads, 1, n,
                                                  c.capacity))
    out, err = torch.full_like(q, 9.0), new_err()
    kvd.kvd_q4_attn(q, c, out, ws, lens=_i32(*[L] * B), dev_err=err, **kw)
    torch.cuda.synchronize()
    assert int(err) == 0
    return out


def _compare(c, q, L, **kw):
    """Every output within what the kernel's roundings allow, with s a row's V step and p its
    normalised weight:
      p s to binary16: half a step of 2^-11 of each row's share, below the normal range 2^-25
        where the largest p s of a row that is not zero stands at 2^7 or more: 2^-32 of it times
        |n - z|, for every row;
      the tensor cores add 16 products at a time, aligned by their factors' exponents, where n,
        held as n 2^-24 (half of K's as n 2^-20), counts as 2^-14: every product is cut at 2^-15
        of the largest other factor. For the output that is 16 times 2^-15 of the largest p s of
        16 positions; for a score 32 times 2^-15 (and 32 times 2^-19) of the largest |q| times
        the step of K;
      fp32: the scores (64 products), and 16 roundings of 2^-22 in the sums over n and over z,
        which are formed apart; the output's own rounding.
    A score's error counts twice: in its weight and in their sum."""
    out = _run(c, q, L, **kw)
    kd, vd, par = [t[0, :, :L].cpu().numpy() for t in c._tensors]
    k, v = (ref64.q4_values(d, par[..., a:a + 2]) for d, a in ((kd, 0), (vd, 2)))
    ks, vs = (ref64.q4_values(d, par[..., a:a + 2], size=True) for d, a in ((kd, 0), (vd, 2)))
    kstep, step = ((np.ascontiguousarray(par[..., a:a + 1]).view(np.uint16).astype(np.uint32) <<
                    16).view(np.float32).astype(np.float64) for a in (0, 2))
    grid = np.abs(v) / step                       # |n - z|
    live = np.where((vs == 0).all(-1, keepdims=True), 0.0, step)
    _, n = q.shape[1:3]
    see = ref64.visible(L, n, True, kw.get("window", 0), kw.get("n_sinks", 0))
    group = q.shape[1] // k.shape[0]
    half = ref64.HALF[q.dtype]
    tiny = 2.0 ** -25 if q.dtype == torch.float16 else 2.0 ** -134
    for hq in range(q.shape[1]):
        h = hq // group
        for i in range(n):
            at = np.flatnonzero(see[i])
            x = q[0, hq, i].double().cpu().numpy()
            s = k[h][at] @ x * 0.125
            p = np.exp(s - s.max())
            p = (p / p.sum())[:, None]
            want = (p * v[h][at]).sum(0)
            mag, size = (p * np.abs(v[h][at])).sum(0), (p * vs[h][at]).sum(0)
            smax = (ks[h][at] @ np.abs(x)).max() * 0.125
            ps = p * live[h][at]
            floor = 2.0 ** -32 * ps.max() * grid[h][at].sum(0)
            tops = [ps[at // 16 == j].max() for j in np.unique(at // 16)]
            score = 72 * 2.0 ** -24 * smax + 34 * 2.0 ** -15 * (
                np.abs(x).max() * 0.125 * kstep[h][at].max())
            tol = (mag * (2.0 ** -11 + 2 * score) + size * 16 * 2.0 ** -22 + floor +
                   16 * 2.0 ** -15 * sum(tops))
            tol = tol + half * (np.abs(want) + tol) + tiny
            off = np.abs(out[0, hq, i].double().cpu().numpy() - want)
            assert (off <= tol).all(), (hq, i, float((off / tol).max()), int((off > tol).sum()))
    return out


@pytest.mark.parametrize("up", [15, 17, 20, 30, 60, 100])
@pytest.mark.parametrize("Hq,window", [(2, 40), (8, 40), (8, 0)])
def test_rows_a_query_does_not_see_change_no_bit(up, Hq, window):
    """Finite rows with steps 2^up times the others': before the window and after the sinks inside
    tiles that are read, behind a query's position, past the length."""
    g = torch.Generator().manual_seed(up)
    k, v = (torch.randn(2, 256, 64, generator=g) for _ in "kv")
    q = torch.randn(1, Hq, 4, 64, generator=g).bfloat16().cuda()
    L, kw = 200, dict(window=window, n_sinks=2)
    clean = _compare(_cache(k, v), q, L, **kw)
    # queries stand at 196 .. 199, so a window of 40 starts at 157 .. 160
    hidden = [2, 30, 129, 155, 200, 230] if window else [200, 255]
    for rows, same in ((hidden, (0, 1, 2, 3)), ([199], (0, 1, 2)), ([197], (0,))) + (
            (([157], (1, 2, 3)), ([159], (3,))) if window else ()):
        w = v.clone()
        w[:, rows] *= 2.0 ** up
        out = _compare(_cache(k, w), q, L, **kw)
        for i in same:
            assert torch.equal(out[:, :, i], clean[:, :, i]), (rows, i)


@pytest.mark.parametrize("up", [10, 20, 30, 45, 60])
def test_rows_of_little_weight(up):
    """Rows that a query sees with a weight of about e^-32, their steps 2^up times the others'."""
    g = torch.Generator().manual_seed(up)
    q = torch.randn(1, 1, 1, 64, generator=g).bfloat16()
    k, v = (torch.randn(1, 300, 64, generator=g) for _ in "kv")
    rows = [0, 33, 64, 170, 299]
    k[:, rows] = -32 * 8 * q[0, 0, 0].float() / q[0, 0, 0].float().square().sum()
    v[:, rows] *= 2.0 ** up
    _compare(_cache(k, v), q.cuda(), 300)
    _compare(_cache(k, v), q.cuda(), 300, window=290, n_sinks=3)


@pytest.mark.parametrize("size", [1e-3, 1e-6, 1e-9, 1e-20])
def test_rows_of_zeros_beside_small_values(size):
    """A row of zeros is held with step 1: it adds nothing, whatever its weight."""
    g = torch.Generator().manual_seed(3)
    q = torch.randn(1, 3, 2, 64, generator=g).bfloat16()
    k, v = (torch.randn(1, 280, 64, generator=g) for _ in "kv")
    v *= size
    v[:, torch.rand(280, generator=g) < 0.5] = 0
    v[:, :64] = 0
    k[:, 100:110] = 3 * q[0, 0, 0].float()          # much weight on some of them
    v[:, 100:105] = 0
    for L in (280, 110, 64):
        _compare(_cache(k, v), q.cuda(), L)


@pytest.mark.parametrize("order", ["up", "down", "mixed"])
def test_steps_of_every_size(order):
    g = torch.Generator().manual_seed(7)
    q = torch.randn(1, 4, 3, 64, generator=g).bfloat16().cuda()
    k, v = (torch.randn(2, 512, 64, generator=g) for _ in "kv")
    e = torch.linspace(-90, 90, 512)
    e = {"up": e, "down": e.flip(0), "mixed": e[torch.randperm(512, generator=g)]}[order]
    c = _cache(k, v * torch.exp2(e)[None, :, None])
    for L in (5, 100, 300, 512):
        _compare(c, q, L)
    _compare(c, q, 450, window=77, n_sinks=9)


def test_weights_that_grow_and_fall_along_the_cache():
    """Scores rising and falling by hundreds, with V small where they are high."""
    g = torch.Generator().manual_seed(9)
    q = torch.randn(1, 2, 1, 64, generator=g).bfloat16()
    k, v = (torch.randn(1, 400, 64, generator=g) for _ in "kv")
    a = torch.linspace(-20, 20, 400)
    k += a[None, :, None] * q[0, 0, 0].float()
    for f in (1.0, -1.0):
        w = v * torch.exp2(-f * 2 * a)[None, :, None]
        _compare(_cache(k, w), q.cuda(), 400)
        _compare(_cache(k.flip(1), w.flip(1)), q.cuda(), 400)
