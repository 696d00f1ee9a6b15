"""Plain 64-bit forms of the scaled rotations, the packed batch over a paged cache and token log
probabilities, and the error bounds the GPU tests hold the kernels to. numpy/torch only."""

import math

import numpy as np
import torch

import ref64


def theta(base=10000.0, rot_dim=64, scaling="none", factor=1.0, original_len=0, low=1.0, high=1.0,
          **_):
    """Frequencies of a rotation, a pair at a time, from the header's definitions (its floats)."""
    f = lambda v: float(np.float32(v))  # noqa: E731
    base, factor, low, high = f(base), f(factor), f(low), f(high)
    out = []
    for i in range(rot_dim // 2):
        t = base ** (-2.0 * i / rot_dim)
        s = 1.0
        if scaling == "linear":
            s = 0.0
        elif scaling == "bands":
            s = (original_len * t / (2 * math.pi) - low) / (high - low)
        elif scaling == "ramp":
            def pair(r):
                return rot_dim * math.log(original_len / (2 * math.pi * r)) / (2 * math.log(base))
            a, b = max(0, math.floor(pair(high))), min(rot_dim - 1, math.ceil(pair(low)))
            s = 1 - (i - a) / max(b - a, 0.001)
        s = min(1.0, max(0.0, s))
        out.append(t * (s + (1 - s) / factor) if scaling != "none" else t)
    return np.array(out)


def rotate(x, pos, spec):
    """x [..., 64] float64 (numpy) at integer positions pos (broadcast); returns the values and
    the size |a| + |b| (times the magnitude) that an output's rounding scales with."""
    rot, inter = spec.get("rot_dim", 64), spec.get("interleaved", False)
    mag = float(np.float32(spec.get("magnitude", 1.0)))
    a = np.asarray(pos, np.float64)[..., None] * theta(**spec)
    c, s = np.cos(a) * mag, np.sin(a) * mag
    h = rot // 2
    lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, h), slice(h, rot))
    y, size = x.copy(), np.abs(x)
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    size[..., lo] = size[..., hi] = (np.abs(x[..., lo]) + np.abs(x[..., hi])) * abs(mag)
    return y, size


def rotation_bound(want, size, dtype, pos_max):
    """Roundings of cos, sin, their products and sum: 8 of 2^-24 of the pair's size (sincospi: 2
    ulp, the magnitude, two products); the angle: 2^-31 of half a turn from the fixed-point
    fraction's 32 bits and pos * 2^-52 turns from the frequency's 53; then the output's own."""
    err = size * (8 * 2.0 ** -24 + math.pi * 2.0 ** -30 + 2 * math.pi * abs(pos_max) * 2.0 ** -51)
    return err + ref64.HALF[dtype] * (np.abs(want) + err) + 2.0 ** -24


def paged_rows(k, v, table, b, length):
    """K and V of row b's first `length` positions, [heads, length, 64] float64; pages of the
    table outside the pool are zeros."""
    ps = k.shape[2]
    out = []
    for t in (k, v):
        rows = []
        for i in range(-(-length // ps)):
            pg = int(table[b, i])
            rows.append(t[pg].double() if 0 <= pg < t.shape[0] else torch.zeros_like(t[0]).double())
        out.append(torch.cat(rows, 1)[:, :length])
    return out


def chunk_attention(q, k, v, scale):
    """q [n, hq, 64], the last n of k's positions; k, v [hk, T, 64]; all float64. Output [n, hq,
    64], and for the bound sum p |v|, the largest sum |scale q_d k_d| and 2^-25 sum |v| / sum of
    weights relative to the largest (what binary16 weights lose below their range)."""
    n, hq, _ = q.shape
    hk, T, _ = k.shape
    g = hq // hk
    qq = q.reshape(n, hk, g, 64)
    hide = torch.arange(T, device=q.device)[None] > torch.arange(T - n, T, device=q.device)[:, None]
    s = torch.einsum("nhgd,htd->nhgt", qq, k) * scale
    s = s.masked_fill(hide[:, None, None], -math.inf)
    e = torch.exp(s - s.max(-1, keepdim=True).values)
    z = e.sum(-1, keepdim=True)
    out = torch.einsum("nhgt,htd->nhgd", e / z, v)
    mag = torch.einsum("nhgt,htd->nhgd", e / z, v.abs())
    size = (torch.einsum("nhgd,htd->nhgt", qq.abs(), k.abs()) * abs(scale)).masked_fill(
        hide[:, None, None], 0).max(-1, keepdim=True).values
    low = 2.0 ** -25 * torch.einsum("nt,htd->nhd", (~hide).double(), v.abs())[:, :, None] / z
    return [t.reshape(n, hq, -1) for t in (out, mag, size, low)]


def logprobs(x, tokens, T=1.0, top=0):
    """One row in 64 bits: (logprob, rank per token, entropy, lse, top ids, top logprobs)."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    order = np.lexsort((np.arange(len(x)), -x))
    place = np.empty(len(x), np.int64)
    place[order] = np.arange(len(x))
    m = x.max()
    if m == -np.inf:
        return ([-np.inf if t >= 0 else 0.0 for t in tokens],
                [int(place[t]) if t >= 0 else -1 for t in tokens], 0.0, -np.inf, [-1] * top,
                [-np.inf] * top)
    with np.errstate(invalid="ignore"):
        d = np.where(x == m, 0.0, (x - m) / np.float64(T))
    w = np.exp(d)
    n = int((x == m).sum())
    log_s = np.log1p(w[x != m].sum()) if n == 1 else np.log(n + w[x != m].sum())
    lp = np.where(d == -np.inf, -np.inf, d - log_s)
    ent = log_s - (w[w > 0] * d[w > 0]).sum() / (n + w[x != m].sum())
    live = order[:top][x[order[:top]] > -np.inf]
    ids = list(live) + [-1] * (top - len(live))
    return ([lp[t] if t >= 0 else 0.0 for t in tokens],
            [int(place[t]) if t >= 0 else -1 for t in tokens], ent, m / T + log_s, ids,
            [lp[i] if i >= 0 else -np.inf for i in ids])
