"""Plain 64-bit forms of the head norm with rotation, windowed attention and the 4-bit cache,
and the error bounds the GPU tests hold the kernels to. numpy/torch on the CPU only."""

import numpy as np
import torch

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def visible(length, qlen, causal=True, window=0, sinks=0):
    """[qlen, length] of bool: what query i of a block ending at `length` sees."""
    p = length - qlen + np.arange(qlen)[:, None]
    t = np.arange(length)[None, :]
    if not causal:
        return np.ones((qlen, length), bool)
    see = t <= p
    if window > 0:
        see &= (t < sinks) | (t > p - window)
    return see


def attention(q, k, v, see, scale, kmag=None):
    """q [Hq, n, 64], k and v [Hk, T, 64], see [n, T], all float64 (torch). Returns the output
    and, for the bounds, sum_t p_t |v_t| and the largest sum_d |scale q_d| kmag_d seen (kmag:
    the size of what a kernel adds up for k, |k| without one). Only what a query sees enters
    its sums, whatever lies elsewhere."""
    kmag = k.abs() if kmag is None else kmag
    hq, n, _ = q.shape
    hk = k.shape[0]
    out = torch.zeros(hq, n, 64, dtype=torch.float64)
    mag = torch.zeros_like(out)
    smax = torch.zeros(hq, n, 1, dtype=torch.float64)
    for i in range(n):
        at = torch.from_numpy(np.flatnonzero(see[i]))
        if len(at) == 0:
            continue
        for h in range(hq):
            kk, vv = k[h // (hq // hk)][at], v[h // (hq // hk)][at]
            s = (kk @ q[h, i]) * scale
            p = torch.exp(s - s.max())
            p = p / p.sum()
            out[h, i] = p @ vv
            mag[h, i] = p @ vv.abs()
            smax[h, i] = ((kmag[h // (hq // hk)][at] @ q[h, i].abs()) * abs(scale)).max()
    return out, mag, smax


def attention_bound(want, mag, smax, dtype, weights=None, floor=0.0):
    """Largest error of a 16-bit output: its own rounding; the weights' rounding to 16 bits
    (half a step each in the products, and once more in a normaliser of rounded weights);
    fp32 scores (64 products and sums, at most 72 roundings of 2^-24 of smax, twice: weight
    and normaliser) and 16 roundings in weights and sums; `floor`: an absolute term."""
    h = HALF[dtype]
    w = HALF[weights or dtype]
    f32 = 2.0 * 72 * 2.0 ** -24 * smax + 16 * 2.0 ** -22
    err = mag * (2 * w + f32) + floor
    return err + h * (want.abs() + err) + 2.0 ** -24  # the last: subnormal binary16 outputs


def bf16_round(x):
    """float32 -> nearest bfloat16 (ties to even), as float32; finite inputs."""
    u = np.asarray(x, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


@np.errstate(over="ignore")
def q4_quantise(x):
    """The 4-bit format of finite rows x [..., 64] (float32): n (int), step, zero point."""
    x = np.asarray(x, np.float32)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    step = bf16_round((np.float32(0.5) * hi - np.float32(0.5) * lo) / np.float32(7.5))
    flat = step == 0
    one = bf16_round(np.abs(lo) / np.float32(15))
    one = np.where(one == 0, np.float32(1), one)
    z = (-lo / np.where(flat, np.float32(1), step)).astype(np.float16).astype(np.float32) + 0
    z = np.where(flat, np.where(lo < 0, np.float32(15), np.float32(0)), z)
    step = np.where(flat, one, step)
    n = np.clip(np.rint(x / step + z), 0, 15)
    return n.astype(np.int64), step.astype(np.float32), z.astype(np.float32)


def q4_pack(n):
    n = n.astype(np.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def q4_params(step, z):
    """[..., 1] float32 step and zero point -> [..., 2] int16 bits."""
    s = (np.asarray(step, np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return np.concatenate([s, np.asarray(z, np.float16).view(np.uint16)], -1).view(np.int16)


def q4_values(data, params, size=False):
    """Stored rows -> float64 values step * (n - z), or with `size` step * (n + |z|). data
    [..., 32] uint8, params [..., 2] int16 bits."""
    n = np.empty((*data.shape[:-1], 64))
    n[..., 0::2] = data & 15
    n[..., 1::2] = data >> 4
    u = np.ascontiguousarray(params).view(np.uint16)
    step = (u[..., 0:1].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    z = np.ascontiguousarray(u[..., 1:2]).view(np.float16).astype(np.float64)
    with np.errstate(invalid="ignore"):
        return step * (n + np.abs(z)) if size else step * (n - z)


def norm_rope(x, w, pos, eps, base):
    """x [B, H, n, 64] float64, w [64] or None, pos [B, n] int; returns the values and the
    bound's scale |y_i| + |y_{i+32}| of each output."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * w
    a, b = y[..., :32], y[..., 32:]
    mag = np.concatenate([np.abs(a) + np.abs(b)] * 2, -1)
    if base == 0:
        return y, mag
    theta = np.float64(np.float32(base)) ** (-np.arange(32) / 32.0)
    t = pos[:, None, :, None].astype(np.float64) * theta
    c, s = np.cos(t), np.sin(t)
    return np.concatenate([a * c - b * s, b * c + a * s], -1), mag


def sample(x, u, T=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """One row of kvd_sample_filtered in 64 bits: (token, logprob, n_kept)."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    order = np.lexsort((np.arange(len(x)), -x))
    order = order[x[order] > -np.inf]
    if len(order) == 0:
        return -1, -np.inf, 0
    if T == 0:
        return int(order[0]), 0.0, 1
    y = x[order]
    with np.errstate(invalid="ignore", over="ignore"):
        d = np.where(y == y[0], 0.0, (y - y[0]) / np.float64(T))
    if top_k > 0:
        order, d = order[:top_k], d[:top_k]
    w = np.exp(d)
    keep = len(w)
    if top_p < 1:
        c = np.cumsum(w)
        keep = min(keep, max(1, int((c - w < np.float64(top_p) * c[-1]).sum())))
    if min_p > 0:
        keep = min(keep, max(1, int((w >= min(1.0, np.float64(min_p))).sum())))
    ids, w = order[:keep], w[:keep]
    at = np.argsort(ids)
    ids, w = ids[at], w[at]
    c = np.cumsum(w)
    over = np.flatnonzero(c > np.float64(u) * c[-1])
    i = int(over[0]) if len(over) else int(np.flatnonzero(w > 0)[-1])
    rest = np.delete(w, i).sum()
    lp = np.log1p(-rest / c[-1]) if w[i] > c[-1] / 2 else np.log(w[i] / c[-1])
    return int(ids[i]), float(lp), keep
