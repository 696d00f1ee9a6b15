"""Cases of the decoder-step operators: each as its plain form in elementary torch
operations and as the calls a user of the library makes.

Four groups: the norm of queries and keys with the rotation (``norm_rope``), attention
with a sliding window and sinks over a 16-bit cache (``window``, ``window_prefill``), the
4-bit cache (``q4_prompt``: append and read back; ``q4_attn``: attention), and sampling
with temperature, top-k, top-p and min-p (``sample``).
"""

import math

import numpy as np
import torch

own = False  # True: the library's calls; False: the plain forms

D = 64  # head size of the library
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases ------------
def listed():
    return [
        # one decode step of 8 sequences deep in their context: q and k heads of a fused
        # QKV projection
        dict(name="norm_rope_step", op="norm_rope", dtype="bf16", batch=8, n=1, hq=32, hk=8,
             far=32768),
        # a prompt chunk of 4 sequences
        dict(name="norm_rope_prompt", op="norm_rope", dtype="f16", batch=4, n=4096, hq=32, hk=8,
             far=8192),
        # one sequence, grouped heads, a step far past the window
        dict(name="window_step_1", op="window", dtype="f16", batch=1, hq=20, hk=4, qlen=1,
             len=32767, window=1024, sinks=4),
        # a batch of plain multi-head rows of ragged length, odd window
        dict(name="window_step_32", op="window", dtype="bf16", batch=32, hq=20, hk=20, qlen=1,
             len=8191, window=2047, sinks=5),
        # a speculative block of 5 tokens on grouped heads
        dict(name="window_verify_8", op="window", dtype="f16", batch=8, hq=32, hk=8, qlen=5,
             len=16384, window=4096, sinks=16),
        # a long prompt through a windowed layer
        dict(name="window_prefill", op="window_prefill", dtype="bf16", batch=1, hq=20, hk=4,
             n=8192, prefix=0, window=1024, sinks=4),
        # a ragged prompt batch written to the 4-bit cache and read back in 16 bits
        dict(name="q4_prompt", op="q4_prompt", dtype="f16", batch=4, hk=8, n=4096, prefix=100),
        # one sequence, one token
        dict(name="q4_step_1", op="q4_attn", dtype="f16", batch=1, hq=32, hk=8, qlen=1, len=8192,
             window=0, sinks=0),
        # many long grouped-head sequences of ragged length: the size the format is for
        dict(name="q4_step_16", op="q4_attn", dtype="bf16", batch=16, hq=32, hk=8, qlen=1,
             len=32768, window=0, sinks=0),
        # a speculative block on plain multi-head rows with a window
        dict(name="q4_verify_window", op="q4_attn", dtype="f16", batch=4, hq=20, hk=20, qlen=5,
             len=16384, window=4000, sinks=4),
        # one row of a speech vocabulary
        dict(name="sample_1", op="sample", batch=1, vocab=51865, top_k=50, top_p=0.9, min_p=0.0,
             temperature=0.8, spread=3.0),
        # a serving batch over a large vocabulary, nucleus and min-p, every row its own values
        dict(name="sample_64", op="sample", batch=64, vocab=128000, top_k=0, top_p=0.95,
             min_p=0.02, temperature=1.0, spread=2.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "window", "window", "window_prefill", "q4_prompt", "q4_attn",
                     "q4_attn", "sample", "sample"])
    c = {"op": op}
    if op != "sample":
        c["dtype"] = rng.choice(["f16", "bf16"])
    hk = rng.choice([1, 2, 4, 5, 8, 20])
    hq = hk * rng.choice([1, 1, 3, 4, 5, 8])
    if op == "norm_rope":
        c.update(hq=hq, hk=hk, batch=_log(rng, 1, 64), n=_log(rng, 1, 8192),
                 far=_log(rng, 1, 131072))
        while work(c)["bytes"] > 1.6e8:
            c["n"] = max(1, c["n"] // 2)
            c["batch"] = max(1, c["batch"] - c["batch"] // 4)
            if c["n"] == 1 and c["batch"] == 1:
                break
    elif op in ("window", "q4_attn"):
        length = _log(rng, 1, 32768)
        c.update(hq=hq, hk=hk, batch=_log(rng, 1, 64), qlen=rng.choice([1, 1, 1, 2, 5, 8, 16]),
                 len=length, window=_log(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 17, 64, 130]))
        c["len"] = max(c["len"], c["qlen"])
        if op == "q4_attn" and rng.random() < 0.5:
            c.update(window=0, sinks=0)
        most = 2.5e8 if op == "q4_attn" else 1.2e9  # of the whole cache, as it is held
        row = 72 if op == "q4_attn" else 256
        while c["batch"] > 1 and (work(c)["bytes"] > 2.5e8 or
                                  c["batch"] * c["hk"] * c["len"] * row > most):
            c["batch"] = max(1, c["batch"] * 2 // 3)
    elif op == "window_prefill":
        c.update(hq=hq, hk=hk, batch=rng.choice([1, 1, 2, 3]), n=_log(rng, 1, 8192),
                 prefix=rng.choice([0, 0, 1, 77, 500]), window=_log(rng, 1, 8192),
                 sinks=rng.choice([0, 1, 4, 17, 64, 130]))
        # scores of the plain form: every pair of the prompt
        while c["batch"] * c["hq"] * c["n"] * (c["n"] + c["prefix"]) > 1.2e9 or \
                work(c)["flops"] > 4.0e10:
            c["n"] = c["n"] * 3 // 4
    elif op == "q4_prompt":
        c.update(hk=hk, batch=_log(rng, 1, 16), n=_log(rng, 1, 8192),
                 prefix=rng.choice([0, 1, 63, 100, 1000]))
        while c["n"] > 1 and work(c)["bytes"] > 1.0e8:
            c["n"] = c["n"] // 2
    else:
        c.update(batch=_log(rng, 1, 256), vocab=_log(rng, 1000, 262144),
                 top_k=rng.choice([0, 0, 1, 20, 50, 200, 1000]),
                 top_p=rng.choice([1.0, 1.0, 0.5, 0.9, 0.95, 0.99]),
                 min_p=rng.choice([0.0, 0.0, 0.02, 0.1]),
                 temperature=round(rng.uniform(0.3, 2.0), 3), spread=round(rng.uniform(1, 4), 2))
        while c["batch"] > 1 and c["batch"] * c["vocab"] > 64 * 128000:
            c["batch"] //= 2
    return c


def _visible(c):
    """(rows of K read, visible pairs) of one row's block of qlen queries at length len."""
    L, q, w, s = c["len"], c["qlen"], c["window"], c["sinks"]
    if w <= 0:
        return L, sum(L - q + i + 1 for i in range(q))
    pairs = 0
    for i in range(q):
        pos = L - q + i
        lo = max(0, pos - w + 1)
        pairs += pos + 1 - lo + min(lo, s)
    lo = max(0, L - q - w + 1)
    return L - lo + min(lo, s), pairs


def work(c):
    op = c["op"]
    if op == "norm_rope":
        rows = c["batch"] * c["n"] * (c["hq"] + c["hk"])
        return {"bytes": rows * D * 2 * 2, "flops": rows * D * 8}
    if op in ("window", "q4_attn"):
        B = c["batch"]
        row = (2 * D * 2) if op == "window" else (2 * (D // 2) + 8)
        # ragged rows are 3/4 of the longest on average
        share = 1.0 if B == 1 else 0.75 if c["window"] <= 0 else 1.0
        keys, pairs = _visible(c)
        byts = B * c["hk"] * keys * row * share + 2 * B * c["hq"] * c["qlen"] * D * 2
        return {"bytes": byts, "flops": 4.0 * D * B * c["hq"] * pairs * share}
    if op == "window_prefill":
        n, s0, w, s = c["n"], c["prefix"], c["window"], c["sinks"]
        pos = np.arange(s0, s0 + n, dtype=np.float64)
        lo = np.maximum(0, pos - w + 1)
        pairs = float((pos + 1 - lo + np.minimum(lo, s)).sum())
        byts = c["batch"] * (2 * c["hq"] * n + 2 * c["hk"] * (2 * n + min(s0, w + s))) * D * 2
        return {"bytes": byts, "flops": 4.0 * D * c["batch"] * c["hq"] * pairs}
    if op == "q4_prompt":
        rows = 2 * c["batch"] * c["hk"] * c["n"] * (1.0 if c["batch"] == 1 else 0.75)
        # 16-bit rows in, 4-bit rows out; 4-bit rows in, 16-bit rows out
        return {"bytes": rows * 2 * (D * 2 + D // 2 + 4), "flops": rows * D * 8}
    n = c["batch"] * c["vocab"]
    return {"bytes": n * 4, "flops": n * 8}


# ------------------------------------------------------------------ inputs -----------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _ragged(batch, longest, least, g):
    """int32 lengths: the first is the longest, the others between half of it and it."""
    lens = torch.randint(max(least, longest // 2), longest + 1, (batch,), generator=g,
                         device="cuda", dtype=torch.int32)
    lens[0] = longest
    return lens


def _quantise(x):
    """Rows of 64 values -> (n in 0..15, step bf16, zero point fp16), as fp32 values: the
    definition of the 4-bit format, every operation rounded to fp32 once."""
    x = x.float()
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    f15, f7h = (torch.tensor(v, dtype=torch.float32, device=x.device) for v in (15.0, 7.5))
    # (hi - lo) / 15, halved so that no finite range overflows
    step = ((0.5 * hi - 0.5 * lo) / f7h).to(torch.bfloat16).float()
    flat = step == 0  # equal values: 15 steps from 0 to the value
    one = (lo.abs() / f15).to(torch.bfloat16).float()
    one = torch.where(one == 0, 1.0, one)
    zp = torch.where(flat, torch.where(lo < 0, 15.0, 0.0),
                     (-lo / torch.where(flat, one, step)).to(torch.float16).float())
    step = torch.where(flat, one, step)
    n = torch.clamp(torch.round(x / step + zp), 0, 15)
    return n, step, zp


def _pack(n):
    n = n.to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4)


def _bits(step, zp):
    return torch.cat([step.to(torch.bfloat16).view(torch.int16),
                      zp.to(torch.float16).view(torch.int16)], dim=-1)


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    op = c["op"]
    if op == "sample":
        B, V = c["batch"], c["vocab"]
        st["logits"] = rnd(B, V) * c["spread"]
        st["u"] = torch.rand(B, generator=g, device="cuda")
        f = lambda v: torch.full((B,), v, dtype=torch.float32, device="cuda")  # noqa: E731
        # every request its own values around the case's
        vary = torch.rand(B, generator=g, device="cuda")
        st["temperature"] = f(c["temperature"]) * (0.75 + 0.5 * vary)
        st["top_k"] = (torch.full((B,), c["top_k"], dtype=torch.int32, device="cuda") +
                       (vary * 8 * (c["top_k"] > 1)).to(torch.int32))
        st["top_p"] = f(c["top_p"]) - 0.04 * vary * (c["top_p"] < 1)
        st["min_p"] = f(c["min_p"]) * (0.5 + vary)
        st["token"] = torch.empty(B, dtype=torch.int32, device="cuda")
        st["logprob"] = torch.empty(B, dtype=torch.float32, device="cuda")
        st["n_kept"] = torch.empty(B, dtype=torch.int32, device="cuda")
        return st
    dt = DT[c["dtype"]]
    B, hk = c["batch"], c["hk"]
    if op == "norm_rope":
        n, hq = c["n"], c["hq"]
        # the fused projection: [batch, tokens, q heads + k heads + v heads, 64]
        st["qkv"] = rnd(B, n, hq + 2 * hk, D).to(dt)
        st["wq"] = (1 + 0.2 * rnd(D)).to(dt)
        st["wk"] = (1 + 0.2 * rnd(D)).to(dt)
        st["pos0"] = _ragged(B, c["far"], 0, g)
        st["q_out"] = torch.empty(B, hq, n, D, dtype=dt, device="cuda")
        st["k_out"] = torch.empty(B, hk, n, D, dtype=dt, device="cuda")
        return st
    if op == "q4_prompt":
        n, s0 = c["n"], c["prefix"]
        st["k"] = (rnd(B, hk, n, D) + 0.5 * rnd(1, hk, 1, D)).to(dt)
        st["v"] = rnd(B, hk, n, D).to(dt)
        st["counts"] = _ragged(B, n, 1, g)
        st["pos0"] = torch.full((B,), s0, dtype=torch.int32, device="cuda")
        cap = s0 + n
        st["kq"] = torch.zeros(B, hk, cap, D // 2, dtype=torch.uint8, device="cuda")
        st["vq"] = torch.zeros_like(st["kq"])
        st["params"] = torch.zeros(B, hk, cap, 4, dtype=torch.int16, device="cuda")
        st["k_back"] = torch.empty(B, hk, n, D, dtype=dt, device="cuda")
        st["v_back"] = torch.empty_like(st["k_back"])
        return st
    hq = c["hq"]
    if op == "window_prefill":
        n, s0 = c["n"], c["prefix"]
        cap = s0 + n
        st["q"] = rnd(B, hq, n, D).to(dt)
        st["k_new"] = rnd(B, hk, n, D).to(dt)
        st["v_new"] = rnd(B, hk, n, D).to(dt)
        st["plens"] = _ragged(B, n, 1, g)
        st["lens_in"] = torch.full((B,), s0, dtype=torch.int32, device="cuda")
        st["k"] = rnd(B, hk, cap, D).to(dt)
        st["v"] = rnd(B, hk, cap, D).to(dt)
        st["out"] = torch.empty_like(st["q"])
        return st
    q, cap = c["qlen"], c["len"]
    st["q"] = rnd(B, hq, q, D).to(dt)
    st["lens"] = _ragged(B, cap, q, g)
    st["out"] = torch.empty_like(st["q"])
    st["workspace"] = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")
    if op == "window":
        st["k"] = rnd(B, hk, cap, D).to(dt)
        st["v"] = rnd(B, hk, cap, D).to(dt)
        return st
    st["kq"] = torch.empty(B, hk, cap, D // 2, dtype=torch.uint8, device="cuda")
    st["vq"] = torch.empty_like(st["kq"])
    st["params"] = torch.empty(B, hk, cap, 4, dtype=torch.int16, device="cuda")
    for b in range(B):  # a sequence at a time: the 32-bit values of all would not be small
        for name, at in (("kq", 0), ("vq", 2)):
            n, step, zp = _quantise(rnd(hk, cap, D) + 0.5 * rnd(hk, 1, D))
            st[name][b] = _pack(n)
            st["params"][b, :, :, at:at + 2] = _bits(step, zp)
    return st


# ------------------------------------------------------------------ plain forms ------
def _norm_rope(x, w, pos0, eps=1e-6, base=10000.0):
    """x [B, H, n, 64] of any strides -> normed, scaled, rotated."""
    n, dt = x.shape[2], x.dtype
    x = x.float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.float()
    i = torch.arange(D // 2, device=x.device, dtype=torch.float64)
    theta = base ** (-i / (D // 2))
    pos = (pos0[:, None].double() + torch.arange(n, device=x.device, dtype=torch.float64))
    a = pos[:, None, :, None] * theta  # angles of far positions: 64 bits
    cos, sin = torch.cos(a).float(), torch.sin(a).float()
    lo, hi = y[..., :D // 2], y[..., D // 2:]
    return torch.cat([lo * cos - hi * sin, hi * cos + lo * sin], dim=-1).to(dt)


def _softmax_pv(q, k, v, seen, scale):
    """q [B, Hk, G, n, 64], k and v [B, Hk, T, 64] in fp32, seen [B, n, T]."""
    B, Hk, G, n, _ = q.shape
    s = torch.matmul(q.reshape(B, Hk, G * n, D), k.transpose(-1, -2)).reshape(B, Hk, G, n, -1)
    s = torch.where(seen[:, None, None], s * scale, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = torch.matmul(p.reshape(B, Hk, G * n, -1), v)
    return o.reshape(B, Hk, G, n, D)


def _window_rows(lens, qlen, window, sinks, cap):
    """Positions a block of qlen queries can see, [B, J], and who sees which, [B, qlen, J]."""
    dev = lens.device
    lens = lens.long()
    pos = lens[:, None] - qlen + torch.arange(qlen, device=dev)
    if window <= 0:
        t = torch.arange(cap, device=dev)[None].expand(lens.shape[0], -1)
        return None, t[:, None, :] <= pos[:, :, None]
    first = torch.clamp(lens - qlen - window + 1, min=sinks)
    near = first[:, None] + torch.arange(min(cap, window + qlen - 1), device=dev)
    far = torch.arange(min(sinks, cap), device=dev)[None].expand(lens.shape[0], -1)
    t = torch.cat([far, near], dim=1)
    p = pos[:, :, None]
    seen = (t[:, None, :] <= p) & ((t[:, None, :] < sinks) | (t[:, None, :] > p - window))
    return t.clamp(0, cap - 1), seen


def _take(x, t):
    """x [B, H, cap, e] at positions t [B, J] -> [B, H, J, e]"""
    if t is None:
        return x
    b = torch.arange(x.shape[0], device=x.device)[:, None]
    return x[b, :, t].transpose(1, 2)


def _values(data, params):
    """4-bit rows -> fp32 values: step * (n - zero point)."""
    n = torch.stack([data & 15, data >> 4], dim=-1).reshape(*data.shape[:-1], D).float()
    params = params.contiguous()
    step = params[..., 0:1].contiguous().view(torch.bfloat16).float()
    zp = params[..., 1:2].contiguous().view(torch.float16).float()
    return step * (n - zp)


def _plain_attn(c, st):
    B, hq, hk, q = c["batch"], c["hq"], c["hk"], c["qlen"]
    t, seen = _window_rows(st["lens"], q, c["window"], c["sinks"], c["len"])
    if c["op"] == "window":
        k, v = _take(st["k"], t).float(), _take(st["v"], t).float()
    else:
        par = _take(st["params"], t)
        k = _values(_take(st["kq"], t), par[..., 0:2])
        v = _values(_take(st["vq"], t), par[..., 2:4])
    o = _softmax_pv(st["q"].float().reshape(B, hk, hq // hk, q, D), k, v, seen, 0.125)
    return {"out": o.reshape(B, hq, q, D).to(st["q"].dtype)}


def _plain_prefill(c, st):
    B, hq, hk, n = c["batch"], c["hq"], c["hk"], c["n"]
    cap = st["k"].shape[2]
    dev = st["q"].device
    t = torch.arange(cap, device=dev)
    j = t[None, :] - st["lens_in"][:, None]  # the prompt row written at position t
    new = ((j >= 0) & (j < st["plens"][:, None]))[:, None, :, None]
    jj = j.clamp(0, n - 1)
    for name in ("k", "v"):
        st[name].copy_(torch.where(new, _take(st[name + "_new"], jj), st[name]))
    pos = st["lens_in"][:, None] + torch.arange(n, device=dev)
    live = torch.arange(n, device=dev)[None] < st["plens"][:, None]
    p = pos[:, :, None]
    seen = (t <= p) & ((t < c["sinks"]) | (t > p - c["window"])) & live[:, :, None]
    o = _softmax_pv(st["q"].float().reshape(B, hk, hq // hk, n, D), st["k"].float(),
                    st["v"].float(), seen, 0.125)
    return {"out": o.reshape(B, hq, n, D).to(st["q"].dtype), "k": st["k"], "v": st["v"]}


def _plain_prompt(c, st):
    live = (torch.arange(c["n"], device="cuda")[None] < st["counts"][:, None])[:, None, :, None]
    out = {}
    for name in ("k", "v"):
        n, step, zp = _quantise(st[name])
        # rows past a prompt's end were never written: the cache holds zeros there
        out[name] = torch.where(live, step * (n - zp), 0.0).to(st[name].dtype)
    return out


def _plain_sample(c, st):
    V = c["vocab"]
    x = st["logits"].double()  # sums of a whole vocabulary, and draws next to a border
    T = st["temperature"].double()[:, None]
    y = (x - x.amax(-1, keepdim=True)) / T
    ys, ids = torch.sort(y, dim=-1, descending=True, stable=True)
    r = torch.arange(V, device=x.device)
    w = torch.exp(ys)
    k = torch.where(st["top_k"] > 0, st["top_k"], V)[:, None]
    w = w * (r < k)
    run = torch.cumsum(w, -1)
    p = st["top_p"].double()[:, None]
    kept = (r < k) & ((run - w < p * run[:, -1:]) | (p >= 1) | (r == 0))
    kept &= (w >= st["min_p"].double()[:, None]) | (r == 0)
    wi = torch.zeros_like(w).scatter_(-1, ids, w * kept)
    run = torch.cumsum(wi, -1)
    total = run[:, -1]
    token = (run <= (st["u"].double() * total)[:, None]).sum(-1).clamp_max(V - 1)
    lp = torch.log(torch.gather(wi, 1, token[:, None])[:, 0] / total)
    return {"token": token.to(torch.int32), "logprob": lp.float(),
            "n_kept": kept.sum(-1).to(torch.int32)}


# ------------------------------------------------------------------ the library ------
def _own(c, st):
    import kv_cached_decode_gb300 as kvd

    op = c["op"]
    if op == "norm_rope":
        hq, hk = c["hq"], c["hk"]
        heads = st["qkv"].transpose(1, 2)  # [batch, heads, tokens, 64], strided
        kvd.kvd_qk_norm_rope(heads[:, :hq], heads[:, hq:hq + hk], st["q_out"], st["k_out"],
                             q_weight=st["wq"], k_weight=st["wk"], pos0=st["pos0"], eps=1e-6,
                             base=10000.0)
        return {"q": st["q_out"], "k": st["k_out"]}
    if op == "sample":
        kvd.kvd_sample_filtered(st["logits"], st["u"], st["token"],
                                temperature=st["temperature"], top_k=st["top_k"],
                                top_p=st["top_p"], min_p=st["min_p"], logprob=st["logprob"],
                                n_kept=st["n_kept"])
        return {"token": st["token"], "logprob": st["logprob"], "n_kept": st["n_kept"]}
    if op == "q4_prompt":
        cache = kvd.make_q4_cache(st["kq"], st["vq"], st["params"])
        kvd.kvd_q4_append(cache, st["k"], st["v"], st["pos0"], counts=st["counts"])
        kvd.kvd_q4_dequant(cache, st["k_back"], st["v_back"], pos0=st["pos0"])
        return {"k": st["k_back"], "v": st["v_back"]}
    if op == "window":
        kvd.kvd_window_attn(st["q"], kvd.make_cache(st["k"], st["v"]), st["out"],
                            st["workspace"], c["window"], c["sinks"], lens=st["lens"])
        return {"out": st["out"]}
    if op == "window_prefill":
        kvd.kvd_prefill_window_attn(st["q"], kvd.make_cache(st["k"], st["v"]), st["k_new"],
                                    st["v_new"], st["plens"], st["out"], c["window"], c["sinks"],
                                    lens_in=st["lens_in"])
        return {"out": st["out"], "k": st["k"], "v": st["v"]}
    cache = kvd.make_q4_cache(st["kq"], st["vq"], st["params"])
    kvd.kvd_q4_attn(st["q"], cache, st["out"], st["workspace"], lens=st["lens"],
                    window=c["window"], n_sinks=c["sinks"])
    return {"out": st["out"]}


def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    if c["op"] == "norm_rope":
        heads = state["qkv"].transpose(1, 2)
        hq, hk = c["hq"], c["hk"]
        return {"q": _norm_rope(heads[:, :hq], state["wq"], state["pos0"]),
                "k": _norm_rope(heads[:, hq:hq + hk], state["wk"], state["pos0"])}
    if c["op"] == "sample":
        return _plain_sample(c, state)
    if c["op"] == "q4_prompt":
        return _plain_prompt(c, state)
    if c["op"] == "window_prefill":
        return _plain_prefill(c, state)
    return _plain_attn(c, state)


# ------------------------------------------------------------------ in 64 bits -------
def _exact_attention(q, k, v, first, live, window, sinks):
    """One sequence: q [hq, n, 64] whose first query stands at position `first` and whose
    rows from `live` on are padding; k and v [hk, T, 64]; 64 bits, a key-value head at a
    time, from the definition."""
    hq, n, _ = q.shape
    hk, T, _ = k.shape
    g = hq // hk
    where = torch.arange(first, first + n, device=q.device).view(1, n, 1)
    key = torch.arange(T, device=q.device).view(1, 1, T)
    hide = key > where
    if window > 0:
        hide = hide | ((key <= where - window) & (key >= sinks))
    out = torch.zeros(hq, n, D, dtype=torch.float64, device=q.device)
    for h in range(hk):
        a = torch.einsum("gnd,td->gnt", q[h * g:(h + 1) * g].double(), k[h].double()) / 8.0
        a = a.masked_fill(hide, -math.inf)
        top = a.max(dim=-1, keepdim=True).values
        e = torch.exp(a - top)
        e = torch.nan_to_num(e, nan=0.0)
        z = e.sum(dim=-1, keepdim=True)
        o = torch.einsum("gnt,td->gnd", e, v[h].double()) / torch.where(z > 0, z, 1.0)
        out[h * g:(h + 1) * g] = o
    if live < n:
        out[:, live:] = 0
    return out


def _exact_rows(x):
    """The 4-bit format's rows, from its definition, in 64 bits (the step and the zero point
    are numbers of 16 bits by definition)."""
    x = x.double()
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    step = ((hi - lo) / 15).float().to(torch.bfloat16).double()
    zp = (-lo / step).float().to(torch.float16).double()
    return (torch.round(x / step + zp).clamp(0, 15) - zp) * step


def _exact_stored(data, params, at):
    n = torch.empty(*data.shape[:-1], D, dtype=torch.float64, device=data.device)
    n[..., 0::2] = (data % 16).double()
    n[..., 1::2] = torch.div(data, 16, rounding_mode="floor").double()
    step = params[..., at].clone().view(torch.bfloat16).double()
    zp = params[..., at + 1].clone().view(torch.float16).double()
    return (n - zp[..., None]) * step[..., None]


def _exact_sample(c, st):
    x = st["logits"].cpu().numpy().astype(np.float64)
    par = {k: st[k].cpu().numpy() for k in ("u", "temperature", "top_k", "top_p", "min_p")}
    token, lp, kept = [], [], []
    for b in range(c["batch"]):
        order = np.lexsort((np.arange(c["vocab"]), -x[b]))
        k = int(par["top_k"][b])
        order = order[:k] if k > 0 else order
        e = np.exp((x[b][order] - x[b].max()) / np.float64(par["temperature"][b]))
        keep = len(order)
        p = float(par["top_p"][b])
        if p < 1:
            c0 = np.cumsum(e)
            keep = min(keep, int(np.searchsorted(c0, p * c0[-1], side="left")) + 1)
        keep = min(keep, max(1, int((e >= float(par["min_p"][b])).sum())))
        at = np.argsort(order[:keep])
        ids, e = order[:keep][at], e[:keep][at]
        c1 = np.cumsum(e)
        i = min(int(np.searchsorted(c1, float(par["u"][b]) * c1[-1], side="right")), keep - 1)
        token.append(ids[i])
        lp.append(math.log(e[i] / c1[-1]))
        kept.append(keep)
    return {"token": np.array(token, np.int32), "logprob": np.array(lp),
            "n_kept": np.array(kept, np.int32)}


def exact(case, seed):
    c, st = case, prepare(case, seed)
    op = c["op"]
    if op == "sample":
        return _exact_sample(c, st)
    if op == "norm_rope":
        out = {}
        for name, w, h0, h1 in (("q", "wq", 0, c["hq"]), ("k", "wk", c["hq"], c["hq"] + c["hk"])):
            x = st["qkv"][:, :, h0:h1].double()
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / D + 1e-6) * st[w].double()
            z = torch.complex(x[..., :D // 2], x[..., D // 2:])
            pos = st["pos0"].double()[:, None] + torch.arange(c["n"], device="cuda").double()
            turn = pos[..., None] * torch.tensor([10000.0 ** (-i / 32) for i in range(32)],
                                                 dtype=torch.float64, device="cuda")
            z = z * torch.polar(torch.ones_like(turn), turn)[:, :, None]
            out[name] = torch.cat([z.real, z.imag], -1).transpose(1, 2)
        return out
    if op == "q4_prompt":
        out = {}
        for name in ("k", "v"):
            x = _exact_rows(st[name])
            for b in range(c["batch"]):
                x[b, :, int(st["counts"][b]):] = 0
            out[name] = x
        return out
    if op == "window_prefill":
        s0, out = c["prefix"], []
        k, v = st["k"].clone(), st["v"].clone()
        for b in range(c["batch"]):
            m = int(st["plens"][b])
            k[b, :, s0:s0 + m] = st["k_new"][b, :, :m]
            v[b, :, s0:s0 + m] = st["v_new"][b, :, :m]
            out.append(_exact_attention(st["q"][b], k[b], v[b], s0, m, c["window"], c["sinks"]))
        return {"out": torch.stack(out), "k": None, "v": None}
    out = []
    for b in range(c["batch"]):
        m = int(st["lens"][b])
        if op == "window":
            k, v = st["k"][b, :, :m], st["v"][b, :, :m]
        else:
            k = _exact_stored(st["kq"][b, :, :m], st["params"][b, :, :m], 0)
            v = _exact_stored(st["vq"][b, :, :m], st["params"][b, :, :m], 2)
        out.append(_exact_attention(st["q"][b], k, v, m - c["qlen"], c["qlen"], c["window"],
                                    c["sinks"]))
    return {"out": torch.stack(out)}
