"""Cases of the operators of a served batch: each as its plain form in elementary torch
operations and as the calls a user of the library makes.

Four groups: rotary positions in other layouts and scalings (``rope``), new tokens written to
a paged cache with their rotation (``append``), attention of a chunk of new tokens over a
paged cache (``attn``), and log probabilities of given tokens with entropy and top
alternatives (``logprob``).
"""

import math
import random

import numpy as np
import torch

own = False  # True: the library's calls; False: the plain forms

D = 64  # head size of the library
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}

PLAIN = dict(base=10000.0, rot=64, inter=False, scaling="none", factor=1.0, trained=0, low=1.0,
             high=1.0, mag=1.0)
# contexts eight times the trained length: frequencies scaled by wavelength bands
BANDS = dict(base=500000.0, rot=64, inter=False, scaling="bands", factor=8.0, trained=8192,
             low=1.0, high=4.0, mag=1.0)
# a ramp over the pairs, with the magnitude that goes with it
RAMP = dict(base=10000.0, rot=64, inter=False, scaling="ramp", factor=16.0, trained=4096,
            low=1.0, high=32.0, mag=1.2772588)
# interleaved pairs in the first half of the head
PART = dict(base=10000.0, rot=32, inter=True, scaling="linear", factor=4.0, trained=0, low=1.0,
            high=1.0, mag=1.0)


# ------------------------------------------------------------------ cases ------------
def listed():
    return [
        # one decode step of 16 sequences far in their context: q and k heads of a fused
        # projection
        dict(name="rope_step", op="rope", dtype="bf16", batch=16, n=1, hq=20, hk=4, far=60000,
             rope="bands"),
        # a prompt chunk of 4 sequences, half of each head, interleaved
        dict(name="rope_prompt", op="rope", dtype="f16", batch=4, n=4096, hq=20, hk=4, far=8192,
             rope="part"),
        # one token each of 64 sequences into pages of 16, queries rotated along
        dict(name="append_step", op="append", dtype="bf16", batch=64, hq=32, hk=4, page=16,
             order="head", chunk_rows=0, chunk=0, block=1, len=1024, rope="bands"),
        # ragged prompts of 6 sequences into pages of 64 tokens of all heads
        dict(name="append_prompt", op="append", dtype="f16", batch=6, hq=20, hk=4, page=64,
             order="token", chunk_rows=6, chunk=2000, block=1, len=2500, rope="ramp"),
        # one sequence, one token
        dict(name="attn_step_1", op="attn", dtype="f16", batch=1, hq=32, hk=8, page=16,
             order="head", chunk_rows=0, chunk=0, block=1, len=8192),
        # a serving batch of ragged long sequences, one token each
        dict(name="attn_step_32", op="attn", dtype="bf16", batch=32, hq=32, hk=8, page=16,
             order="head", chunk_rows=0, chunk=0, block=1, len=16384),
        # a speculative block on plain multi-head rows, odd lengths
        dict(name="attn_verify_8", op="attn", dtype="f16", batch=8, hq=20, hk=20, page=32,
             order="token", chunk_rows=0, chunk=0, block=5, len=4095),
        # the last chunk of a long prompt
        dict(name="attn_chunk_1", op="attn", dtype="bf16", batch=1, hq=32, hk=8, page=64,
             order="head", chunk_rows=1, chunk=512, block=1, len=16384),
        # decoding sequences and two prompt chunks in one batch
        dict(name="attn_mixed_30", op="attn", dtype="bf16", batch=30, hq=20, hk=4, page=16,
             order="head", chunk_rows=2, chunk=1000, block=1, len=8000),
        # the sampled token of one row of a speech vocabulary, five alternatives
        dict(name="logprob_1", op="logprob", dtype="f32", rows=1, vocab=51865, pad=0, given=1,
             top=5, spread=3.0, temper=False),
        # the sampled tokens of a serving batch over a large vocabulary
        dict(name="logprob_64", op="logprob", dtype="bf16", rows=64, vocab=128000, pad=256,
             given=1, top=20, spread=2.5, temper=True),
        # a prompt scored: 2000 positions, some of them padding
        dict(name="logprob_prompt", op="logprob", dtype="f32", rows=2000, vocab=51865, pad=0,
             given=1, top=1, spread=3.0, temper=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "append", "attn", "attn", "attn", "attn", "logprob",
                     "logprob"])
    c = {"op": op}
    if op == "logprob":
        c.update(dtype=rng.choice(["f32", "f32", "f16", "bf16"]), rows=_log(rng, 1, 3000),
                 vocab=_log(rng, 1000, 262144), pad=rng.choice([0, 0, 1, 64, 247]),
                 given=rng.choice([0, 1, 1, 1, 4]), top=rng.choice([0, 1, 5, 20, 32]),
                 spread=round(rng.uniform(1, 4), 2), temper=rng.random() < 0.5)
        while work(c)["bytes"] > 4.0e8:
            c["rows"] = max(1, c["rows"] * 2 // 3)
        return c
    c["dtype"] = rng.choice(["f16", "bf16"])
    hk = rng.choice([1, 2, 4, 5, 8, 20])
    hq = hk * rng.choice([1, 1, 3, 4, 5, 8])
    c.update(hq=hq, hk=hk)
    if op != "attn":
        c["rope"] = rng.choice(sorted(ROPES))
    if op == "rope":
        c.update(batch=_log(rng, 1, 64), n=_log(rng, 1, 8192), far=_log(rng, 1, 131072))
        while work(c)["bytes"] > 1.0e8 and (c["n"] > 1 or c["batch"] > 1):
            c["n"] = max(1, c["n"] // 2)
            c["batch"] = max(1, c["batch"] - c["batch"] // 4)
        return c
    c.update(batch=_log(rng, 1, 128), page=rng.choice([8, 16, 16, 32, 64, 128, 256]),
             order=rng.choice(["head", "head", "token"]), block=rng.choice([1, 1, 1, 2, 5, 16]),
             len=_log(rng, 16, 2048 if op == "append" else 32768))
    c["chunk_rows"] = rng.choice([0, 0, 1, 1, 2, c["batch"]])
    c["chunk_rows"] = min(c["chunk_rows"], c["batch"])
    c["chunk"] = min(_log(rng, 16, 8192), c["len"]) if c["chunk_rows"] else 0
    if op == "append":
        # the pools are outputs: 200 MB of them at most
        while c["batch"] > 1 and (2 * c["batch"] * c["len"] * hk * 128 > 2.0e8 or
                                  work(c)["bytes"] > 1.0e8):
            c["batch"] = c["batch"] * 2 // 3
            c["chunk_rows"] = min(c["chunk_rows"], c["batch"])
        return c
    while c["batch"] > 1 and work(c)["bytes"] > 4.0e8:
        c["batch"] = c["batch"] * 2 // 3
        c["chunk_rows"] = min(c["chunk_rows"], c["batch"])
    # scores of the plain form: every pair of the padded chunk rows
    while c["chunk_rows"] * c["hq"] * c["chunk"] * c["len"] > 6.0e8 or work(c)["flops"] > 6.0e10:
        if c["chunk_rows"] > 2:
            c["chunk_rows"] = c["chunk_rows"] * 2 // 3
        else:
            c["chunk"] = max(16, c["chunk"] * 3 // 4)
            c["len"] = max(c["chunk"], c["len"] * 3 // 4)
    return c


def _new_tokens(c):
    """New tokens of the batch, chunks ragged between half of the longest and it."""
    R = c["chunk_rows"]
    share = 1.0 if R == 1 else 0.75
    return (c["batch"] - R) * c["block"], R * c["chunk"] * share


def work(c):
    op = c["op"]
    if op == "rope":
        rows = c["batch"] * c["n"] * (c["hq"] + c["hk"])
        return {"bytes": rows * D * 2 * 2, "flops": rows * D * 3}
    if op == "logprob":
        n = c["rows"] * c["vocab"]
        per = 8 + c["given"] * 12 + c["top"] * 8
        return {"bytes": n * (4 if c["dtype"] == "f32" else 2) + c["rows"] * per, "flops": n * 6}
    few, many = _new_tokens(c)
    if op == "append":
        rows = (few + many) * (c["hq"] + 2 * c["hk"])
        return {"bytes": rows * D * 2 * 2, "flops": rows * D * 3}
    B, R = c["batch"], c["chunk_rows"]
    mean = c["len"] * (1.0 if B == 1 else 0.75)  # ragged rows: 3/4 of the longest on average
    byts = 2 * B * c["hk"] * mean * D * 2 + 2 * (few + many) * c["hq"] * D * 2
    pairs = few * mean + (many * (mean - 0.5 * many / R) if R else 0)
    return {"bytes": byts, "flops": 4.0 * D * c["hq"] * pairs}


# ------------------------------------------------------------------ inputs -----------
ROPES = {"plain": PLAIN, "bands": BANDS, "ramp": RAMP, "part": PART}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _batch(c, seed):
    """New tokens and lengths (new tokens included) of every row, the chunk rows first. The
    seed changes which row has which; their sums are the case's."""
    rng, order = random.Random(c["len"] + c["chunk"]), random.Random(seed)
    R = c["chunk_rows"]
    half = lambda most: rng.randint((most + 1) // 2, most)  # noqa: E731
    n = [c["chunk"] if b == 0 else half(c["chunk"]) for b in range(R)]
    n += [c["block"]] * (c["batch"] - R)
    rows = [(x, max(x, c["len"] if b == 0 else half(c["len"]))) for b, x in enumerate(n)]
    chunks, rest = rows[:R], rows[R:]
    order.shuffle(chunks)
    order.shuffle(rest)
    return tuple(list(x) for x in zip(*(chunks + rest)))


def _pages(c, st, lens, g):
    """A pool with some free pages, and a table that gives every row its pages in any order;
    entries past a row's pages hold -1."""
    ps, hk, dt = c["page"], c["hk"], DT[c["dtype"]]
    need = [-(-x // ps) for x in lens]
    n_pages = sum(need) + 8
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((c["batch"], max(need) + 2), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = order[at:at + k]
        at += k
    st["table"] = table
    shape = (n_pages, hk, ps, D) if c["order"] == "head" else (n_pages, ps, hk, D)
    for name in ("k", "v"):
        pool = torch.empty(shape, dtype=dt, device="cuda")
        for p0 in range(0, n_pages, 4096):  # the 32-bit values of all would not be small
            part = pool[p0:p0 + 4096]
            part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
        st[name + "_pool"] = pool
        st[name] = pool if c["order"] == "head" else pool.transpose(1, 2)


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    dt = DT[c["dtype"]]
    if c["op"] == "logprob":
        R, V, m = c["rows"], c["vocab"], c["given"]
        buf = torch.empty(R, V + c["pad"], dtype=dt, device="cuda")
        for r0 in range(0, R, 256):
            part = buf[r0:r0 + 256]
            part.copy_(rnd(*part.shape) * c["spread"])
        st["logits"] = buf[:, :V]
        # half of the given tokens are likely ones, as sampled tokens are
        t = torch.randint(0, V, (R, max(m, 1)), generator=g, device="cuda")
        best = buf[:, :V].float().argmax(-1, keepdim=True).expand_as(t)
        t = torch.where(torch.rand(t.shape, generator=g, device="cuda") < 0.5, t, best)
        if R > 8:  # padding: rows that score nothing
            t[R - R // 8:] = -1
        st["tokens"] = t[:, :m].to(torch.int32).contiguous()
        st["temperature"] = (0.5 + torch.rand(R, generator=g, device="cuda")) if c["temper"] \
            else None
        f, i = (dict(dtype=x, device="cuda") for x in (torch.float32, torch.int32))
        st["out"] = {"entropy": torch.empty(R, **f), "lse": torch.empty(R, **f)}
        if m:
            st["out"].update(logprob=torch.empty(R, m, **f), rank=torch.empty(R, m, **i))
        if c["top"]:
            st["out"].update(top_id=torch.empty(R, c["top"], **i),
                             top_logprob=torch.empty(R, c["top"], **f))
        return st
    hq, hk = c["hq"], c["hk"]
    if c["op"] == "rope":
        B, n = c["batch"], c["n"]
        # the fused projection: [batch, tokens, q heads + k heads + v heads, 64]
        st["qkv"] = rnd(B, n, hq + 2 * hk, D).to(dt)
        pos0 = torch.randint(0, c["far"] + 1, (B,), generator=g, device="cuda")
        pos0[0] = c["far"]
        st["pos0"] = pos0.to(torch.int32)
        st["q_out"] = torch.empty(B, hq, n, D, dtype=dt, device="cuda")
        st["k_out"] = torch.empty(B, hk, n, D, dtype=dt, device="cuda")
        return st
    n, lens = _batch(c, seed)
    T = sum(n)
    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    st["starts"], st["lens"], st["max_new"] = _i32(starts), _i32(lens), max(n)
    _pages(c, st, lens, g)
    if c["op"] == "append":
        st["lens_in"] = _i32([y - x for x, y in zip(n, lens)])
        st["lens_out"] = torch.empty_like(st["lens_in"])
        st["qkv"] = rnd(T, hq + 2 * hk, D).to(dt)
        st["q_out"] = torch.empty(T, hq, D, dtype=dt, device="cuda")
        return st
    st["q"] = rnd(T, hq, D).to(dt)
    st["out"] = torch.empty_like(st["q"])
    st["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms ------
def _theta(r, device):
    """Scaled frequencies of the pairs, in radians per position, 64 bits."""
    rot = r["rot"]
    i = torch.arange(rot // 2, device=device, dtype=torch.float64)
    theta = r["base"] ** (-2.0 * i / rot)
    if r["scaling"] == "linear":
        return theta / r["factor"]
    if r["scaling"] == "bands":
        turns = r["trained"] * theta / (2 * math.pi)
        keep = ((turns - r["low"]) / (r["high"] - r["low"])).clamp(0, 1)
        return theta * (keep + (1 - keep) / r["factor"])
    if r["scaling"] == "ramp":
        at = lambda t: rot * math.log(r["trained"] / (2 * math.pi * t)) / (  # noqa: E731
            2 * math.log(r["base"]))
        lo = max(math.floor(at(r["high"])), 0)
        hi = min(math.ceil(at(r["low"])), rot - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return theta * (keep + (1 - keep) / r["factor"])
    return theta


def _rotate(x, pos, r):
    """x [..., 64] at positions pos [...] (broadcast), in 32 bits, rounded once."""
    a = pos.double()[..., None] * _theta(r, x.device)  # angles of far positions: 64 bits
    cos, sin = (torch.cos(a) * r["mag"]).float(), (torch.sin(a) * r["mag"]).float()
    y, h = x.float().clone(), r["rot"] // 2
    if r["inter"]:
        lo, hi = y[..., 0:2 * h:2].clone(), y[..., 1:2 * h:2].clone()
        y[..., 0:2 * h:2], y[..., 1:2 * h:2] = lo * cos - hi * sin, hi * cos + lo * sin
    else:
        lo, hi = y[..., :h].clone(), y[..., h:2 * h].clone()
        y[..., :h], y[..., h:2 * h] = lo * cos - hi * sin, hi * cos + lo * sin
    return y.to(x.dtype)


def _rows(starts, T):
    """The row of every packed token, and its place in the row."""
    t = torch.arange(T, device=starts.device)
    row = torch.searchsorted(starts.long(), t, right=True) - 1
    return row, t - starts.long()[row]


def _plain_append(c, st):
    r, hq, hk, qkv = ROPES[c["rope"]], c["hq"], c["hk"], st["qkv"]
    row, j = _rows(st["starts"], qkv.shape[0])
    pos = st["lens_in"].long()[row] + j
    page = st["table"].long()[row, pos // c["page"]]
    slot = pos % c["page"]
    q = _rotate(qkv[:, :hq], pos[:, None], r)
    st["k"][page, :, slot] = _rotate(qkv[:, hq:hq + hk], pos[:, None], r)
    st["v"][page, :, slot] = qkv[:, hq + hk:]
    return {"q": q, "k": st["k_pool"], "v": st["v_pool"],
            "lens": st["lens_in"] + (st["starts"][1:] - st["starts"][:-1])}


def _attend(c, st, b0, b1, n, out):
    """Rows b0 .. b1-1, n new tokens each at most, padded to one shape."""
    if b1 <= b0:
        return
    hq, hk, ps, R = c["hq"], c["hk"], c["page"], b1 - b0
    starts, lens = st["starts"][b0:b1 + 1].long(), st["lens"][b0:b1].long()
    dev = starts.device
    width = -(-c["len"] // ps)
    table = st["table"][b0:b1, :width].long().clamp(min=0)
    L = table.shape[1] * ps
    # [R, pages, heads, page, 64] -> [R, heads, L, 64]
    k, v = (st[x][table].transpose(1, 2).reshape(R, hk, L, D).float() for x in ("k", "v"))
    j = torch.arange(n, device=dev)
    live = j < (starts[1:] - starts[:-1])[:, None]
    at = (starts[:-1, None] + j).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][at].float().permute(0, 2, 1, 3).reshape(R, hk, (hq // hk) * n, D)
    pos = (lens - (starts[1:] - starts[:-1]))[:, None] + j
    seen = (torch.arange(L, device=dev) <= pos[:, :, None]) & live[:, :, None]
    s = (torch.matmul(q, k.transpose(-1, -2)) * 0.125).reshape(R, hk, hq // hk, n, L)
    s = torch.where(seen[:, None, None], s, float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == float("-inf"), 0.0, m))
    p = p / p.sum(-1, keepdim=True).clamp_min(1e-30)
    o = torch.matmul(p.reshape(R, hk, (hq // hk) * n, L), v)
    o = o.reshape(R, hq, n, D).transpose(1, 2).to(out.dtype)
    t0 = 0 if b0 == 0 else out.shape[0] - R * n  # the rows behind the chunks are equally long
    t1 = out.shape[0] - (c["batch"] - c["chunk_rows"]) * c["block"] if b0 == 0 and \
        c["chunk_rows"] else out.shape[0]
    row, i = _rows(starts - starts[0], t1 - t0)
    out[t0:t1] = o[row, i]


def _plain_attn(c, st):
    out, R = st["out"], c["chunk_rows"]
    _attend(c, st, 0, R, c["chunk"], out)
    _attend(c, st, R, c["batch"], c["block"], out)
    return {"out": out}


def _plain_logprob(c, st):
    x = st["logits"].float()
    V, m = c["vocab"], c["given"]
    y = x if st["temperature"] is None else x / st["temperature"][:, None]
    z = y - y.amax(-1, keepdim=True)
    e = torch.exp(z)
    s = e.sum(-1, keepdim=True)
    log_s = torch.log(s)
    out = {"entropy": (log_s - (e * z).sum(-1, keepdim=True) / s)[:, 0],
           "lse": (log_s + y.amax(-1, keepdim=True))[:, 0]}
    if m:
        t = st["tokens"].long()
        some = t >= 0
        at = t.clamp(min=0)
        out["logprob"] = torch.where(some, torch.gather(z, 1, at) - log_s, 0.0)
        mine = torch.gather(x, 1, at)
        ids = torch.arange(V, device=x.device)
        before = (x[:, None] > mine[..., None]) | \
                 ((x[:, None] == mine[..., None]) & (ids < at[..., None]))
        out["rank"] = torch.where(some, before.sum(-1), -1).to(torch.int32)
    if c["top"]:
        # one whole number per id, ordered by logit, then lower id first
        b = (x + 0.0).contiguous().view(torch.int32)
        key = torch.where(b < 0, b ^ 0x7fffffff, b).long() * 2 ** 20
        key += V - 1 - torch.arange(V, device=x.device)
        top = V - 1 - torch.topk(key, c["top"], dim=-1).values % 2 ** 20
        out["top_id"] = top.to(torch.int32)
        out["top_logprob"] = torch.gather(z, 1, top) - log_s
    return out


# ------------------------------------------------------------------ the library ------
def _spec(kvd, st):
    """The rotation of the model, made once by its program."""
    if "spec" not in st:
        r = ROPES[st["case"]["rope"]]
        st["spec"] = kvd.make_rope(base=r["base"], rot_dim=r["rot"], interleaved=r["inter"],
                                   scaling=r["scaling"], factor=r["factor"],
                                   original_len=r["trained"], low=r["low"], high=r["high"],
                                   magnitude=r["mag"])
    return st["spec"]


def _own(c, st):
    import kv_cached_decode_gb300 as kvd

    op = c["op"]
    if op == "logprob":
        kvd.kvd_token_logprobs(st["logits"], st["tokens"] if c["given"] else None,
                               temperature=st["temperature"], **st["out"])
        return st["out"]
    hq, hk = c["hq"], c["hk"]
    if op == "rope":
        heads = st["qkv"].transpose(1, 2)  # [batch, heads, tokens, 64], strided
        kvd.kvd_rope_scaled(heads[:, :hq], heads[:, hq:hq + hk], st["q_out"], st["k_out"],
                            rope=_spec(kvd, st), pos0=st["pos0"])
        return {"q": st["q_out"], "k": st["k_out"]}
    if "cache" not in st:  # a layer's cache, described once
        st["cache"] = kvd.make_paged_cache(st["k"], st["v"], st["table"])
    if op == "append":
        qkv = st["qkv"]
        kvd.kvd_paged_append(st["cache"], qkv[:, hq:hq + hk], qkv[:, hq + hk:], st["starts"],
                             st["lens_in"], lens_out=st["lens_out"], q=qkv[:, :hq],
                             q_out=st["q_out"], rope=_spec(kvd, st))
        return {"q": st["q_out"], "k": st["k_pool"], "v": st["v_pool"], "lens": st["lens_out"]}
    kvd.kvd_paged_attn(st["q"], st["cache"], st["out"], st["workspace"], st["starts"],
                       st["lens"], max_new=st["max_new"])
    return {"out": st["out"]}


def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    if c["op"] == "rope":
        heads = state["qkv"].transpose(1, 2)
        hq, hk, r = c["hq"], c["hk"], ROPES[c["rope"]]
        pos = (state["pos0"].long()[:, None] +
               torch.arange(c["n"], device=heads.device))[:, None]
        return {"q": _rotate(heads[:, :hq], pos, r), "k": _rotate(heads[:, hq:hq + hk], pos, r)}
    if c["op"] == "append":
        return _plain_append(c, state)
    if c["op"] == "attn":
        return _plain_attn(c, state)
    return _plain_logprob(c, state)


# ------------------------------------------------------------------ in 64 bits -------
def _exact_turn(r):
    """Radians per position of every pair, from the definitions, as Python numbers."""
    out = []
    for i in range(r["rot"] // 2):
        t = r["base"] ** (-(2 * i) / r["rot"])
        if r["scaling"] == "linear":
            w = 0.0
        elif r["scaling"] == "bands":
            length = 2 * math.pi / t
            w = min(1.0, max(0.0, (r["trained"] / length - r["low"]) / (r["high"] - r["low"])))
        elif r["scaling"] == "ramp":
            ln = 2 * math.log(r["base"]) / r["rot"]
            a = math.floor(math.log(r["trained"] / (2 * math.pi * r["high"])) / ln)
            b = math.ceil(math.log(r["trained"] / (2 * math.pi * r["low"])) / ln)
            a, b = max(a, 0), min(b, r["rot"] - 1)
            w = 1.0 - min(1.0, max(0.0, (i - a) / (b - a if b > a else 0.001)))
        else:
            w = 1.0
        out.append(w * t + (1.0 - w) * t / r["factor"])
    return out


def _exact_rotate(x, pos, r):
    x, h = x.double(), r["rot"] // 2
    turn = pos.double()[..., None] * torch.tensor(_exact_turn(r), dtype=torch.float64,
                                                  device=x.device)
    w = torch.polar(torch.full_like(turn, r["mag"]), turn)
    if r["inter"]:
        z = torch.view_as_complex(x[..., :2 * h].reshape(*x.shape[:-1], h, 2).contiguous()) * w
        y = torch.view_as_real(z).reshape(*x.shape[:-1], 2 * h)
    else:
        z = torch.complex(x[..., :h], x[..., h:2 * h]) * w
        y = torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., 2 * h:]], -1)


def _exact_logprob(c, st):
    R, V = c["rows"], c["vocab"]
    keep = {k: [] for k in st["out"]}
    for r0 in range(0, R, 128):
        x = st["logits"][r0:r0 + 128].double()
        y = x
        if st["temperature"] is not None:
            y = x / st["temperature"][r0:r0 + 128].double()[:, None]
        lse = torch.logsumexp(y, -1, keepdim=True)
        lp = y - lse
        keep["lse"].append(lse[:, 0])
        keep["entropy"].append(-(torch.exp(lp) * lp).sum(-1))
        order = None
        if c["top"] or c["given"]:
            order = torch.sort(x, dim=-1, descending=True, stable=True).indices
        if c["top"]:
            keep["top_id"].append(order[:, :c["top"]].to(torch.int32))
            keep["top_logprob"].append(torch.gather(lp, 1, order[:, :c["top"]]))
        if c["given"]:
            t = st["tokens"][r0:r0 + 128].long()
            place = torch.empty_like(order).scatter_(
                1, order, torch.arange(V, device=x.device).expand_as(order))
            pad = t < 0
            t = t.masked_fill(pad, 0)
            keep["logprob"].append(torch.gather(lp, 1, t).masked_fill(pad, 0.0))
            keep["rank"].append(torch.gather(place, 1, t).masked_fill(pad, -1).to(torch.int32))
    return {k: torch.cat(v) for k, v in keep.items()}


def exact(case, seed):
    c, st = case, prepare(case, seed)
    op = c["op"]
    if op == "logprob":
        return _exact_logprob(c, st)
    hq, hk = c["hq"], c["hk"]
    if op == "rope":
        r, out = ROPES[c["rope"]], {}
        pos = st["pos0"].double()[:, None] + torch.arange(c["n"], device="cuda").double()
        for name, h0, h1 in (("q", 0, hq), ("k", hq, hq + hk)):
            x = st["qkv"][:, :, h0:h1]
            out[name] = _exact_rotate(x, pos[:, :, None], r).transpose(1, 2)
        return out
    n, lens = _batch(c, seed)
    table, ps = st["table"].cpu().numpy(), c["page"]
    if op == "append":
        r, t, q = ROPES[c["rope"]], 0, []
        k, v = st["k"].double(), st["v"].double()
        for b in range(c["batch"]):
            rows = st["qkv"][t:t + n[b]]
            pos = np.arange(lens[b] - n[b], lens[b])
            page = torch.from_numpy(table[b, pos // ps].astype(np.int64)).cuda()
            slot = torch.from_numpy(pos % ps).cuda()
            turned = _exact_rotate(rows[:, :hq + hk], torch.from_numpy(pos).cuda()[:, None], r)
            q.append(turned[:, :hq])
            k[page, :, slot] = turned[:, hq:]
            v[page, :, slot] = rows[:, hq + hk:].double()
            t += n[b]
        if c["order"] == "token":
            k, v = k.transpose(1, 2), v.transpose(1, 2)
        return {"q": torch.cat(q), "k": k.contiguous(), "v": v.contiguous(),
                "lens": _i32(lens)}
    out, t, g = [], 0, hq // hk
    for b in range(c["batch"]):
        page = torch.from_numpy(table[b, :-(-lens[b] // ps)].astype(np.int64)).cuda()
        o = torch.empty(n[b], hq, D, dtype=torch.float64, device="cuda")
        hide = torch.arange(lens[b], device="cuda")[None] > \
            torch.arange(lens[b] - n[b], lens[b], device="cuda")[:, None]
        for h in range(hk):
            k, v = (st[x][page, h].reshape(-1, D)[:lens[b]].double() for x in ("k", "v"))
            q = st["q"][t:t + n[b], h * g:(h + 1) * g].double()
            a = torch.einsum("ngd,td->gnt", q, k) / 8.0
            w = torch.softmax(a.masked_fill(hide, -math.inf), dim=-1)
            o[:, h * g:(h + 1) * g] = torch.einsum("gnt,td->ngd", w, v)
        out.append(o)
        t += n[b]
    return {"out": torch.cat(out)}
