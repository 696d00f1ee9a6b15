"""The calls of a decoder-only step together, as a program would chain them: a prompt through a
windowed layer, then tokens one by one -- head norm with rotation, append, windowed attention,
filtered sampling -- over the 4-bit and over the 16-bit cache; every stage against 64 bits on
the values the stage before it produced, and the whole chain captured in a graph with dependent
launches, replayed, equal to the eager chain."""

import numpy as np
import pytest
import torch

import ref64
from gpu_util import new_err, require_gpu

pytestmark = pytest.mark.gpu
B, HQ, HK, CAP, V = 3, 8, 2, 300, 3000
WINDOW, SINKS, BASE, EPS = 48, 4, 10000.0, 1e-6
STEPS = 6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Layer:
    """One layer's weights and buffers. The embedding of a token is its fused projection."""

    def __init__(self, q4):
        import kv_cached_decode_gb300 as kvd

        g = torch.Generator(device="cuda").manual_seed(9)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.emb = r(V, HQ + 2 * HK, 64).half()
        self.wq, self.wk = (1 + 0.2 * r(64)).half(), (1 + 0.2 * r(64)).half()
        self.head = r(HQ * 64, V) * 0.4
        self.q4 = q4
        if q4:
            self.cache = kvd.new_q4_cache(B, HK, CAP)
        else:
            self.kv = torch.zeros(2, B, HK, CAP, 64, dtype=torch.float16, device="cuda")
            self.cache = kvd.make_cache(self.kv[0], self.kv[1])
        op = kvd.KVD_OP_Q4_ATTN if q4 else kvd.KVD_OP_WINDOW_ATTN
        self.ws = kvd.new_workspace(kvd.kvd_workspace_size(op, B, HQ, HK, 1, 1, CAP))
        e = lambda *s, t=torch.float16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
        self.q, self.k, self.out = e(B, HQ, 1, 64), e(B, HK, 1, 64), e(B, HQ, 1, 64)
        self.lens, self.lens_out = e(B, t=torch.int32), e(B, t=torch.int32)
        self.token, self.n_kept = e(B, t=torch.int32), e(B, t=torch.int32)
        self.logprob, self.u = e(B, t=torch.float32), e(B, t=torch.float32)
        self.T = torch.tensor([0.7, 1.0, 1.3], device="cuda")
        self.top_k = torch.tensor([40, 0, 300], dtype=torch.int32, device="cuda")
        self.top_p = torch.tensor([0.9, 0.95, 1.0], device="cuda")
        self.min_p = torch.tensor([0.0, 0.0, 0.02], device="cuda")
        self.err = new_err()

    def rotate(self, qkv, q, k, pos0, flags=0):
        """qkv [B, n, heads, 64]: normed and rotated q and k, and v, [B, heads, n, 64]."""
        import kv_cached_decode_gb300 as kvd

        h = qkv.transpose(1, 2)
        kvd.kvd_qk_norm_rope(h[:, :HQ], h[:, HQ:HQ + HK], q, k, self.wq, self.wk, pos0, EPS, BASE,
                             flags=flags, dev_err=self.err)
        return h[:, HQ + HK:].contiguous()

    def prompt(self, tokens, plens):
        """A ragged prompt [B, n] through the windowed layer; returns its attention."""
        import kv_cached_decode_gb300 as kvd

        n = tokens.shape[1]
        qkv = self.emb[tokens.long()]
        q = torch.empty(B, HQ, n, 64, dtype=torch.float16, device="cuda")
        k = torch.empty(B, HK, n, 64, dtype=torch.float16, device="cuda")
        zero = torch.zeros(B, dtype=torch.int32, device="cuda")
        v = self.rotate(qkv, q, k, zero)
        out = torch.empty_like(q)
        if self.q4:  # attention on a 16-bit cache of the prompt, the rows kept in 4 bits
            kv = torch.zeros(2, B, HK, n, 64, dtype=torch.float16, device="cuda")
            kvd.kvd_prefill_window_attn(q, kvd.make_cache(kv[0], kv[1]), k, v, plens, out, WINDOW,
                                        SINKS, dev_err=self.err)
            kvd.kvd_q4_append(self.cache, k, v, zero, self.lens, counts=plens, dev_err=self.err)
        else:
            kvd.kvd_prefill_window_attn(q, self.cache, k, v, plens, out, WINDOW, SINKS,
                                        lens_in=zero, lens_out=self.lens, dev_err=self.err)
        return qkv, q, k, v, out

    def step(self, flags=0):
        import kv_cached_decode_gb300 as kvd

        qkv = self.emb[self.token.long()][:, None]
        v = self.rotate(qkv, self.q, self.k, self.lens, flags)
        if self.q4:
            kvd.kvd_q4_append(self.cache, self.k, v, self.lens, self.lens_out, flags=flags,
                              dev_err=self.err)
            kvd.kvd_q4_attn(self.q, self.cache, self.out, self.ws, lens=self.lens_out,
                            window=WINDOW, n_sinks=SINKS, flags=flags, dev_err=self.err)
        else:
            kvd.kvd_window_attn(self.q, self.cache, self.out, self.ws, WINDOW, SINKS,
                                lens=self.lens, append=(self.k, v, self.lens_out), flags=flags,
                                dev_err=self.err)
        logits = self.out.reshape(B, HQ * 64).float() @ self.head
        kvd.kvd_sample_filtered(logits, self.u, self.token, self.T, self.top_k, self.top_p,
                                self.min_p, self.logprob, self.n_kept, flags=flags,
                                dev_err=self.err)
        self.lens.copy_(self.lens_out)
        return qkv, v, logits

    def values(self, b, L):
        """The cached K and V of row b as float64, and the size of K's parts."""
        if not self.q4:
            k, v = (self.kv[i, b, :, :L].double().cpu() for i in (0, 1))
            return k, v, k.abs()
        kd, vd, par = (t[b, :, :L].cpu().numpy() for t in self.cache._tensors)
        f = lambda *a, **kw: torch.from_numpy(ref64.q4_values(*a, **kw))  # noqa: E731
        return (f(kd, par[..., :2]), f(vd, par[..., 2:]), f(kd, par[..., :2], size=True))


def _near_norm(got, x, w, pos):
    want, mag = ref64.norm_rope(x.double().cpu().numpy(), w.double().cpu().numpy(), pos, EPS, BASE)
    err = mag * 2.0 ** -18  # as in the call's own tests
    tol = err + 2.0 ** -11 * (np.abs(want) + err) + 2.0 ** -24
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()


def _start(layer):
    g = torch.Generator(device="cuda").manual_seed(10)
    tokens = torch.randint(0, V, (B, 90), generator=g, device="cuda", dtype=torch.int32)
    plens = torch.tensor([90, 51, 1], dtype=torch.int32, device="cuda")
    got = layer.prompt(tokens, plens)
    layer.token.copy_(torch.tensor([5, 6, 7], dtype=torch.int32))
    return plens, got


def _uniforms():
    return torch.rand(STEPS, B, generator=torch.Generator().manual_seed(11)).cuda()


@pytest.mark.parametrize("q4", [False, True])
def test_every_stage_of_the_chain(q4):
    layer = Layer(q4)
    plens, (qkv, q, k, v, out) = _start(layer)
    assert torch.equal(layer.lens, plens)
    h = qkv.transpose(1, 2)
    pos = np.arange(90)[None].repeat(B, 0)
    _near_norm(q, h[:, :HQ], layer.wq, pos)
    _near_norm(k, h[:, HQ:HQ + HK], layer.wk, pos)
    for b in range(B):
        m = int(plens[b])
        see = ref64.visible(m, m, True, WINDOW, SINKS)
        want, mag, smax = ref64.attention(q[b, :, :m].double().cpu(), k[b, :, :m].double().cpu(),
                                          v[b, :, :m].double().cpu(), see, 0.125)
        tol = ref64.attention_bound(want, mag, smax, torch.float16)
        assert ((out[b, :, :m].double().cpu() - want).abs() <= tol).all()
    us = _uniforms()
    for s in range(STEPS):
        layer.u.copy_(us[s])
        before = layer.lens.clone()
        qkv, v, logits = layer.step()
        torch.cuda.synchronize()
        assert int(layer.err) == 0 and torch.equal(layer.lens, before + 1)
        h = qkv.transpose(1, 2)
        pos = before.cpu().numpy()[:, None].astype(np.int64)
        _near_norm(layer.q, h[:, :HQ], layer.wq, pos)
        _near_norm(layer.k, h[:, HQ:HQ + HK], layer.wk, pos)
        for b in range(B):
            L = int(layer.lens[b])
            kk, vv, size = layer.values(b, L)
            if not q4:
                assert torch.equal(kk[:, -1:], layer.k[b].double().cpu())
            see = ref64.visible(L, 1, True, WINDOW, SINKS)
            want, mag, smax = ref64.attention(layer.q[b].double().cpu(), kk, vv, see, 0.125, size)
            floor = L * 2.0 ** -25 * float(vv.abs().max()) * 4 if q4 else 0.0
            tol = ref64.attention_bound(want, mag, smax, torch.float16, floor=floor)
            assert ((layer.out[b].double().cpu() - want).abs() <= tol).all()
            f = lambda t: float(t[b])  # noqa: E731
            w = ref64.sample(logits[b].cpu().numpy(), float(us[s, b]), f(layer.T),
                             int(layer.top_k[b]), f(layer.top_p), f(layer.min_p))
            assert int(layer.token[b]) == w[0] and int(layer.n_kept[b]) == w[2]
            assert abs(f(layer.logprob) - w[1]) <= 1e-5


@pytest.mark.parametrize("q4", [False, True])
def test_a_captured_chain_equals_the_eager_one(q4):
    import kv_cached_decode_gb300 as kvd

    us = _uniforms()
    eager, graphed = Layer(q4), Layer(q4)
    _start(eager)
    _start(graphed)
    want = []
    for s in range(STEPS):
        eager.u.copy_(us[s])
        eager.step()
        want.append(eager.token.tolist())
    # warm up on copies of the state, then capture one step and replay it
    state = [t.clone() for t in (graphed.token, graphed.lens)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.step(kvd.KVD_FLAG_PDL)
    torch.cuda.current_stream().wait_stream(side)
    for t, x in zip((graphed.token, graphed.lens), state):
        t.copy_(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step(kvd.KVD_FLAG_PDL)
    got = []
    for s in range(STEPS):
        graphed.u.copy_(us[s])
        graph.replay()
        got.append(graphed.token.tolist())
    assert got == want and int(graphed.err) == 0
    assert torch.equal(graphed.out, eager.out) and torch.equal(graphed.lens, eager.lens)
