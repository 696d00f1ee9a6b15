"""A served batch, layer by layer: queries and keys of a fused projection rotated and appended to
pages, attention over them, the chosen tokens scored; prompts in chunks, then single tokens, against
64-bit forms, eager and captured."""

import numpy as np
import pytest
import torch

import ref64
import ref64_serving as ref
from gpu_util import new_err, require_gpu

pytestmark = pytest.mark.gpu
SPEC = dict(base=10000.0, scaling="bands", factor=4.0, original_len=128, low=1.0, high=4.0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


class Server:
    def __init__(self, batch, hq, hk, page, width, dtype):
        import kv_cached_decode_gb300 as kvd

        self.hq, self.hk, self.dtype, self.B = hq, hk, dtype, batch
        i32 = dict(dtype=torch.int32, device="cuda")
        pages = batch * width
        self.k, self.v = (torch.zeros(pages, hk, page, 64, dtype=dtype, device="cuda")
                          for _ in "kv")
        self.table = torch.randperm(pages, device="cuda").to(torch.int32).view(batch, width)
        self.cache = kvd.make_paged_cache(self.k, self.v, self.table)
        self.lens = torch.zeros(batch, **i32)
        self.rope, self.err = kvd.make_rope(**SPEC), new_err()
        self.lens_out = torch.empty_like(self.lens)
        self.rows = [[] for _ in range(batch)]  # every token's projection, on the CPU

    def layer(self, qkv, starts, max_new, q, out, ws, flags=0):
        import kv_cached_decode_gb300 as kvd

        hq, hk = self.hq, self.hk
        kvd.kvd_paged_append(self.cache, qkv[:, hq:hq + hk], qkv[:, hq + hk:], starts, self.lens,
                             lens_out=self.lens_out, q=qkv[:, :hq], q_out=q, rope=self.rope,
                             flags=flags, dev_err=self.err)
        kvd.kvd_paged_attn(q, self.cache, out, ws, starts, self.lens_out, max_new=max_new,
                           flags=flags, dev_err=self.err)

    def check(self, qkv, counts, out):
        torch.cuda.synchronize()
        assert int(self.err) == 0
        hq, hk, t = self.hq, self.hk, 0
        for b, n in enumerate(counts):
            self.rows[b] += list(qkv[t:t + n].double().cpu().numpy())
            if n:
                x = np.stack(self.rows[b])
                pos = np.arange(len(x))[:, None]
                # the cache and the queries hold the rotation rounded to 16 bits: kept as they
                # are for the bound, after a check against the rotation
                got, _ = ref.paged_rows(self.k, self.v, self.table.cpu(), b, len(x))
                want, size = ref.rotate(x[:, hq:hq + hk], pos, SPEC)
                tol = ref.rotation_bound(want, size, self.dtype, len(x))
                assert (np.abs(got.cpu().numpy().transpose(1, 0, 2) - want) <= tol).all()
                q = torch.from_numpy(ref.rotate(x[-n:, :hq], pos[-n:], SPEC)[0]).to(self.dtype)
                v = torch.from_numpy(x[:, hq + hk:].transpose(1, 0, 2).copy()).cuda()
                o, mag, size, low = ref.chunk_attention(q.double().cuda(), got, v, 0.125)
                # a query off by half a 16-bit step moves every score by that much of its size
                h = ref64.HALF[self.dtype]
                tol = ref64.attention_bound(o, mag, size, self.dtype, floor=low) + \
                    mag * 2 * h * size
                bad = ~((out[t:t + n].double() - o).abs() <= tol)
                assert not bad.any(), (b, int(bad.sum()))
            t += n
        self.lens.copy_(self.lens_out)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("hq,hk,page", [(8, 2, 16), (5, 5, 64)])
def test_chunks_then_tokens(dtype, hq, hk, page):
    import kv_cached_decode_gb300 as kvd

    s = Server(4, hq, hk, page, -(-600 // page), dtype)
    g = torch.Generator(device="cuda").manual_seed(hq)
    ws = kvd.new_workspace(kvd.kvd_workspace_size(kvd.KVD_OP_PAGED_ATTN, 4, hq, hk, qlen=300))
    steps = [[200, 64, 1, 0], [300, 1, 1, 33], [1, 1, 0, 5], [1, 1, 1, 1], [5, 5, 5, 5]]
    for step, counts in enumerate(steps):
        T = sum(counts)
        qkv = torch.randn(T, hq + 2 * hk, 64, generator=g, device="cuda").to(dtype)
        starts = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
        q = torch.empty(T, hq, 64, dtype=dtype, device="cuda")
        out = torch.empty_like(q)
        s.layer(qkv, starts, max(counts), q, out, ws, flags=kvd.KVD_FLAG_PDL * (step % 2))
        s.check(qkv, counts, out)


def test_captured_decode_steps_with_their_scores():
    """One captured step, replayed while lengths, inputs and pages' contents move on."""
    import kv_cached_decode_gb300 as kvd

    hq, hk, B, V = 8, 2, 4, 5003
    s = Server(B, hq, hk, 16, 20, torch.bfloat16)
    f32, i32 = dict(dtype=torch.float32, device="cuda"), dict(dtype=torch.int32, device="cuda")
    starts = torch.arange(B + 1, **i32)
    qkv = torch.zeros(B, hq + 2 * hk, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(B, hq, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    ws = kvd.new_workspace(kvd.kvd_workspace_size(kvd.KVD_OP_PAGED_ATTN, B, hq, hk))
    logits, u = torch.zeros(B, V, **f32), torch.zeros(B, **f32)
    token, lp = torch.zeros(B, **i32), torch.zeros(B, **f32)
    score, ent = torch.zeros(B, 1, **f32), torch.zeros(B, **f32)
    top_id, top_lp = torch.zeros(B, 5, **i32), torch.zeros(B, 5, **f32)

    def step():
        s.layer(qkv, starts, 1, q, out, ws, kvd.KVD_FLAG_PDL)
        kvd.kvd_sample_filtered(logits, u, token, logprob=lp, flags=kvd.KVD_FLAG_PDL,
                                dev_err=s.err)
        kvd.kvd_token_logprobs(logits, token[:, None], logprob=score, entropy=ent, top_id=top_id,
                               top_logprob=top_lp, flags=kvd.KVD_FLAG_PDL, dev_err=s.err)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(40):
        qkv.copy_(torch.randn_like(qkv, dtype=torch.float32))
        logits.copy_(torch.randn_like(logits) * 3)
        u.copy_(torch.rand_like(u))
        graph.replay()
        s.check(qkv, [1] * B, out)
        for b in range(B):
            want = ref.logprobs(logits[b].cpu().numpy(), [int(token[b])], 1.0, 5)
            assert abs(float(score[b, 0]) - want[0][0]) <= 2e-5 * abs(want[0][0])
            # the sampler's own log probability of the same token, nothing filtered
            assert abs(float(score[b, 0]) - float(lp[b])) <= 2e-5 * abs(want[0][0])
            assert top_id[b].tolist() == want[4] and abs(float(ent[b]) - want[2]) <= 2e-5 * want[2]
