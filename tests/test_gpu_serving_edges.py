"""The serving calls (scaled rotations, paged append and attention, token log probabilities) where
a program may take them and no other test does: offsets past 32 bits, the largest pages and batches,
launches that overlap, graphs that share a workspace, rows without tokens."""

import numpy as np
import pytest
import torch

from gpu_util import new_err, require_gpu
from paged_util import Batch
from test_gpu_rope_scaled import check as check_rotation
from test_gpu_token_logprobs import check as check_logprobs
from test_gpu_token_logprobs import run as logprobs
from test_gpu_token_logprobs import tokens_for

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# ------------------------------------------------------------ offsets past 32 bits ----
def test_rotation_of_rows_far_apart():
    import kv_cached_decode_gb300 as kvd

    buf = torch.empty((1 << 31) + (1 << 20), dtype=BF16, device="cuda")
    x = buf.as_strided((2, 5, 3, 64), (1 << 31, 3 * 64, 64, 1))
    x.copy_(torch.randn(2, 5, 3, 64, device="cuda"))
    out = torch.empty(2, 5, 3, 64, dtype=BF16, device="cuda")
    kvd.kvd_rope_scaled(k=x, k_out=out, rope=kvd.make_rope())
    torch.cuda.synchronize()
    check_rotation(out, x, np.arange(3), dict())


def far_pages(b):
    """The batch's pages at the end of pools of more than 2^31 elements."""
    n = (1 << 31) // (b.hk * b.page * 64) + b.n_pages + 1
    at = torch.arange(n - b.n_pages, n, device="cuda")
    for name in "kv":
        small = getattr(b, name)
        big = torch.empty(n, b.hk, b.page, 64, dtype=b.dtype, device="cuda")
        big[at] = small
        setattr(b, name, big)
    inside = b.table < b.n_pages
    b.table = torch.where(inside, b.table + (n - b.n_pages), b.table).to(torch.int32)
    b.n_pages = n
    return b


def test_attention_and_append_in_a_pool_past_32_bits():
    import kv_cached_decode_gb300 as kvd

    b = far_pages(Batch([(1, 300), (40, 200), (3, 5)], 8, 2, 16, BF16, seed=1))
    b.check(b.attend())
    qkv = torch.randn(b.T, 12, 64, device="cuda").to(BF16)
    lens = torch.tensor([x - n for n, x in b.rows], dtype=torch.int32, device="cuda")
    kvd.kvd_paged_append(b.cache(), qkv[:, 8:10], qkv[:, 10:], b.starts, lens)
    torch.cuda.synchronize()
    table = b.table.cpu()
    for row, (n, length) in enumerate(b.rows):
        for j in range(n):
            t, pos = b.host_starts[row] + j, length - n + j
            pg = int(table[row, pos // 16])
            assert torch.equal(b.k[pg, :, pos % 16], qkv[t, 8:10])
            assert torch.equal(b.v[pg, :, pos % 16], qkv[t, 10:])
    b.check(b.attend())


def test_tokens_past_32_bits_of_bytes():
    b = Batch([(2, 90), (0, 10), (3, 65)], 128, 2, 16, F16, lead=140000, trail=1)
    assert b.q.numel() * 2 > 1 << 31
    b.check(b.attend(max_new=3))


def test_logits_past_32_bits():
    R, V = 16500, 131072
    x = torch.zeros(R, V, dtype=BF16, device="cuda")
    x[-2:] = torch.randn(2, V, device="cuda").to(BF16) * 3
    tokens = tokens_for(R, 1, V)
    out = logprobs(x, tokens, top=3)
    check_logprobs({k: v[-2:] for k, v in out.items()}, x[-2:], tokens[-2:], 3)


# ------------------------------------------------------------------ sizes -------------
def test_the_largest_pages():
    b = Batch([(1, 70000), (2, 65536), (5, 5)], 4, 1, 65536, F16, seed=3)
    b.check(b.attend())


def test_more_rows_than_the_list_has_entries():
    rows = [(1 if i % 3 else 0, 1 + i % 40) for i in range(4200)]
    rows[4100] = (30, 500)
    b = Batch(rows, 2, 1, 8, F16, seed=4)
    b.check(b.attend())


def test_rows_without_tokens_may_have_any_length():
    b = Batch([(0, 10), (3, 70), (0, 0), (0, 33), (1, 20)], 4, 2, 16, F16)
    b.lens[0], b.lens[2], b.lens[3] = -7, 1 << 30, -(1 << 31)
    err = new_err()
    b.check(b.attend(dev_err=err))
    assert int(err) == 0


def test_the_same_token_asked_for_twice():
    x = torch.randn(5, 5000, device="cuda")
    tokens = torch.tensor([[7, 7, -1, 4999]] * 5, dtype=torch.int32, device="cuda")
    out = logprobs(x, tokens, top=2)
    check_logprobs(out, x, tokens, 2)
    assert torch.equal(out["rank"][:, 0], out["rank"][:, 1])


# ------------------------------------------------------- launches side by side --------
@pytest.mark.parametrize("captured", [False, True])
def test_a_chain_of_overlapping_launches(captured):
    """Append and attention of two layers and the scores, each launched early (PDL), equal to the
    plain launches bit for bit."""
    import kv_cached_decode_gb300 as kvd

    rows, hq, hk = [(1, 700), (33, 100), (2, 2)], 8, 2
    rope = kvd.make_rope(scaling="linear", factor=2.0)
    got = []
    for flags in (0, kvd.KVD_FLAG_PDL):
        layers = [Batch(rows, hq, hk, 16, BF16, seed=s) for s in (1, 2)]
        T = layers[0].T
        ws = layers[0].workspace(33)
        lens = torch.tensor([x - n for n, x in rows], dtype=torch.int32, device="cuda")
        qkv = torch.randn(T, hq + 2 * hk, 64, device="cuda",
                          generator=torch.Generator(device="cuda").manual_seed(5)).to(BF16)
        q = torch.empty(T, hq, 64, dtype=BF16, device="cuda")
        outs = [torch.empty_like(q) for _ in layers]
        top = torch.empty(T, 4, dtype=torch.int32, device="cuda")
        caches = [b.cache() for b in layers]

        def step():
            for b, cache, out in zip(layers, caches, outs):
                kvd.kvd_paged_append(cache, qkv[:, hq:hq + hk], qkv[:, hq + hk:], b.starts, lens,
                                     q=qkv[:, :hq], q_out=q, rope=rope, flags=flags)
                kvd.kvd_paged_attn(q, cache, out, ws, b.starts, b.lens, max_new=33, flags=flags)
            kvd.kvd_token_logprobs(outs[1].view(T, -1), top_id=top, flags=flags)

        step()
        torch.cuda.synchronize()
        if captured:
            for t in outs + [top, q]:
                t.zero_()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            for _ in range(3):
                graph.replay()
            torch.cuda.synchronize()
        else:
            for _ in range(5):
                step()
            torch.cuda.synchronize()
        got.append([t.clone() for t in outs + [top, q]])
    assert all(torch.equal(x, y) for x, y in zip(*got))


def test_two_graphs_that_share_a_workspace_replayed_in_turn():
    a = Batch([(1, 5000), (40, 300)], 8, 2, 16, F16, seed=1)
    b = Batch([(1, 100)] * 50 + [(3, 9000)], 4, 1, 16, BF16, seed=2)
    ws = max((a.workspace(40), b.workspace(3)), key=lambda t: t.numel())
    outs, graphs = [], []
    for x, m in ((a, 40), (b, 3)):
        out = torch.full_like(x.q, 7.0)
        x.attend(out=out, workspace=ws, max_new=m)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            x.attend(out=out, workspace=ws, max_new=m)
        outs.append(out)
        graphs.append(graph)
    for _ in range(4):
        for g, out in zip(graphs, outs):
            out.fill_(7.0)
            g.replay()
    a.check(outs[0])
    b.check(outs[1])


def test_calls_on_two_streams_at_once():
    import kv_cached_decode_gb300 as kvd

    side = torch.cuda.Stream()
    xs = [torch.randn(3, 100000, device="cuda") for _ in range(2)]
    ids = [torch.empty(3, 5, dtype=torch.int32, device="cuda") for _ in range(2)]
    lse = [torch.empty(3, device="cuda") for _ in range(2)]
    x = torch.randn(2, 300, 6, 64, device="cuda").to(F16).transpose(1, 2)
    out = [torch.empty(2, 6, 300, 64, dtype=F16, device="cuda") for _ in range(2)]
    ropes = [kvd.make_rope(), kvd.make_rope(rot_dim=32, interleaved=True)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, stream in enumerate((None, side)):
            kvd.kvd_token_logprobs(xs[i], top_id=ids[i], lse=lse[i], stream=stream)
            kvd.kvd_rope_scaled(x, None, out[i], rope=ropes[i], stream=stream)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(ids[i].long(), xs[i].topk(5).indices)
        assert (lse[i].double() - xs[i].double().logsumexp(1)).abs().max() < 1e-4
        check_rotation(out[i], x, np.arange(300), dict() if i == 0 else dict(rot_dim=32,
                                                                            interleaved=True))


def test_tensors_of_another_device_or_stream_are_refused():
    import kv_cached_decode_gb300 as kvd

    class Elsewhere:
        device_index, cuda_stream = 1, 0

    b = Batch([(1, 20)], 4, 2, 16, F16)
    x = torch.zeros(2, 100, device="cuda")
    lse = torch.full((2,), 9.0, device="cuda")
    for call in (lambda: b.attend(stream=Elsewhere()),
                 lambda: kvd.kvd_token_logprobs(x, lse=lse, stream=Elsewhere()),
                 lambda: kvd.kvd_token_logprobs(x, lse=lse.cpu()),
                 lambda: kvd.kvd_paged_append(b.cache(), b.q[:, :2], b.q[:, 2:], b.starts.cpu(),
                                              b.lens)):
        with pytest.raises(ValueError):
            call()
    assert (lse == 9.0).all()


@pytest.mark.parametrize("pad", [0, 60])
def test_one_long_chunk_of_many_vectors(pad):
    """A unit of 128 vectors cut into many pieces, alone or in a batch padded with empty rows."""
    b = Batch([(0, 5)] * (pad // 2) + [(16, 30000)] + [(0, 9)] * (pad // 2), 8, 1, 64, F16, seed=2)
    first = b.attend()
    b.check(first)
    assert torch.equal(b.attend(), first)
