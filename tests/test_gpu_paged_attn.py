"""kvd_paged_attn against its 64-bit form: row mixes, groups, page sizes and layouts, splits,
tokens of no row, stale slots, lengths that do not fit, pages outside the pool."""

import pytest
import torch

from gpu_util import new_err, require_gpu
from paged_util import Batch

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 128, 200])
def test_one_token(dtype, length):
    b = Batch([(1, length)], 4, 1, 16, dtype, seed=length)
    b.check(b.attend())


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 31, 33, 64, 65, 128])
def test_groups(group):
    b = Batch([(1, 100), (3, 300), (0, 50), (2, 2), (40, 130)], 2 * group, 2, 16, BF16, seed=group)
    b.check(b.attend())


@pytest.mark.parametrize("order", ["head", "token"])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_pages(page, order):
    b = Batch([(1, 257), (5, 100), (70, 70), (1, 8), (2, 1000)], 8, 2, page, F16, order, page)
    b.check(b.attend())


@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 1), (6, 2), (20, 20), (8, 1)])
@pytest.mark.parametrize("n,length", [(1, 3000), (130, 130), (129, 700), (300, 333), (17, 2049)])
def test_one_row(hq, hk, n, length):
    b = Batch([(n, length)], hq, hk, 16, F16, seed=n)
    b.check(b.attend())


def test_one_long_row_over_many_blocks():
    b = Batch([(1, 40000)], 4, 1, 64, F16, seed=5)
    b.check(b.attend())


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_mixed_batch(dtype):
    rows = [(600, 900), (200, 4000)] + [(1, 37 * i + 1) for i in range(40)] + [(5, 512), (16, 16)]
    b = Batch(rows, 8, 2, 16, dtype, "token", 3)
    b.check(b.attend())


@pytest.mark.parametrize("rows", [33, 100, 700])
def test_many_rows(rows):
    b = Batch([((i * 7) % 4, 1 + (i * 131) % 300 + 4) for i in range(rows)], 4, 2, 8, BF16,
              seed=rows)
    b.check(b.attend())


def test_tokens_of_no_row_are_left():
    b = Batch([(3, 90), (0, 10), (2, 65)], 4, 2, 16, F16, lead=5, trail=9)
    b.check(b.attend())


def test_scores_of_any_size_and_sign():
    for peak, scale in ((16.0, 0.125), (4.0, -0.5), (1.0, 0.0), (1.0, 1e-30)):
        b = Batch([(1, 500), (150, 400)], 4, 2, 16, F16, seed=9, peak=peak)
        b.check(b.attend(scale=scale), scale=scale)


def test_growing_scores_move_the_reference():
    """Keys whose scores grow along the row, past every reference taken before."""
    b = Batch([(1, 2000), (100, 1000)], 4, 1, 16, F16, seed=2)
    b.q.fill_(1.0)
    for row, (_, length) in enumerate(b.rows):
        for t in range(0, length):
            pg, at = int(b.table[row, t // 16]), t % 16
            b.k[pg, :, at] = t / 128.0
    b.check(b.attend())


def test_strided_queries_of_a_fused_projection():
    b = Batch([(4, 100), (1, 30)], 6, 2, 16, BF16)
    qkv = torch.randn(b.T, 10, 64, device="cuda").to(BF16)
    qkv[:, :6] = b.q
    b.check(b.attend(q=qkv[:, :6]))
    heads_first = b.q.transpose(0, 1).contiguous().transpose(0, 1)
    b.check(b.attend(q=heads_first))


def test_a_loose_bound_and_a_shared_workspace():
    b = Batch([(5, 3000), (1, 9000), (64, 200)], 8, 1, 16, F16, seed=1)
    ws = b.workspace(200)
    for _ in range(3):
        b.check(b.attend(max_new=200, workspace=ws))
    assert (ws[:65536] == 0).all()


def test_the_same_bits_on_every_run():
    b = Batch([(5, 3000), (1, 9000), (64, 200)], 8, 1, 16, F16, seed=1)
    first = b.attend()
    for _ in range(5):
        assert torch.equal(b.attend(), first)


def test_shared_pages():
    """Two rows with the same prefix pages."""
    b = Batch([(1, 200), (3, 200)], 4, 2, 16, F16, seed=4)
    b.table[1, :10] = b.table[0, :10]
    b.check(b.attend())


def test_rows_that_do_not_fit_are_flagged_and_left():
    rows = [(2, 100), (3, 70), (1, 60), (4, 50), (1, 40)]
    for row, length in ((1, 2), (2, 1 << 20), (3, -5)):
        b = Batch(rows, 4, 2, 16, F16, seed=row)
        b.lens[row] = length
        err = new_err()
        b.check(b.attend(dev_err=err), skip=(row,))
        assert int(err) == 16
    b = Batch(rows, 4, 2, 16, F16)
    err = new_err()
    b.check(b.attend(max_new=3, dev_err=err), skip=(3,))  # 4 new tokens
    assert int(err) == 16
    # a row that ends behind the packed tokens
    b = Batch(rows, 4, 2, 16, F16)
    b.starts[5] += 3
    err = new_err()
    b.check(b.attend(dev_err=err), skip=(4,))
    assert int(err) == 16
    # nothing to do at all
    b = Batch([(0, 10), (0, 0)], 4, 2, 16, F16, trail=2)
    err = new_err()
    b.check(b.attend(dev_err=err))
    assert int(err) == 0


def test_pages_outside_the_pool_count_as_zeros():
    for bad in (-1, 1 << 29, -(1 << 31)):
        b = Batch([(1, 100), (70, 300), (2, 50)], 4, 2, 16, F16, seed=6)
        b.table[1, 3] = bad
        b.table[0, 0] = b.n_pages
        err = new_err()
        b.check(b.attend(dev_err=err))
        assert int(err) == 17


def test_captured_and_replayed_with_other_lengths():
    b = Batch([(1, 5000), (1, 300), (1, 64)], 8, 2, 16, BF16, seed=8)
    out, ws = torch.full_like(b.q, 7.0), b.workspace(1)
    b.attend(out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.attend(out=out, workspace=ws)
    for lens in ([5000, 300, 64], [17, 299, 1], [4000, 1, 33]):
        b.rows = [(1, x) for x in lens]
        b.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        b.check(out)


def test_two_streams_with_a_workspace_each():
    a = Batch([(1, 20000), (30, 400)], 4, 1, 16, F16, seed=1)
    b = Batch([(3, 10000)], 4, 1, 32, F16, seed=2)
    s = torch.cuda.Stream()
    wa, wb = a.workspace(30), b.workspace(3)
    oa, ob = torch.full_like(a.q, 7.0), torch.full_like(b.q, 7.0)
    torch.cuda.synchronize()
    for _ in range(10):
        a.attend(out=oa, workspace=wa)
        b.attend(out=ob, workspace=wb, stream=s)
    a.check(oa)
    b.check(ob)


def test_a_wait_that_runs_out_is_reported():
    import kv_cached_decode_gb300 as kvd

    b = Batch([(1, 300), (80, 200)], 4, 2, 16, F16)
    err = new_err()
    out = b.attend(dev_err=err, flags=kvd.KVD_FLAG_TEST_STALL)
    torch.cuda.synchronize()
    assert int(err) == 20 and (out == 7.0).all()
    b.check(b.attend())  # the stream and the tensor memory are as before
