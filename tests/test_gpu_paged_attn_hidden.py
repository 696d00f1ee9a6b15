"""kvd_paged_attn: what stands behind the mask does not reach an output, whatever it is, and what a
token sees does; stretches of tokens that overlap."""

import math

import pytest
import torch

from gpu_util import new_err, require_gpu
from paged_util import Batch

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def put(b, pool, row, pos, head, dim, value):
    pool[b.table[row, pos // b.page].long(), head, pos % b.page, dim] = value


# (row, position from the row's end, KV head, dim, value)
ODD = [(0, 1, 0, 3, INF), (0, 2, 1, 63, NAN), (0, 1, 0, 4, -INF), (0, 3, 0, 4, INF),
       (1, 1, 0, 0, NAN), (1, 33, 1, 17, INF), (1, 30, 1, 17, -INF), (1, 2, 0, 31, -INF),
       (2, 1, 1, 5, NAN), (3, 1, 0, 8, INF), (3, 100, 0, 9, -INF), (3, 100, 0, 10, NAN)]


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", [1, 3, 4, 16, 128])
@pytest.mark.parametrize("rows", [
    [(4, 300), (40, 41), (1, 20), (130, 1000)],
    [(4, 4), (60, 500), (1, 129), (200, 333)] + [(2, 128 * i + 1) for i in range(1, 40)],
    [(3, 9000), (33, 129), (1, 64), (110, 257)],
])
def test_infinities_and_nans_of_new_tokens(rows, group, dtype):
    b = Batch(rows, 2 * group, 2, 16, dtype, seed=group)
    at = [(row, rows[row][1] - back, h, d, v) for row, back, h, d, v in ODD]
    for row, pos, h, d, _ in at:
        put(b, b.v, row, pos, h, d, 0.0)
    plain = b.attend()
    b.check(plain)
    for row, pos, h, d, v in at:
        put(b, b.v, row, pos, h, d, v)
    out = b.attend()
    extra = torch.zeros_like(out, dtype=torch.float32)  # what the positions that a token sees add
    for row, pos, h, d, v in at:
        n, length = rows[row]
        first = b.host_starts[row] + max(pos - (length - n), 0)
        extra[first:b.host_starts[row] + n, h * group:(h + 1) * group, d] += v
    clean = extra == 0
    assert torch.equal(out[clean], plain[clean])
    # an infinity that is seen makes the output that infinity, or NaN where a product by a weight of
    # 0 meets it (a weight that is rounded to 0, or the same vector held several times)
    assert out[extra.isnan()].isnan().all() and not out[~clean].isfinite().any()
    assert ((out.float() == extra) | out.isnan())[~clean].all()
    # and nothing of it stays for the next call
    for row, pos, h, d, _ in at:
        put(b, b.v, row, pos, h, d, 0.0)
    assert torch.equal(b.attend(), plain)


@pytest.mark.parametrize("group", [1, 4])
def test_infinities_and_nans_among_the_keys(group):
    """A key that a token does not see changes nothing; the others' outputs are theirs."""
    rows = [(4, 300), (40, 41), (130, 1000)]
    b = Batch(rows, 2 * group, 2, 16, F16, seed=group)
    plain = b.attend()
    for row, (_, length) in enumerate(rows):
        for dim, v in ((0, NAN), (1, INF), (2, -INF)):
            put(b, b.k, row, length - 1, 0, dim, v)
    out = b.attend()
    last = [b.host_starts[row] + n - 1 for row, (n, _) in enumerate(rows)]
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[last, :group] = True
    assert torch.equal(out[~hit], plain[~hit]) and out[hit].isnan().all()


def test_a_whole_row_of_odd_values_in_every_new_token():
    """Every token sees its own. The first unit (32 tokens) meets infinities only where
    not all of its tokens see them."""
    b = Batch([(70, 200)], 4, 1, 16, BF16)
    for pos in range(130, 200):
        put(b, b.v, 0, pos, 0, slice(0, 32), INF)
        put(b, b.v, 0, pos, 0, slice(32, 64), NAN)
    out = b.attend()
    assert (out[:32, :, :32] == INF).all() and out[:, :, 32:].isnan().all()
    assert not out.isfinite().any() and not (out == -INF).any()


@pytest.mark.parametrize("T,rows", [(8192, 128), (14000, 32)])
def test_overlapping_stretches_too_long_for_the_list(T, rows):
    """Tokens claimed by half the rows of 2^19 positions each: more tiles than the list can
    count."""
    page = 65536
    b = Batch([(1, 8)], 128, 1, page, F16)
    b.starts = torch.tensor([0, T] * (rows // 2) + [0], dtype=torch.int32, device="cuda")
    b.lens = torch.full((rows,), 8 * page, dtype=torch.int32, device="cuda")
    b.table = torch.zeros(rows, 8, dtype=torch.int32, device="cuda")
    b.q = torch.zeros(T, 128, 64, dtype=F16, device="cuda")
    b.rows = [(T, 8 * page)] * rows
    err = new_err()
    out = b.attend(dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 16 and (out == 7.0).all()


def test_overlapping_stretches_that_fit():
    """Two rows of the same tokens, lengths and pages: the outputs are theirs."""
    b = Batch([(5, 100), (1, 30)], 4, 2, 16, F16)
    plain = b.attend()
    b.starts = torch.tensor([0, 5, 0], dtype=torch.int32, device="cuda")
    err = new_err()
    out = b.attend(dev_err=err)
    assert int(err) == 16 and torch.equal(out[:5], plain[:5]) and (out[5:] == 7.0).all()
