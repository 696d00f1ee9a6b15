"""kvd_paged_attn: infinities and NaN in V that every token of a row sees, among them the rows of
one token."""

import math

import pytest
import torch

from gpu_util import require_gpu
from paged_util import Batch
from test_gpu_paged_attn_hidden import put

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def check(b, at):
    """at: (row, position, KV head, dim, value), seen by all of the row's tokens. Scores are small,
    so every weight rounds to more than 0: an infinity is the output, both are NaN."""
    for row, pos, h, d, _ in at:
        put(b, b.v, row, pos, h, d, 0.0)
    plain = b.attend()
    b.check(plain)
    for row, pos, h, d, v in at:
        put(b, b.v, row, pos, h, d, v)
    out = b.attend()
    g = b.hq // b.hk
    extra = torch.zeros_like(out, dtype=torch.float32)
    for row, pos, h, d, v in at:
        n, length = b.rows[row]
        assert pos <= length - n
        s = b.host_starts[row]
        extra[s:s + n, h * g:(h + 1) * g, d] += v
    clean = extra == 0
    assert torch.equal(out[clean], plain[clean])
    same = (out.float() == extra) | (out.isnan() & extra.isnan())
    assert same[~clean].all(), (~same & ~clean).nonzero()[:4].tolist()
    assert torch.equal(b.attend().view(torch.int16), out.view(torch.int16))
    # and nothing of it stays for the next call
    for row, pos, h, d, _ in at:
        put(b, b.v, row, pos, h, d, 0.0)
    assert torch.equal(b.attend(), plain)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", [1, 3, 4, 16, 17, 32, 33, 128])
def test_rows_of_one_token(group, dtype):
    rows = [(1, 1), (1, 90), (1, 300), (1, 128), (1, 5000), (1, 129)]
    b = Batch(rows, 2 * group, 2, 16, dtype, seed=group)
    check(b, [(0, 0, 0, 7, INF), (0, 0, 1, 8, NAN), (1, 89, 0, 0, -INF), (1, 31, 1, 63, INF),
              (2, 0, 0, 5, INF), (2, 299, 0, 5, INF), (2, 40, 0, 6, INF), (2, 200, 0, 6, -INF),
              (2, 130, 1, 9, NAN), (3, 127, 1, 1, INF), (4, 0, 0, 2, INF), (4, 4999, 1, 2, -INF),
              (4, 2500, 1, 3, INF), (4, 70, 0, 60, -INF), (5, 128, 0, 33, INF)])


@pytest.mark.parametrize("group", [1, 4, 8])
@pytest.mark.parametrize("n", [2, 3, 4, 20])
def test_blocks_of_tokens(group, n):
    """Beside what only some tokens see in the same unit and dims."""
    rows = [(n, 100), (n, 260), (n, 3000)]
    b = Batch(rows, group, 1, 32, F16, seed=n)
    at = [(0, 3, 0, 5, INF), (1, 20, 0, 5, -INF), (1, 250 - n, 0, 6, INF), (2, 1, 0, 63, INF),
          (2, 2900, 0, 0, -INF), (2, 1500, 0, 1, NAN), (2, 3000 - n, 0, 9, INF)]
    check(b, at)
    # a position that the last token alone sees, in a dim that all see an infinity in, and another
    for row, pos, h, d, v in at + [(r, x - 1, 0, d, NAN) for r, (_, x) in enumerate(rows)
                                   for d in (5, 20)]:
        put(b, b.v, row, pos, h, d, v)
    out = b.attend()
    for row in range(3):
        s = b.host_starts[row]
        assert out[s + n - 1, :, [5, 20]].isnan().all()
        assert out[s:s + n - 1, :, 20].isfinite().all()
    s = b.host_starts[0]
    assert (out[s:s + n - 1, :, 5] == INF).all()


def test_a_whole_cache_of_infinities():
    b = Batch([(1, 700), (3, 400)], 8, 2, 16, BF16)
    b.v.fill_(INF)
    assert (b.attend() == INF).all()
    b.v[..., 32:] = -INF
    out = b.attend()
    assert (out[..., :32] == INF).all() and (out[..., 32:] == -INF).all()
