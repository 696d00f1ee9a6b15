"""kvd_paged_attn: many positions of little weight beside one of much (a position that every token
attends to, and a long rest)."""

import pytest
import torch

import ref64
import ref64_serving as ref
from gpu_util import require_gpu
from paged_util import Batch

pytestmark = pytest.mark.gpu
F16, BF16 = torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def sink(rows, hq, hk, dtype, at, score):
    """Position `at` of every row has this score, the others 0; V is 0 there, near 1 elsewhere."""
    b = Batch(rows, hq, hk, 64, dtype, seed=1)
    b.q.fill_(1.0)
    for row, (_, length) in enumerate(rows):
        pages = b.table[row, :-(-length // 64)].long()
        b.k[pages] = 0.0
        b.v[pages] = (1 + b.v[pages].nan_to_num(0.0) / 16).to(dtype)
        b.k[b.table[row, at // 64].long(), :, at % 64] = score / 8
        b.v[b.table[row, at // 64].long(), :, at % 64] = 0.0
    return b


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("score", [10.0, 16.0, 17.75, 19.0, 21.0])
@pytest.mark.parametrize("rows,at", [([(1, 131072)], 0), ([(1, 100000), (40, 30000)], 3),
                                     ([(30, 65536)], 40000), ([(5, 20000), (1, 777)], 700)])
def test_a_long_rest_keeps_its_weight(rows, at, score, dtype):
    """A weight of 2^(s - m) is held in 16 bits. binary16 has steps of 2^-24 at its lower end, so
    half a step is lost of 2^7 times the weight at most: 2^-32 of the reference's. (That is the
    bound's absolute term, 2^-25 of the form's `low` less 7 bits.)"""
    b = sink(rows, 4, 1, dtype, at, score)
    out = b.attend()
    table = b.table.cpu()
    for row, (n, length) in enumerate(rows):
        s = b.host_starts[row]
        k, v = ref.paged_rows(b.k, b.v, table, row, length)
        want, mag, size, low = ref.chunk_attention(b.q[s:s + n].double(), k, v, 0.125)
        tol = ref64.attention_bound(want, mag, size, dtype,
                                    floor=low * 2.0 ** -7 if dtype == F16 else 0.0)
        err = (out[s:s + n].double() - want).abs()
        assert (err <= tol).all(), (row, float(err.max()), float(want.max()), float(tol.min()))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_weights_up_to_the_largest(dtype):
    """Scores that grow by less than the reference's slack from tile to tile: weights of 2^8 and
    sums of a tile of them stay in the range of the storage type."""
    b = Batch([(1, 4000), (100, 1500)], 4, 1, 16, dtype, seed=3)
    b.q.fill_(1.0)
    for row, (_, length) in enumerate(b.rows):
        for t in range(length):
            # a tile of 128 positions 5.5 nats (7.9 bits) above the one before, for ten tiles
            b.k[int(b.table[row, t // 16]), :, t % 16] = 5.5 / 8 * min(t // 128, 10)
    b.check(b.attend())
