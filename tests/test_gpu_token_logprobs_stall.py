"""kvd_token_logprobs with a wait that runs out: the row's outputs are left as they were, whichever
of the blocks that share the row it is."""

import pytest
import torch

from gpu_util import new_err, require_gpu
from test_gpu_token_logprobs import check, run, tokens_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


# (a row of one block; of sixteen, rows 0 .. 15 stalled in block 0 .. 15; of two)
@pytest.mark.parametrize("R,V", [(1, 1000), (400, 9000), (16, 128000), (100, 20000)])
@pytest.mark.parametrize("given,top", [(1, 1), (16, 32)])
def test_rows_are_left(R, V, given, top):
    import kv_cached_decode_gb300 as kvd

    x = torch.randn(R, V, device="cuda")
    t = tokens_for(R, given, V) if given else None
    err = new_err()
    out = run(x, t, top, dev_err=err, flags=kvd.KVD_FLAG_TEST_STALL)
    assert int(err) == 20
    for name, v in out.items():
        assert (v == (-9 if v.dtype == torch.int32 else 9.0)).all(), name
    err = new_err()
    out = run(x[:20], None if t is None else t[:20], top, dev_err=err)  # and nothing is left behind
    check(out, x[:20], None if t is None else t[:20], top)
    assert int(err) == 0
