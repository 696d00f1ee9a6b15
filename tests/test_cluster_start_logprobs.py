"""As test_cluster_start.py, for the kernel of kvd_token_logprobs."""

import os
import re

from test_cluster_start import BARRIER, CSRC, REMOTE, body


def test_a_cluster_barrier_before_the_first_remote_access():
    source = open(os.path.join(CSRC, "token_logprobs.cu"), encoding="utf-8").read()
    text = body(source, "token_logprobs_kernel")
    remote, barrier = re.search(REMOTE, text), re.search(BARRIER, text)
    assert remote and barrier and barrier.start() < remote.start()
    # every block of a cluster arrives there before it waits
    assert re.search(r"if \(p\.cluster > 1\) cluster_arrive_relaxed\(\);", text).start() < barrier.start()
