"""Shared memory of another CTA of a cluster may be touched only once that CTA has started: in
the kernels that exchange through it, a cluster barrier stands before the first access. Checked
in the sources, as the other way round must not run."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "kv_cached_decode_gb300", "csrc")
REMOTE = r"\b(st_cluster_\w+|ld_cluster\w*|st_async_v4|map_shared)\s*\("
BARRIER = r"\b(cluster_wait|cluster_sync_q4|cluster_sync_all|sync_row)\s*\("
# a kernel's helpers, as far as they touch other CTAs, are called behind its own first access
KERNELS = [("sample_filtered.cu", "sample_filtered_kernel"), ("q4_attn.cu", "q4_attn_kernel"),
           ("beam_select.cu", "beam_select_kernel"), ("sample_accept.cu", "sample_accept_kernel")]


def body(source, kernel):
    """The kernel's body without comments."""
    at = re.search(r"__global__[^;{]*\b%s\(" % kernel, source).start()
    text = re.sub(r"//[^\n]*", "", source[at:])
    depth, start = 0, text.index("{")
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i]
    raise AssertionError("unbalanced")


@pytest.mark.parametrize("file,kernel", KERNELS)
def test_a_cluster_barrier_before_the_first_remote_access(file, kernel):
    text = body(open(os.path.join(CSRC, file), encoding="utf-8").read(), kernel)
    remote, barrier = re.search(REMOTE, text), re.search(BARRIER, text)
    assert remote and barrier and barrier.start() < remote.start(), text[remote.start():][:60]
