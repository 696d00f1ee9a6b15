"""kvd_paged_append reads nothing of tokens that belong to no row (a padded batch may not have them).
A read cannot be seen in a result, and one out of range must not run, so the source is checked:
rows are loaded within a test of the token against the outermost entries of `starts` alone."""

import os
import re

from test_cluster_start import CSRC, body


def block(text, at):
    """The braces that open behind `at`."""
    depth, start = 0, text.index("{", at)
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return start, i
    raise AssertionError("unbalanced")


def test_tokens_of_no_row_are_not_read():
    with open(os.path.join(CSRC, "paged_append.cu"), encoding="utf-8") as f:
        text = body(f.read(), "paged_append_kernel")
    bounds = text.index("const int first = p.starts[0], end = min(p.starts[p.batch], p.n_tokens);")
    test = text.index("if (t >= first && t < end) {")
    start, end = block(text, test)
    assert bounds < test
    reads = [m.start() for m in re.finditer(r"\*reinterpret_cast<const uint4\*>\(", text)]
    assert reads and all(start < at < end for at in reads)
    assert len(re.findall(r"p\.x\[", text)) == len(re.findall(r"p\.x\[", text[start:end]))
