"""Properties of the kernels' sources that no run can be relied on to show."""
import glob
import os
import re

import pytest

from block_sparse_long_10_b200 import build as qbuild

SOURCES = sorted(glob.glob(os.path.join(qbuild.CSRC, "*.cu*")))


def _statements(text):
    """asm statements, whole: up to the closing parenthesis."""
    for m in re.finditer(r"\basm\s*(volatile)?\s*\(", text):
        depth, at, quoted = 1, m.end(), False
        while depth:
            c = text[at]
            if c == '"' and text[at - 1] != "\\":
                quoted = not quoted
            elif not quoted:
                depth += (c == "(") - (c == ")")
            at += 1
        yield text[m.start():at]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_asynchronous_copies_are_ordered_with_plain_accesses(path):
    """An asm statement that starts, commits or waits for copies into shared memory tells the
    compiler that memory changes: without it ordinary loads of the copied bytes may be moved
    across the wait."""
    for s in _statements(open(path).read()):
        if "cp.async" in s:
            assert s.startswith("asm volatile") and '"memory"' in s, (os.path.basename(path), s)


def _body(text, at):
    """The braces that open behind `at`, with what they enclose."""
    start = text.index("{", at)
    depth, at = 1, start + 1
    while depth:
        depth += (text[at] == "{") - (text[at] == "}")
        at += 1
    return text[start:at]


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_dependent_kernels_wait_before_they_return(path):
    """A kernel launched under its predecessor that ends without waiting for it lets what comes
    next in the stream start while the predecessor still runs."""
    text = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"__global__", text):
        body = _body(text, m.end())
        if "griddep_wait();" in body:
            before = body[:body.index("griddep_wait();")]
            # (a lambda's return ends the lambda)
            before = re.sub(r"\[[&=]?\]\s*\([^)]*\)\s*\{[^{}]*\}", "", before)
            assert not re.search(r"\breturn\b", before), os.path.basename(path)
