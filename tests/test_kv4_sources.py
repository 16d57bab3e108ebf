"""What the sources of the 4-bit cache's kernels have to hold to, checked on
the host.

The kernels are launched with programmatic ordering: one may be resident, and
past its first instructions, while the grid before it still writes.  Loads by
the read-only path (ld.global.nc: __ldg, or what the compiler makes of const
__restrict__) are defined only for memory that nobody writes in the reading
kernel's lifetime.  Every buffer that the cache's kernels load can be the
output of the call before: pages, tables, lengths and lists of slots, but also
queries (another call's result) and tokens (another cache's).
"""
import glob
import os
import re

import pytest

from conftest import ROOT

SOURCES = sorted(glob.glob(os.path.join(ROOT, "block_sparse_attention_18_b200", "csrc", "kv4*")))


def code_of(path):
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def test_the_sources_are_found():
    assert len(SOURCES) == 6


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_no_read_only_loads(path):
    found = re.findall(r"\b__ldg\b|__restrict__|\.global\.nc\b|\.L1::no_allocate\.nc\b", code_of(path))
    assert not found, "%s: %s" % (os.path.basename(path), sorted(set(found)))
