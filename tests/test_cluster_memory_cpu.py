"""Kernels whose CTAs reach into one another's shared memory first wait until all of the cluster run.

That order is in the source and nowhere else: without it a run nearly always goes well, so no result
shows it missing.  Read here from the kernels' text: the first access through a mapped address comes
after a barrier of the whole cluster that every thread passes.
"""
import glob
import os
import re

import pytest

from exact_io_aware_gb300.build import CSRC

BARRIER = r"\bcluster\.(?:sync|barrier_wait)\(|\bsync_cluster\(\)"


def code(path):
    with open(path) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def bodies(text):
    """Each kernel's name and body."""
    for m in re.finditer(r"__global__[^{;]*?(\w+)\s*\((?:[^(){};]|\([^()]*\))*\)\s*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1), text[m.end():i]


def first_access(body):
    """Where a mapped address is first read or written: at once, or by the name that it was given."""
    at = [m.start() for m in re.finditer(r"map_shared_rank\([^()]*\)\s*(?:->|\[)", body)]
    for name in re.findall(r"(\w+)\s*=\s*cluster\.map_shared_rank\(", body):
        at += [m.start() for m in re.finditer(rf"\b{name}\s*(?:->|\[)|\*\s*{name}\b(?!\s*=)", body)]
    return min(at)


KERNELS = [(os.path.basename(path), name, body) for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*")))
           for name, body in bodies(code(path)) if "map_shared_rank(" in body]


def test_the_kernels_are_found():
    texts = [code(path) for path in glob.glob(os.path.join(CSRC, "*.cu*"))]
    assert sum(x.count("map_shared_rank(") for x in texts) == sum(x.count("map_shared_rank(") for _, _, x in KERNELS)
    assert {x[:2] for x in KERNELS} >= {("draft_verify.cu", "verify_kernel")}


@pytest.mark.parametrize("file,name,body", KERNELS, ids=[x[1] for x in KERNELS])
def test_a_barrier_comes_first(file, name, body):
    barriers = [m.start() for m in re.finditer(BARRIER, body)]
    assert barriers and min(barriers) < first_access(body), (file, name)
