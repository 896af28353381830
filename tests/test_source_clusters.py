"""A block of a cluster may write into another's shared memory once that block has started: every kernel that addresses
another block's shared memory goes through a barrier of its cluster before (host only, by the text)."""
import re

import pytest

from test_source_loads import CSRC, code

REMOTE = re.compile(r"\bmap_shared_rank\b|\bmapa_shared\s*\(")
BARRIER = re.compile(r"\bcluster_sync\s*\(|\bcluster_wait\s*\(|\bbarrier_wait\s*\(|\bcluster\.sync\s*\(")


def kernels():
    """(file and name, text) of every kernel."""
    for path in sorted(CSRC.iterdir()):
        if path.suffix not in (".cu", ".cuh"):
            continue
        for text in code(path).split("__global__")[1:]:
            name = re.search(r"\b(\w+_kernel)\s*\(", text)
            yield f"{path.name}: {name.group(1) if name else '?'}", text.split("\n}\n")[0]


REACHING = [(name, text) for name, text in kernels() if REMOTE.search(text)]


def test_some_kernels_reach_others():
    assert len(REACHING) >= 4, [name for name, _ in REACHING]


@pytest.mark.parametrize("name,text", REACHING, ids=[name for name, _ in REACHING])
def test_a_barrier_stands_before_the_first_remote_access(name, text):
    barrier = BARRIER.search(text)
    assert barrier and barrier.start() < REMOTE.search(text).start()
