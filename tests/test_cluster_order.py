"""No kernel touches another CTA's shared memory before a cluster barrier: until then the
other CTA need not have started. Read from the sources (a run that goes wrong would need a
CTA that starts late, and is not a thing to try)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dsa_sparse_mla_paged_gb300", "csrc")
SOURCES = sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu")))
REMOTE = re.compile(r"map_shared_rank|\bdsm_\w+\(|\bst_async_\w+\(|\bst_cluster_\w+\(|\bmbar_arrive_remote\(|\bmma_commit_to\(")
BARRIER = re.compile(r"\bcluster_sync\(\)|\bcluster_wait\(\)|\bcl\.sync\(\)")


def _kernels(src):
    """(name, body) of each __global__ function."""
    src = re.sub(r"//[^\n]*|/\*.*?\*/", "", src, flags=re.S)
    for m in re.finditer(r"__global__", src):
        at = src.index("{", m.end())
        head, depth, end = src[m.end():at], 0, at
        while True:
            depth += {"{": 1, "}": -1}.get(src[end], 0)
            end += 1
            if depth == 0:
                break
        yield re.findall(r"(\w+)\s*\(", head)[-1], src[at:end]


def _early(src):
    """The kernels that reach another CTA before a barrier."""
    out = []
    for name, body in _kernels(src):
        first = REMOTE.search(body)
        if first and not BARRIER.search(body, 0, first.start()):
            out.append(name)
    return out


@pytest.mark.parametrize("name", SOURCES)
def test_barrier_before_the_first_remote_access(name):
    assert _early(open(os.path.join(CSRC, name)).read()) == []


def test_the_search_finds_what_it_is_for():
    head = "template <int N>\n__global__ void __launch_bounds__(32) k(int* a) {\n  if (a) { a[0] = 1; }\n"
    assert _early(head + "*cl.map_shared_rank(a, 1) = 2; cl.sync(); }") == ["k"]
    assert _early(head + "ptx::cluster_sync(); ptx::st_async_f1(a, 0, 0); }") == []
    assert _early(head + "// cl.sync()\n dsm_st_u32(a, 1); }") == ["k"]
    found = sum(bool(REMOTE.search(body)) for name in SOURCES for _, body in _kernels(open(os.path.join(CSRC, name)).read()))
    assert found >= 5
