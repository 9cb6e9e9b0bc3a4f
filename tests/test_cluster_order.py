"""A kernel may touch another CTA's shared memory only once every CTA of its
cluster is known to have started: a cluster barrier comes before the first
remote access.  A late CTA shows this rarely and only as a fault or a lost
word, so the order is read from the sources."""
import glob
import os
import re

import pytest

import speculative_decoding_verify_kv_gb300 as va

CSRC = os.path.join(os.path.dirname(va.__file__), "csrc")
REMOTE = r"map_shared_rank\(|team\.at\(|\bnote_error\(|\bread_error\(|\bshare_count\("
BARRIER = r"\bcluster\.sync\(\)|\bteam\.sync\(\)|\bcluster_met\(\)|\bjoin_chunks<"


def _bodies(text):
    """(name, body) of every kernel, and of the join that kernels end in."""
    text = re.sub(r"//[^\n]*", "", text)
    text = re.sub(r"__(?:launch_bounds|maxnreg)__\s*\((?:[^()]|\((?:[^()]|\([^()]*\))*\))*\)", "", text)
    for m in re.finditer(r"__global__\s+void\s+(\w+)\s*\([^{;]*\{|\bvoid\s+(join_chunks)\s*\([^{;]*\{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield m.group(1) or m.group(2), text[m.end():i]


def _kernels():
    found = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(path) as f:
            for name, body in _bodies(f.read()):
                if re.search(REMOTE, body):
                    found[name] = body
    return found


KERNELS = _kernels()


def test_the_kernels_of_clusters_are_found():
    assert {"accept_walk_kernel", "pages_fork_kernel", "pages_free_kernel", "pages_compact_kernel"} <= set(KERNELS)


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_the_cluster_meets_before_its_memory_is_shared(name):
    body = KERNELS[name]
    met, first = re.search(BARRIER, body), re.search(REMOTE, body)
    assert met and met.start() < first.start()
