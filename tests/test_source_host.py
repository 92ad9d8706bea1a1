"""Rules that every kernel's source keeps, checked on its text: what breaks them
shows on a GPU once in a long while, or as a fault."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "top_routed_grouped_gb300", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")))


def source(path):
    """The text without comments."""
    text = open(path).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def kernels(path):
    """(name, parameters, body) of each __global__ function."""
    text = source(path)
    for m in re.finditer(r"__global__[^;{]*?\bvoid\b[^;{]*?(\w+)\s*\(([^{;]*)\)\s*\{", text, flags=re.S):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        head = text[m.start():m.end()]
        yield re.findall(r"(\w+)\s*\((?!\d|[A-Z_]+\s*[,)]|CtCfg)", head)[-1], head, text[m.end():i]


def test_kernels_are_found():
    names = {n for f in FILES for n, _, _ in kernels(f)}
    assert {"grad_norm_kernel", "ce_pair_kernel", "combine_kernel", "permute_cluster_kernel"} <= names, sorted(names)


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_clusters_meet_before_remote_stores(path):
    """A CTA's shared memory is there to be written by others once all CTAs of the cluster run."""
    for name, _, body in kernels(path):
        store = body.find("st.shared::cluster")
        if store >= 0:
            meet = [body.find(s) for s in ("cluster_sync()", "cluster_meet_wait()") if s in body[:store]]
            assert meet, f"{name}: a remote store before the cluster is known to run"


@pytest.mark.parametrize("path", FILES, ids=os.path.basename)
def test_no_load_may_pass_the_wait_for_the_kernel_before(path):
    """Kernels start while the one before them runs.  A load through the read-only
    path, or one that the compiler takes for a pure function of its address, may be
    moved above the wait and read what is not written yet."""
    found = re.findall(r"__ld(?:g|cs|cg|ca|lu|cv)\b|\bld\.global\.(?:\w+\.)*nc\b|__restrict__|\b__constant__", source(path))
    assert not found, found
    for m in re.finditer(r"asm\s+(volatile)?[^;]*?\bld\.global\b", source(path)):
        assert m.group(1), "a load that is not volatile"
