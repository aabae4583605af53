"""Kernels that reach into the shared memory of other CTAs of their cluster wait at a cluster
barrier first: before it a CTA of the cluster may not have started, and an access to its shared
memory is undefined.  Read from the sources, since a run that goes well shows nothing."""
from __future__ import annotations

import glob
import os
import re

import pytest

from bit_asymmetric_kv_gb300 import build as kbuild

REMOTE = re.compile(r"map_shared_rank\b|\bmapa\.")  # how an address in another CTA is made
BARRIER = re.compile(r"\.sync\(\)|\bbarrier_wait\(\)|barrier\.cluster\.wait|\bcluster\.sync\(\)")
HEAD = re.compile(r"(__global__|__device__)[^;{}]*?\b(\w+)\s*\([^;{}]*\)\s*(?:const\s*)?\{")


def functions(text):
    """{name: (is a kernel, body)} of the device functions of a source, without comments."""
    text = re.sub(r"/\*.*?\*/", " ", re.sub(r"//[^\n]*", "", text), flags=re.S)
    out = {}
    for m in HEAD.finditer(text):
        head = text[m.start():m.end()]
        names = [n for n in re.findall(r"(\w+)\s*\(", head) if n not in ("__launch_bounds__", "__cluster_dims__", "__align__")]
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        out[names[0]] = (m.group(1) == "__global__", text[m.end():i])
    return out


def events(funcs, name, seen=()):
    """Cluster barriers (B) and accesses to other CTAs' shared memory (R), in the order of the text, calls
    followed."""
    body = funcs[name][1]
    found = [(m.start(), "R") for m in REMOTE.finditer(body)] + [(m.start(), "B") for m in BARRIER.finditer(body)]
    for m in re.finditer(r"\b(\w+)\s*(?:<[^;{}()]*>)?\s*\(", body):
        f = m.group(1)
        if f in funcs and f != name and f not in seen:
            found.append((m.start(), events(funcs, f, seen + (name,))))
    return "".join(e for _, e in sorted(found))


def kernels():
    out = []
    for path in sorted(glob.glob(os.path.join(kbuild.CSRC, "*.cu"))):
        with open(path) as f:
            funcs = functions(f.read())
        for name, (kernel, _) in funcs.items():
            if kernel and "R" in events(funcs, name):
                out.append((os.path.basename(path), name, events(funcs, name)))
    return out


KERNELS = kernels()


def test_the_kernels_are_found():
    assert {k for _, k, _ in KERNELS} >= {"pool_reserve_kernel", "pool_reorder_kernel", "pool_compact_kernel",
                                          "decode_cluster_kernel"}


@pytest.mark.parametrize("source,name,order", KERNELS, ids=[k for _, k, _ in KERNELS])
def test_a_cluster_barrier_comes_first(source, name, order):
    assert order.startswith("B"), (source, name, order)
