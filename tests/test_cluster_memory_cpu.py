"""Shared memory of another block of a cluster is touched only between two of the cluster's barriers: the block has started by
the first, and is there until the second (read in the sources: on the GPU the blocks start together as a rule, and a wrong
order shows nothing)."""
import os
import re

import pytest

from comm_gemm_tile_gb300 import build

TOUCHES = re.compile(r"\b(mapa_shared|st_shared_cluster_f32|mbar_arrive_cluster)\(")
WAITS = re.compile(r"\bcluster_(sync_all|wait)\(\)")
ARRIVES = re.compile(r"\bcluster_(sync_all|arrive)\(\)")


def kernels(text):
    """(name, body) of every kernel of a source."""
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)
    for m in re.finditer(r"__global__[^;{]*?\b(\w+)\(const __grid_constant__[^{;]*\{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        yield m.group(1), text[m.end():at]


def in_order(body):
    """Whether a body's touches stand behind a wait that has an arrival, and ahead of another arrival."""
    touches = [m.start() for m in TOUCHES.finditer(body)]
    if not touches:
        return True
    waits = [m.start() for m in WAITS.finditer(body) if m.start() < touches[0]]
    started = bool(waits) and any(m.start() <= waits[-1] for m in ARRIVES.finditer(body))
    return started and any(m.start() > touches[-1] for m in ARRIVES.finditer(body))


@pytest.mark.parametrize("source", [s for s in build.SOURCES])
def test_touches_stand_between_barriers(source):
    with open(os.path.join(build.CSRC, source)) as f:
        found = list(kernels(f.read()))
    for name, body in found:
        assert in_order(body), name
    if source == "mk_route.cu":
        assert any("cluster_sync_all()" in body for _, body in found)


def test_the_order_is_told():
    assert not in_order("st_shared_cluster_f32(a, v); cluster_sync_all();")
    assert not in_order("cluster_sync_all(); st_shared_cluster_f32(a, v);")
    assert not in_order("cluster_wait(); st_shared_cluster_f32(a, v); cluster_sync_all();")
    assert not in_order("cluster_arrive(); st_shared_cluster_f32(a, v); cluster_wait(); cluster_sync_all();")
    assert in_order("cluster_arrive(); x(); cluster_wait(); st_shared_cluster_f32(a, v); cluster_sync_all();")
    assert in_order("cluster_sync_all(); mapa_shared(a, 0); cluster_sync_all();")
