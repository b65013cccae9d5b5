"""A 4-bit weight goes by the addresses of its tensors: one that has been given other memory is refused, and not read where it
was (CPU only)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
from bind_util import FakeWorkspace, library, stand_in
from comm_gemm_tile_gb300 import build as mkbuild
from test_layer_calls_cpu import t, w4


@pytest.mark.parametrize("name", ["codes", "scales", "zeros"])
def test_other_memory_is_refused(name, monkeypatch, tmp_path):
    mkbuild.build()
    lib = library(tmp_path, "static int n; int entry(void) { ++n; return 0; } int count(void) { return n; } unsigned long size(void) { return 0; }")
    stand_in(monkeypatch, lib.entry, lib.size)
    w = w4(zeros=t(40, 4))
    call = lambda: mk.w4_gemm(t(3, 256), w, out=t(3, 40), workspace=FakeWorkspace())   # noqa: E731
    call()
    tensor = getattr(w, name)
    was, tensor._ptr = tensor._ptr, 0x50000                # t.data = other
    with pytest.raises(ValueError, match="other memory"):
        call()
    assert lib.count() == 1
    tensor._ptr = was
    call()
    assert lib.count() == 2
    monkeypatch.undo()
    mk._bound = None


def test_the_tensors_are_the_weights():
    mkbuild.build()
    w = w4()
    assert w.zeros is None and w.codes.dtype == torch.uint8
    for name in ("codes", "scales", "zeros"):
        with pytest.raises(AttributeError):
            setattr(w, name, None)
