"""A cache goes by the addresses of its tensors: one of them with other memory is refused, and not read or written where it
was (CPU only)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
from bind_util import Fake, FakeWorkspace, library, stand_in
from comm_gemm_tile_gb300 import build as mkbuild

BF, I32, F32 = torch.bfloat16, torch.int32, torch.float32


@pytest.mark.parametrize("dtype,name", [(BF, "k"), (BF, "v"), (mk.FP8, "k"), (mk.FP8, "v"), (mk.FP8, "k_scale"), (mk.FP8, "v_scale")])
def test_other_memory_is_refused(dtype, name, monkeypatch, tmp_path):
    mkbuild.build()
    lib = library(tmp_path, "static int n; int entry(void) { ++n; return 0; } int count(void) { return n; } unsigned long size(void) { return 256; }")
    stand_in(monkeypatch, lib.entry, lib.size)
    scales = [Fake((8, 2), F32) for _ in range(2)] if dtype == mk.FP8 else []
    cache = mk.KVCache(Fake((8, 2, 16, 64), dtype), Fake((8, 2, 16, 64), dtype), *scales)
    seqs = Fake((3,), I32), Fake((2,), I32), Fake((2, 4), I32)
    row = Fake((4, 2, 64), BF)
    ws = dict(workspace=FakeWorkspace())
    calls = [lambda: mk.kv_append(cache, row, row, *seqs, **ws), lambda: mk.paged_attention(row, cache, *seqs, out=row, **ws)]
    for call in calls:
        call()
    tensor = getattr(cache, name)
    was, tensor._ptr = tensor._ptr, 0x50000                # t.data = other
    for call in calls:
        with pytest.raises(ValueError, match="other memory"):
            call()
    assert lib.count() == 2
    tensor._ptr = was
    for call in calls:
        call()
    assert lib.count() == 4
    monkeypatch.undo()
    mk._bound = None
