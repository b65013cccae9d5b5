"""4-bit forms of matrices without rows, of one row, and of rows that do not lie one after another (CPU only)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk


@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("n", [0, 1, 5])
def test_packing(n, symmetric):
    w = torch.randn(n, 128, generator=torch.Generator().manual_seed(1))
    c, s, z = mk.W4Weight.pack(w, group=32, symmetric=symmetric)
    assert c.shape == (n, 64) and s.shape == (n, 4) and (z is None or z.shape == (n, 4))
    wide = torch.zeros(n, 200)
    wide[:, 9:137] = w
    for other in (wide[:, 9:137], w.t().contiguous().t()):
        again = mk.W4Weight.pack(other, group=32, symmetric=symmetric)
        assert all(a is None or torch.equal(a, b) for a, b in zip(again, (c, s, z)))
    held = mk.W4Weight.__new__(mk.W4Weight)                 # (a weight itself is on a GPU)
    held._tensors = c, s, z
    back = held.dequantize(torch.float32)
    assert back.shape == (n, 128)
    step = s.float().repeat_interleave(32, dim=1)
    assert bool(((back - w).abs() <= step * 0.6).all())
