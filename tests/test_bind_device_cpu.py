"""The sequence operators launch on the current device: tensors of another one are refused before any launch (CPU only)."""
import pytest

import comm_gemm_tile_gb300 as mk
from bind_util import calls, library, stand_in
from comm_gemm_tile_gb300 import build as mkbuild


@pytest.fixture()
def launches(monkeypatch, tmp_path):
    """A library whose calls are counted; tensors and current device are given by the test."""
    mkbuild.build()
    L = library(tmp_path, "static int n; int entry(void) { ++n; return 0; } int count(void) { return n; }"
                          "unsigned long size(void) { return 256; }")
    yield lambda current: stand_in(monkeypatch, L.entry, L.size, current), L.count
    monkeypatch.undo()
    mk._bound = None                    # the next call takes the real functions again


@pytest.mark.parametrize("which", range(3))
@pytest.mark.parametrize("device,current", [(1, 0), (0, 1), (3, 2)])
def test_tensors_of_another_device_are_refused(launches, which, device, current):
    use, count = launches
    use(current)
    with pytest.raises(ValueError, match="device"):
        calls(device)[which][1]()
    assert count() == 0


@pytest.mark.parametrize("which", range(3))
@pytest.mark.parametrize("device", [0, 2])
def test_tensors_of_the_current_device_are_launched(launches, which, device):
    use, count = launches
    use(device)
    calls(device)[which][1]()
    assert count() == 1
