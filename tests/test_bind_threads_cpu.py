"""The sequence operators let other Python threads run while the library is in a call (CPU only): a launch into a full
queue waits there."""
import threading
import time

import pytest

import comm_gemm_tile_gb300 as mk
from bind_util import calls, library, stand_in
from comm_gemm_tile_gb300 import build as mkbuild


@pytest.mark.parametrize("which", range(3))
def test_other_threads_run_during_a_call(monkeypatch, tmp_path, which):
    mkbuild.build()
    L = library(tmp_path, "#include <unistd.h>\nint entry(void) { usleep(500000); return 0; }\n"
                          "unsigned long size(void) { return 256; }")
    stand_in(monkeypatch, L.entry, L.size)
    call = calls(0)[which][1]
    call()                               # whatever is set up once
    turns, stop = [], threading.Event()

    def work():
        while not stop.is_set():
            turns.append(time.perf_counter())
            time.sleep(0.01)

    other = threading.Thread(target=work)
    other.start()
    t0 = time.perf_counter()
    call()
    t1 = time.perf_counter()
    stop.set()
    other.join()
    monkeypatch.undo()
    mk._bound = None                     # the next call takes the real functions again
    # of 50 turns; without the lock given up at most one at either end
    assert t1 - t0 >= 0.45 and sum(t0 + 0.05 < t < t1 - 0.05 for t in turns) >= 5
