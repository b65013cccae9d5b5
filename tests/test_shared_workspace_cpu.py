"""Where moe_route and rms_norm_backward take scratch in a Workspace that others use as well (CPU only)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
from bind_util import Fake, library, stand_in
from comm_gemm_tile_gb300 import build as mkbuild
from test_layer_calls_cpu import route, t

F32, U8 = torch.float32, torch.uint8
SOURCE = """
static void *seen; static unsigned long bytes;
int route(void *l, int dt, long long T, int E, long long row, int k, int norm, float s, void *m, void *i, void *g, void *c, void *n,
          void *b, void *z, void *ws, unsigned long size, void *st) { seen = ws; bytes = size; return 0; }
int grad(void *dy, void *dh, void *h, void *w, void *dx, void *dw, int dt, int wdt, long long T, int H, int n, float eps, void *ws,
         unsigned long size, void *st) { seen = ws; bytes = size; return 0; }
unsigned long size(void) { return 4096; }
void *where(void) { return seen; }
unsigned long room(void) { return bytes; }
"""


class Shared:
    """A workspace with a header and flags at 0x20000 that must stay, and scratch at 0x900000."""

    def get(self, nbytes, stream=None):
        return Fake((nbytes,), U8, ptr=0x20000)

    def scratch(self, nbytes, stream=None):
        return Fake((nbytes,), U8, ptr=0x900000)


class Plain:
    def get(self, nbytes, stream=None):
        return Fake((nbytes,), U8, ptr=0x20000)


@pytest.mark.parametrize("which", ["route", "grad"])
def test_partial_sums_are_not_where_flags_are(which, monkeypatch, tmp_path):
    import ctypes
    mkbuild.build()
    lib = library(tmp_path, SOURCE)
    lib.where.restype = ctypes.c_void_p
    lib.room.restype = ctypes.c_ulong
    stand_in(monkeypatch, getattr(lib, which), lib.size)
    for ws, at in ((Shared(), 0x900000), (Plain(), 0x20000)):
        if which == "route":
            mk.moe_route(t(100, 64, dtype=F32), 2, out=route(T=100), workspace=ws)
        else:
            monkeypatch.setattr(torch, "empty", lambda *a, **k: t(64))
            monkeypatch.setattr(mk, "_bound", None)
            mk.rms_norm_backward(t(4, 64), t(4, 64), t(64), out=t(4, 64), workspace=ws)
        assert lib.where() == at and lib.room() == 4096
    monkeypatch.undo()
    mk._bound = None


def test_scratch_is_apart(monkeypatch):
    made = []
    monkeypatch.setattr(mk.Workspace, "get", lambda self, n, stream=None: made.append((self, n, stream)) or self)
    ws = mk.Workspace("cuda:0")
    assert ws.scratch(100, "s") is not ws and ws.scratch(200) is ws.apart and ws.get(5) is ws
    assert made == [(ws.apart, 100, "s"), (ws.apart, 200, None), (ws, 5, None)]
