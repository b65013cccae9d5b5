"""Stand-ins for CUDA tensors and library calls: what the marshalling module reads, without a GPU."""
import ctypes
import subprocess

import torch

import comm_gemm_tile_gb300 as mk


class Fake:
    """What the marshalling module asks of a tensor."""

    def __init__(self, shape, dtype, device=0, ptr=0x10000, stride=None):
        self.shape, self.dtype, self._device, self._ptr = tuple(shape), dtype, device, ptr
        self.device = torch.device("cuda", device)
        if stride is None:
            stride, n = [], 1
            for s in reversed(self.shape):
                stride.insert(0, n)
                n *= max(s, 1)
        self._stride = tuple(stride)

    def data_ptr(self):
        return self._ptr

    def get_device(self):
        return self._device

    def stride(self):
        return self._stride

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n


class FakeWorkspace:
    def __init__(self, device=0):
        self.buf = Fake((1 << 20,), torch.uint8, device)

    def get(self, nbytes, stream=None):
        return self.buf


def library(tmp_path, source):
    """A small C library built from source."""
    path = tmp_path / "stand_in.so"
    (tmp_path / "stand_in.c").write_text(source)
    subprocess.run(["cc", "-O1", "-shared", "-fPIC", str(tmp_path / "stand_in.c"), "-o", str(path)], check=True)
    return ctypes.CDLL(str(path))


def calls(device=0):
    """(name, call) of rope, kv_append and paged_attention on stand-ins of one device."""
    i32 = lambda *shape: Fake(shape, torch.int32, device)   # noqa: E731
    bf = lambda *shape: Fake(shape, torch.bfloat16, device)   # noqa: E731
    seqs = (i32(3), i32(2), i32(2, 4))
    freqs = Fake((32,), torch.float64, device)

    def cache():
        return mk.KVCache(bf(8, 2, 16, 64), bf(8, 2, 16, 64))

    return [
        ("mk_rope", lambda: mk.rope(bf(4, 2, 64), freqs, out=bf(4, 2, 64))),
        ("mk_kv_append", lambda: mk.kv_append(cache(), bf(4, 2, 64), bf(4, 2, 64), *seqs, q=bf(4, 4, 64), freqs=freqs,
                                              q_out=bf(4, 4, 64), workspace=FakeWorkspace(device))),
        ("mk_paged_attention", lambda: mk.paged_attention(bf(4, 4, 64), cache(), *seqs, out=bf(4, 4, 64),
                                                          workspace=FakeWorkspace(device))),
    ]


def stand_in(monkeypatch, entry, size=None, current=0):
    """Calls go to the C functions `entry` (and `size` for workspace sizes); the current device is `current`."""
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value   # noqa: E731
    monkeypatch.setattr(mk, "_address", lambda name: address(size if name.endswith("_size") else entry))
    monkeypatch.setattr(mk, "_bound", None)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current)
