"""Refusals of the norm, router and 4-bit weight entry points, before anything touches a GPU (CPU only)."""
import ctypes

import pytest
import torch

import comm_gemm_tile_gb300 as mk
from bind_util import Fake, FakeWorkspace, library, stand_in
from comm_gemm_tile_gb300 import build as mkbuild

GOOD = 0x10000
NAN, INF = float("nan"), float("inf")
BF, HF, F32, I32 = torch.bfloat16, torch.float16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def L():
    mkbuild.build()
    return mk.lib()


def rows(p=GOOD, token=128, head=64):
    return mk._Rows(p, token, head)


def ref(r):
    return ctypes.byref(r) if r is not None else None


def test_struct_layouts():
    assert ctypes.sizeof(mk._Rows) == 24 and ctypes.sizeof(mk._W4) == 48 and mk._W4.group.offset == 40


def test_norm_refusals(L):
    def call(x=rows(), residual=None, weight=GOOD, y=rows(), h=None, scale=None, dtype=mk.MK_BF16, wdt=mk.MK_BF16,
             odt=mk.MK_BF16, tokens=4, heads=2, n=64, eps=1e-6):
        return L.mk_rms_norm(ref(x), ref(residual), weight, ref(y), ref(h), scale, dtype, wdt, odt, tokens, heads, n, eps, None)

    assert call(tokens=0) == mk.MK_OK == call(heads=0)
    e4 = dict(odt=mk.MK_E4M3)
    for bad in (dict(x=None), dict(y=None), dict(x=rows(None)), dict(x=rows(GOOD + 1)), dict(y=rows(GOOD + 1)),
                dict(residual=rows()), dict(h=rows()), dict(residual=rows(GOOD + 1), h=rows()),
                dict(residual=rows(), h=rows(None)), dict(residual=rows(), h=rows()), dict(residual=rows(), h=rows(2 * GOOD, token=0)), dict(y=rows(token=0)),
                dict(y=rows(head=0)), dict(weight=GOOD + 1), dict(weight=GOOD + 2, wdt=mk.MK_F32), dict(dtype=mk.MK_E4M3),
                dict(dtype=9), dict(wdt=mk.MK_F16), dict(odt=mk.MK_F32), dict(odt=9), e4, dict(e4, scale=GOOD + 2),
                dict(tokens=-1), dict(tokens=1 << 31), dict(tokens=1 << 20, heads=1 << 11), dict(heads=-1), dict(n=0),
                dict(n=16385), dict(eps=0.0), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF)):
        assert call(**bad) == mk.MK_ERR_INVALID, bad


def test_norm_gradient_refusals(L):
    size = L.mk_rms_norm_backward_workspace_size(4, 2, 64)
    assert size == 8 * 64 * 4 and L.mk_rms_norm_backward_workspace_size(1 << 20, 1, 64) == 456 * 64 * 4
    for args in ((-1, 1, 64), (4, -1, 64), (4, 1, 0), (4, 1, 16385), (1 << 31, 1, 64)):
        assert L.mk_rms_norm_backward_workspace_size(*args) == 0

    def call(dy=rows(), dh=None, h=rows(), weight=GOOD, dx=rows(), dw=GOOD, dtype=mk.MK_BF16, wdt=mk.MK_F32, tokens=4,
             heads=2, n=64, eps=1e-6, ws=GOOD, ws_bytes=size):
        return L.mk_rms_norm_backward(ref(dy), ref(dh), ref(h), weight, ref(dx), dw, dtype, wdt, tokens, heads, n, eps, ws,
                                      ws_bytes, None)

    assert call(tokens=0, dw=None) == mk.MK_OK
    for bad in (dict(dy=None), dict(h=None), dict(dx=None), dict(dy=rows(GOOD + 1)), dict(h=rows(None)), dict(dh=rows(None)),
                dict(dx=rows(token=0)), dict(dx=rows(head=0)), dict(weight=None), dict(weight=GOOD + 2), dict(dw=GOOD + 2),
                dict(dtype=mk.MK_E4M3), dict(wdt=mk.MK_F16), dict(n=0), dict(n=16385), dict(eps=0.0), dict(ws=None),
                dict(ws=GOOD + 4), dict(ws_bytes=size - 1), dict(tokens=-1)):
        assert call(**bad) == mk.MK_ERR_INVALID, bad


def test_route_refusals(L):
    size = L.mk_moe_route_workspace_size(1000, 64)
    assert size > 0
    for args in ((-1, 64), (1000, 0), (1000, 257), (1 << 31, 64)):
        assert L.mk_moe_route_workspace_size(*args) == 0
    good = dict(logits=GOOD, dtype=mk.MK_F32, T=1000, E=64, row=64, topk=2, normalize=1, scale=1.0, mask=None, idx=GOOD,
                gates=GOOD, counts=GOOD, tokens=GOOD, balance=GOOD, z=GOOD, ws=GOOD, ws_bytes=size)
    for bad in (dict(logits=None), dict(logits=GOOD + 2), dict(dtype=mk.MK_E4M3), dict(T=-1), dict(T=1 << 31), dict(E=0),
                dict(E=257), dict(topk=0), dict(topk=9), dict(E=4, topk=5), dict(scale=NAN), dict(scale=INF), dict(idx=None),
                dict(gates=None), dict(counts=None), dict(tokens=None), dict(balance=None), dict(z=None), dict(idx=GOOD + 2),
                dict(counts=GOOD + 1), dict(z=GOOD + 2), dict(ws=None), dict(ws=GOOD + 8), dict(ws_bytes=size - 1)):
        assert L.mk_moe_route(*{**good, **bad}.values(), None) == mk.MK_ERR_INVALID, bad
    good = dict(logits=GOOD, dtype=mk.MK_F32, T=10, E=64, row=64, topk=2, normalize=1, scale=1.0, idx=GOOD, counts=GOOD,
                tokens=GOOD, dgates=None, db=None, dz=None, dl=GOOD, dl_row=64)
    assert L.mk_moe_route_backward(*{**good, "T": 0}.values(), None) == mk.MK_OK
    for bad in (dict(logits=None), dict(dtype=mk.MK_E4M3), dict(T=-1), dict(E=257), dict(topk=9), dict(scale=NAN),
                dict(idx=None), dict(counts=None), dict(tokens=None), dict(dl=None), dict(dl=GOOD + 2), dict(dl_row=0),
                dict(dgates=GOOD + 1), dict(db=GOOD + 2), dict(dz=GOOD + 2), dict(tokens=GOOD + 2)):
        assert L.mk_moe_route_backward(*{**good, **bad}.values(), None) == mk.MK_ERR_INVALID, bad


def weight(**kw):
    a = dict(codes=GOOD, scales=GOOD, zeros=None, n=40, k=256, group=64, dtype=mk.MK_BF16)
    a.update(kw)
    return mk._W4(*a.values())


def test_w4_refusals(L):
    size = L.mk_w4_gemm_scratch_size(ref(weight()), 60000)
    assert size > 0 and L.mk_w4_gemm_scratch_size(ref(weight()), 32) == 0
    assert L.mk_w4_gemm_scratch_size(ref(weight(k=0)), 60000) == 0 == L.mk_w4_gemm_scratch_size(ref(weight()), -1)

    def call(x=GOOD, x_row=256, w=weight(), y=GOOD, y_row=40, dtype=mk.MK_BF16, odt=mk.MK_BF16, m=4, scratch=None,
             scratch_bytes=0, ws=None, ws_bytes=0, cfg=None):
        return L.mk_w4_gemm(x, x_row, ref(w), y, y_row, dtype, odt, m, scratch, scratch_bytes, ws, ws_bytes,
                            ref(cfg.c() if cfg else None), None)

    assert call(m=0) == mk.MK_OK == call(w=weight(n=0))
    for bad in (dict(x=None), dict(x=GOOD + 8), dict(x_row=260), dict(w=None), dict(y=None), dict(y=GOOD + 1), dict(y_row=39),
                dict(dtype=mk.MK_F32), dict(dtype=mk.MK_F16), dict(odt=mk.MK_F16), dict(odt=mk.MK_E4M3), dict(m=-1),
                dict(m=1 << 24), dict(odt=mk.MK_F32, y=GOOD + 2), dict(w=weight(codes=None)), dict(w=weight(scales=None)),
                dict(w=weight(codes=GOOD + 8)), dict(w=weight(scales=GOOD + 1)), dict(w=weight(zeros=GOOD + 1)),
                dict(w=weight(group=16)), dict(w=weight(group=256)), dict(w=weight(k=0)), dict(w=weight(k=288)),
                dict(w=weight(n=-1)), dict(w=weight(n=1 << 31)), dict(w=weight(dtype=mk.MK_F32)),
                dict(w=weight(n=(1 << 31) - 1, k=1 << 29)), dict(cfg=mk.Config(mode=1)), dict(cfg=mk.Config(operand=1)),
                dict(cfg=mk.Config(max_ctas=-1))):
        assert call(**bad) == mk.MK_ERR_INVALID, bad
    more = dict(m=60000, scratch=GOOD, scratch_bytes=size, ws=GOOD, ws_bytes=256)
    for bad in (dict(scratch=None), dict(scratch=GOOD + 64), dict(scratch_bytes=size - 1), dict(ws=None), dict(ws=GOOD + 8),
                dict(ws_bytes=255)):
        assert call(**{**more, **bad}) == mk.MK_ERR_INVALID, bad


# ------------------------------------------------------------------ the Python calls, on stand-ins for CUDA tensors

def t(*shape, dtype=BF, device=0, stride=None):
    return Fake(shape, dtype, device, stride=stride)


def route(device=0, T=10, K=2, E=64):
    made = {"topk_idx": t(T, K, dtype=I32, device=device), "gates": t(T, K, dtype=F32, device=device),
            "counts": t(E, dtype=I32, device=device)}
    made.update({name: t(dtype=I32 if name == "tokens" else F32, device=device) for name in ("tokens", "balance_loss", "z_loss")})
    return made


def w4(device=0, **kw):
    a = dict(codes=t(40, 128, dtype=torch.uint8, device=device), scales=t(40, 4, device=device), zeros=None)
    a.update(kw)
    return mk.W4Weight(**a)


def calls(device=0):
    d = dict(device=device)
    return [
        lambda: mk.rms_norm(t(4, 64, **d), t(64, **d), residual=t(4, 64, **d), out=t(4, 64, **d), h_out=t(4, 64, **d)),
        lambda: mk.rms_norm_backward(t(4, 64, **d), t(4, 64, **d), t(64, **d), weight_gradient=False, out=t(4, 64, **d)),
        lambda: mk.moe_route(t(10, 64, dtype=F32, **d), 2, out=route(device)),
        lambda: mk.moe_route_backward(t(10, 64, **d), route(device), out=t(10, 64, **d)),
        lambda: mk.w4_gemm(t(3, 256, **d), w4(device), out=t(3, 40, **d), workspace=FakeWorkspace(device)),
    ]


@pytest.fixture()
def launches(monkeypatch, tmp_path):
    mkbuild.build()
    lib = library(tmp_path, "#include <unistd.h>\nstatic int n, slow; int entry(void) { ++n; if (slow) usleep(300000); return 0; }"
                            "int count(void) { return n; } void wait(void) { slow = 1; } unsigned long size(void) { return 0; }")
    yield lambda current: stand_in(monkeypatch, lib.entry, lib.size, current), lib
    monkeypatch.undo()
    mk._bound = None


@pytest.mark.parametrize("which", range(5))
@pytest.mark.parametrize("device,current", [(1, 0), (0, 1), (0, 0), (2, 2)])
def test_only_the_current_device_is_launched_on(launches, which, device, current):
    use, lib = launches
    use(current)
    if device == current:
        calls(device)[which]()
    else:
        with pytest.raises(ValueError, match="device"):
            calls(device)[which]()
    assert lib.count() == (device == current)


@pytest.mark.parametrize("which", range(5))
def test_other_threads_run_during_a_call(launches, which):
    import threading
    import time
    use, lib = launches
    use(0)
    lib.wait()
    turns, stop = [], threading.Event()

    def work():
        while not stop.is_set():
            turns.append(time.perf_counter())
            time.sleep(0.01)

    other = threading.Thread(target=work)
    other.start()
    t0 = time.perf_counter()
    calls()[which]()
    t1 = time.perf_counter()
    stop.set()
    other.join()
    # of 30 turns; without the lock given up at most one at either end
    assert t1 - t0 >= 0.28 and sum(t0 + 0.05 < x < t1 - 0.05 for x in turns) >= 4


def test_python_refusals(launches):
    use, lib = launches
    use(0)
    x, r, w = t(4, 64), t(4, 64), t(64)
    y, h = t(4, 64), t(4, 64)
    f8 = mk.FP8
    mine = dict(out=y)
    bad = [
        lambda: mk.rms_norm(t(4, 2, 2, 64), w, **mine), lambda: mk.rms_norm(t(64), w, **mine), lambda: mk.rms_norm("x", w),
        lambda: mk.rms_norm(t(4, 0), None, out=t(4, 0)), lambda: mk.rms_norm(t(4, 64, dtype=torch.float64), None, **mine),
        lambda: mk.rms_norm(t(4, 64, stride=(1, 4)), w, **mine), lambda: mk.rms_norm(x, t(63), **mine),
        lambda: mk.rms_norm(x, t(64, dtype=HF), **mine), lambda: mk.rms_norm(x, t(64, device=1), **mine),
        lambda: mk.rms_norm(x, t(64, stride=(2,)), **mine), lambda: mk.rms_norm(x, w, residual=t(4, 65), h_out=h, **mine),
        lambda: mk.rms_norm(x, w, residual=t(4, 64, dtype=F32), h_out=h, **mine), lambda: mk.rms_norm(x, w, h_out=h, **mine),
        lambda: mk.rms_norm(x, w, scale_out=t(4, dtype=F32), **mine), lambda: mk.rms_norm(x, w, out_dtype=F32, **mine),
        lambda: mk.rms_norm(x, w, out_dtype=f8, scale_out=t(4, dtype=F32), **mine),
        lambda: mk.rms_norm(x, w, out_dtype=f8, out=t(4, 64, dtype=f8), scale_out=t(5, dtype=F32)),
        lambda: mk.rms_norm(x, w, out=t(5, 64)), lambda: mk.rms_norm(x, w, out=t(4, 64, dtype=HF)),
        lambda: mk.rms_norm(x, w, eps="a", **mine),
        lambda: mk.rms_norm_backward(x, t(5, 64), w, weight_gradient=False, out=y),
        lambda: mk.rms_norm_backward(t(4, 64, dtype=HF), x, w, weight_gradient=False, out=y),
        lambda: mk.rms_norm_backward(x, x, w, dh=t(4, 64, dtype=F32), weight_gradient=False, out=y),
        lambda: mk.rms_norm_backward(x, x, w, weight_gradient=False, out=t(4, 60)),
        lambda: mk.moe_route(t(10, 64, dtype=I32), 2, out=route()), lambda: mk.moe_route(t(10, 64), 0, out=route()),
        lambda: mk.moe_route(t(10, 64), 9, out=route(K=9)), lambda: mk.moe_route(t(10, 4), 5, out=route(K=5, E=4)),
        lambda: mk.moe_route(t(10, 64), 3, out=route()), lambda: mk.moe_route(t(10, 2, 64), 2, out=route()),
        lambda: mk.moe_route(t(10, 64), 2, mask=t(9, dtype=torch.bool), out=route()),
        lambda: mk.moe_route(t(10, 64), 2, mask=t(10, dtype=I32), out=route()),
        lambda: mk.moe_route(t(10, 64, stride=(1, 10)), 2, out=route()),
        lambda: mk.moe_route(t(10, 64), 2, out={**route(), "tokens": t(1, dtype=I32)}),
        lambda: mk.moe_route_backward(t(10, 64), route(T=9), out=t(10, 64)),
        lambda: mk.moe_route_backward(t(10, 64), route(E=63), out=t(10, 64)),
        lambda: mk.moe_route_backward(t(10, 64), route(), dgates=t(10, 3, dtype=F32), out=t(10, 64)),
        lambda: mk.moe_route_backward(t(10, 64), route(), dgates=t(10, 2), out=t(10, 64)),
        lambda: mk.moe_route_backward(t(10, 64), route(), dz=t(1, dtype=F32), out=t(10, 64)),
        lambda: mk.moe_route_backward(t(10, 64), route(), out=t(10, 64, dtype=F32)),
        lambda: w4(codes=t(40, 128, dtype=I32)), lambda: w4(codes=t(40, 128, dtype=torch.uint8, stride=(256, 1))),
        lambda: w4(scales=t(40, 4, dtype=F32)), lambda: w4(scales=t(39, 4)), lambda: w4(scales=t(40, 3)),
        lambda: w4(scales=t(40, 16)), lambda: w4(scales=t(40, 1)), lambda: w4(scales=t(40, 4, device=1)),
        lambda: w4(zeros=t(40, 4, dtype=HF)), lambda: w4(zeros=t(40, 3)), lambda: w4(scales=t(40, 4, stride=(1, 40))),
        lambda: mk.w4_gemm(t(3, 256), "w"), lambda: mk.w4_gemm(t(3, 256, dtype=HF), w4(), out=t(3, 40, dtype=HF)),
        lambda: mk.w4_gemm(t(3, 255), w4(), out=t(3, 40)), lambda: mk.w4_gemm(t(3, 256), w4(), out=t(3, 41)),
        lambda: mk.w4_gemm(t(3, 256), w4(), out_dtype=F32, out=t(3, 40)),
        lambda: mk.w4_gemm(t(3, 256), w4(), out_dtype=HF, out=t(3, 40, dtype=HF)),
        lambda: mk.w4_gemm(t(256), w4(), out=t(3, 40)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            call()
        assert lib.count() == 0, i
    for call in calls():
        call()
    assert lib.count() == 5


def test_packing_on_the_cpu():
    w = torch.randn(6, 256, generator=torch.Generator().manual_seed(1))
    for symmetric in (True, False):
        c, s, z = mk.W4Weight.pack(w, group=64, symmetric=symmetric, dtype=HF)
        code = torch.stack((c & 15, c >> 4), dim=-1).view(6, 4, 64).float()
        back = (code - (8.0 if z is None else z.float()[..., None])) * s.float()[..., None]
        assert (z is None) == symmetric and c.shape == (6, 128)
        assert bool(((back.flatten(1) - w).abs() <= s.float().repeat_interleave(64, dim=1) * 0.52).all())
    for kw in (dict(group=48), dict(group=256, dtype=HF), dict(dtype=F32)):
        with pytest.raises(ValueError):
            mk.W4Weight.pack(w, **kw)
