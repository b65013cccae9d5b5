"""Refusals of the rotary, cache and paged attention entry points, before anything touches a GPU (CPU only)."""
import ctypes

import pytest
import torch

import comm_gemm_tile_gb300 as mk
from comm_gemm_tile_gb300 import build as mkbuild

GOOD = 0x10000
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    mkbuild.build()
    return mk.lib()


def rotation(**kw):
    a = dict(freqs=GOOD, positions=None, start=0, positions_64=0, rot=64, interleaved=0, inverse=0, magnitude=1.0)
    a.update(kw)
    return mk._Rotation(*a.values())


def cache(**kw):
    a = dict(k=GOOD, v=GOOD, k_scale=None, v_scale=None, page_stride=2 * 16 * 64, head_stride=16 * 64, slot_stride=64,
             n_pages=4, dtype=mk.MK_BF16, heads=2, d=64, page_size=16)
    a.update(kw)
    return mk._Cache(*a.values())


def seqs(**kw):
    a = dict(cu_q=GOOD, kv_len=GOOD, pages=GOOD, pages_stride=4, batch=2, max_pages=4)
    a.update(kw)
    return mk._Seqs(*a.values())


def test_struct_layouts():
    assert ctypes.sizeof(mk._Rotation) == 48 and mk._Rotation.magnitude.offset == 40
    assert ctypes.sizeof(mk._Seqs) == 40 and mk._Seqs.max_pages.offset == 36
    assert ctypes.sizeof(mk._Cache) == 80 and mk._Cache.page_size.offset == 76


def test_rope_refusals(L):
    def call(x=GOOD, y=GOOD, dtype=mk.MK_BF16, tokens=4, heads=2, d=64, strides=(128, 64, 128, 64), r=None):
        r = rotation() if r is None else r
        return L.mk_rope(x, y, dtype, tokens, heads, d, *strides, ctypes.byref(r) if r else None, None)

    assert call(tokens=0) == mk.MK_OK == call(heads=0)
    for bad in (dict(x=None), dict(y=None), dict(x=GOOD + 1), dict(dtype=mk.MK_E4M3), dict(dtype=7), dict(tokens=-1),
                dict(tokens=1 << 31), dict(heads=-1), dict(d=63), dict(d=0), dict(d=1024), dict(r=False),
                dict(r=rotation(rot=66)), dict(r=rotation(rot=7)), dict(r=rotation(rot=-2)), dict(r=rotation(freqs=None)),
                dict(r=rotation(freqs=GOOD + 4)), dict(r=rotation(positions=GOOD + 4, positions_64=1)),
                dict(r=rotation(magnitude=NAN)), dict(r=rotation(magnitude=INF))):
        assert call(**bad) == mk.MK_ERR_INVALID, bad


def _bad_caches():
    e4 = dict(dtype=mk.MK_E4M3, k_scale=GOOD, v_scale=GOOD)
    return [cache(k=None), cache(v=None), cache(k=GOOD + 8), cache(page_size=48), cache(page_size=4),
            cache(page_size=512), cache(page_size=0), cache(heads=0), cache(d=0), cache(dtype=mk.MK_F32),
            cache(slot_stride=65), cache(head_stride=-64), cache(n_pages=-1), cache(dtype=mk.MK_E4M3),
            cache(**{**e4, "k_scale": None}), cache(**{**e4, "v_scale": GOOD + 2}), cache(**{**e4, "slot_stride": 72})]


def _bad_seqs():
    return [seqs(cu_q=None), seqs(kv_len=None), seqs(pages=None), seqs(batch=-1), seqs(max_pages=-1),
            seqs(pages_stride=-1), seqs(cu_q=GOOD + 2), seqs(batch=1 << 25)]


def test_append_refusals(L):
    def call(c=None, k=GOOD, v=GOOD, dtype=mk.MK_BF16, tokens=4, q=None, q_out=None, heads_q=0, s=None, r=None, ws=GOOD,
             ws_bytes=256, k_strides=(128, 64)):
        c, s = c or cache(), s or seqs()
        return L.mk_kv_append(ctypes.byref(c), k, v, dtype, tokens, *k_strides, 128, 64, q, q_out, heads_q, 128, 64, 128,
                              64, ctypes.byref(s), ctypes.byref(r) if r else None, ws, ws_bytes, None)

    assert call(tokens=0) == mk.MK_OK == call(s=seqs(batch=0))
    for c in _bad_caches():
        assert call(c=c) == mk.MK_ERR_INVALID, [getattr(c, n) for n, _ in c._fields_]
    for s in _bad_seqs():
        assert call(s=s) == mk.MK_ERR_INVALID
    e4 = cache(dtype=mk.MK_E4M3, k_scale=GOOD, v_scale=GOOD)
    for bad in (dict(k=None), dict(v=None), dict(k=GOOD + 1), dict(dtype=mk.MK_F32), dict(dtype=mk.MK_F16),
                dict(tokens=-1), dict(q=GOOD), dict(q_out=GOOD), dict(q=GOOD, q_out=GOOD, heads_q=-1), dict(ws=None),
                dict(ws_bytes=255), dict(ws=GOOD + 8), dict(r=rotation(rot=128)), dict(r=rotation(inverse=1)),
                dict(c=e4, r=rotation(rot=24)), dict(c=e4, k_strides=(128, 60)), dict(c=e4, k=GOOD + 2)):
        assert call(**bad) == mk.MK_ERR_INVALID, bad


def test_attention_refusals(L):
    size = mk.paged_attention_workspace_size(4, 4, 2, 64, 2)
    assert size > 0 and size % 16 == 0
    for args in ((-1, 4, 2, 64, 2), (4, 3, 2, 64, 2), (4, 0, 2, 64, 2), (4, 4, 0, 64, 2), (4, 4, 2, 96, 2), (4, 4, 2, 64, -1)):
        assert mk.paged_attention_workspace_size(*args) == 0

    def call(q=GOOD, out=GOOD, lse=None, dtype=mk.MK_BF16, tokens=4, heads_q=4, strides=(256, 64, 256, 64), c=None, s=None,
             scale=0.125, causal=1, window=0, sinks=0, max_q=0, ws=GOOD, ws_bytes=1 << 30, cfg=None):
        c, s = c or cache(), s or seqs()
        return L.mk_paged_attention(q, out, lse, dtype, tokens, heads_q, *strides, ctypes.byref(c), ctypes.byref(s), scale,
                                    causal, window, sinks, max_q, ws, ws_bytes,
                                    ctypes.byref(cfg.c()) if cfg else None, None)

    assert call(tokens=0) == mk.MK_OK == call(s=seqs(batch=0))
    for c in _bad_caches():
        assert call(c=c) == mk.MK_ERR_INVALID, [getattr(c, n) for n, _ in c._fields_]
    for s in _bad_seqs():
        assert call(s=s) == mk.MK_ERR_INVALID
    for bad in (dict(q=None), dict(out=None), dict(q=GOOD + 8), dict(out=GOOD + 2), dict(lse=GOOD + 2),
                dict(dtype=mk.MK_F32), dict(dtype=mk.MK_F16), dict(tokens=-1), dict(tokens=1 << 31), dict(heads_q=3),
                dict(heads_q=0), dict(strides=(256, 60, 256, 64)), dict(strides=(256, 64, 250, 64)),
                dict(strides=(-256, 64, 256, 64)), dict(c=cache(d=96, slot_stride=96)), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(window=-1), dict(sinks=-1), dict(max_q=-1),
                dict(ws=None), dict(ws_bytes=size - 1), dict(ws=GOOD + 4), dict(cfg=mk.Config(operand=1)),
                dict(cfg=mk.Config(mode=1)),
                dict(c=cache(dtype=mk.MK_E4M3, k_scale=GOOD, v_scale=GOOD), dtype=mk.MK_F16)):
        assert call(**bad) == mk.MK_ERR_INVALID, bad


def test_frequencies_on_the_cpu():
    f, m = mk.rope_freqs(64, base=500.0, device="cpu")
    assert f.dtype == torch.float64 and f.shape == (32,) and float(f[0]) == 1.0 and m == 1.0
    assert mk.rope_freqs(0, device="cpu")[0].numel() == 0
    for kw in (dict(rot=3), dict(rot=64, scaling="?"), dict(rot=64, factor=0.5), dict(rot=64, base=0.0),
               dict(rot=2, scaling="ntk"), dict(rot=64, fast=1.0, slow=2.0)):
        with pytest.raises(ValueError):
            mk.rope_freqs(**kw, device="cpu")
