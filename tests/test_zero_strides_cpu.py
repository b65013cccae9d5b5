"""Strides of 0 (expanded tensors): refused where several rows would share memory that is written or that a tensor map
describes, before anything touches a GPU (CPU only)."""
import ctypes

import pytest

import comm_gemm_tile_gb300 as mk
from test_paged_cpu import GOOD, L, cache, rotation, seqs  # noqa: F401


def _attention(L, c=None, tokens=4, heads_q=4, strides=(256, 64, 256, 64)):  # noqa: F811
    c = c or cache()
    return L.mk_paged_attention(GOOD, GOOD, None, mk.MK_BF16, tokens, heads_q, *strides, ctypes.byref(c),
                                ctypes.byref(seqs()), 0.125, 1, 0, 0, 0, GOOD, 1 << 30, None, None)


def _append(L, c=None, qo=(128, 64), tokens=4, heads_q=2):  # noqa: F811
    c = c or cache()
    r = rotation()
    return L.mk_kv_append(ctypes.byref(c), GOOD, GOOD, mk.MK_BF16, tokens, 128, 64, 128, 64, GOOD, GOOD, heads_q, 128, 64,
                          *qo, ctypes.byref(seqs()), ctypes.byref(r), GOOD, 256, None)


@pytest.mark.parametrize("which", ["page_stride", "head_stride", "slot_stride"])
@pytest.mark.parametrize("dtype", [mk.MK_BF16, mk.MK_E4M3])
def test_caches_of_expanded_pages_heads_or_slots(L, which, dtype):  # noqa: F811
    scales = dict(dtype=dtype, k_scale=GOOD, v_scale=GOOD) if dtype == mk.MK_E4M3 else {}
    bad = cache(**{which: 0}, **scales)
    assert _attention(L, bad) == mk.MK_ERR_INVALID
    assert _append(L, bad) == mk.MK_ERR_INVALID


def test_one_page_or_head_has_no_stride_to_speak_of(L):  # noqa: F811
    for c in (cache(page_stride=0, n_pages=1), cache(head_stride=0, heads=1), cache(page_stride=0, n_pages=0)):
        assert _attention(L, c, tokens=0) == mk.MK_OK
        assert _append(L, c, tokens=0) == mk.MK_OK


@pytest.mark.parametrize("strides", [(256, 64, 0, 64), (256, 64, 256, 0)])
def test_expanded_outputs_of_attention(L, strides):  # noqa: F811
    assert _attention(L, strides=strides) == mk.MK_ERR_INVALID


@pytest.mark.parametrize("qo", [(0, 64), (128, 0)])
def test_expanded_rotated_queries(L, qo):  # noqa: F811
    assert _append(L, qo=qo) == mk.MK_ERR_INVALID


@pytest.mark.parametrize("strides", [(0, 64), (128, 0)])
def test_expanded_outputs_of_rope(L, strides):  # noqa: F811
    r = rotation()
    assert L.mk_rope(GOOD, GOOD, mk.MK_BF16, 4, 2, 64, 128, 64, *strides, ctypes.byref(r), None) == mk.MK_ERR_INVALID
