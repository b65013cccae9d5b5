"""8-bit caches where nearly all the weight lies on pages of zeros and a page of large values has nearly none (GPU).

A page of zeros has the smallest scale, 2^-100.  Against it, a key whose score is 2^7 to 2^8 lower in units of log2 has a
weight of 2^-128 to 2^-136 and values that are larger by up to 2^140: the product is of ordinary size, the factors are not.
Weights below the smallest normal fp32 number (2^-126) may count as nothing, and factors may stop at the largest one (2^128): with
weights taken 2^10 high that is at most 2^-118 times the largest value, besides the ordinary bounds."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
import paged_util as P

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("gap", [100.0, 126.0, 130.0, 134.0, 150.0])
@pytest.mark.parametrize("d,page,group", [(128, 16, 4), (64, 64, 3), (128, 32, 16)])
@pytest.mark.parametrize("n", [1, 40])
def test_zeros_outweigh_large_values(n, d, page, group, gap):
    batch = P.Batch([(n, 300), (n, 200)], page, seed=75)
    k, v, ks, vs = P.random_cache(batch.n_pages, 1, page, d, P.E4M3, 76)
    ks.fill_(1.0)
    k.zero_()
    q = torch.zeros(batch.tokens, group, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    for table in batch.table:
        zero, large = table[1], table[2]
        k[zero, 0, :, 0] = 0.0
        v[zero] = 0.0
        vs[zero] = 2.0 ** -100
        for other in table:
            if other != zero:
                k[other, 0, :, 0] = -16.0
                vs[other] = 2.0 ** -100
        vs[large] = 2.0 ** 40
    ks *= gap / 16.0
    P.poison(k, ks, batch)
    P.poison(v, vs, batch)
    scale = 0.6931471805599453                       # scores are whole numbers of log2
    out = mk.paged_attention(q, mk.KVCache(k, v, ks, vs), batch.cu_q, batch.kv_len, batch.pages, scale=scale, causal=False)
    want, _, tol, _ = P.attention(q, k, v, ks, vs, batch, scale=scale, causal=False)
    assert mk.device_status()[0] == mk.MK_OK
    assert bool(torch.isfinite(out).all())
    most = 448.0 * 2.0 ** 40 * 300
    assert float(((out.double().cpu() - want).abs() - tol).max()) <= 2.0 ** -118 * most


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("n", [1, 40])
def test_a_scale_that_is_not_finite_reaches_the_rows_that_see_it(n, bad):
    batch = P.Batch([(n, 300), (n, 200)], 16, seed=77)
    k, v, ks, vs = P.random_cache(batch.n_pages, 1, 16, 64, P.E4M3, 78)
    v.copy_((v.float() + 500).clamp(max=448).to(v.dtype))       # no zeros: infinity times 0 is NaN
    vs[batch.table[0][1]] = bad
    P.poison(k, ks, batch)
    P.poison(v, vs, batch)
    q = torch.randn(batch.tokens, 4, 64, generator=torch.Generator().manual_seed(79)).bfloat16().cuda()
    out = mk.paged_attention(q, mk.KVCache(k, v, ks, vs), batch.cu_q, batch.kv_len, batch.pages)
    assert mk.device_status()[0] == mk.MK_OK
    assert not bool(torch.isfinite(out[:n]).any()) and bool(torch.isfinite(out[n:]).all())
