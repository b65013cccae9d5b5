"""The memory order of the output that rope makes, with and without a stream of its own (GPU)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


@pytest.mark.parametrize("stream", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_the_output_has_the_order_of_the_input(stream, inverse):
    """A [heads x s x d] tensor passed as its transpose comes back as one: the transpose of the result is contiguous,
    as ring_attention reads it."""
    x = torch.randn(3, 40, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    freqs, _ = mk.rope_freqs(64)
    want = mk.rope(x.transpose(0, 1).contiguous(), freqs, inverse=inverse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mk.rope(x.transpose(0, 1), freqs, inverse=inverse, stream=side if stream else None)
    torch.cuda.synchronize()
    assert got.stride() == x.transpose(0, 1).stride() and got.transpose(0, 1).is_contiguous()
    assert torch.equal(got, want)


@pytest.mark.parametrize("stream", [False, True])
def test_a_padded_input_gives_a_dense_output_in_its_order(stream):
    x = torch.randn(3, 40, 96, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()[..., :64].transpose(0, 1)
    freqs, _ = mk.rope_freqs(64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mk.rope(x, freqs, stream=side.cuda_stream if stream else None)
    torch.cuda.synchronize()
    assert got.transpose(0, 1).is_contiguous()
    assert torch.equal(got, mk.rope(x.contiguous(), freqs))
