"""A tensor that a call was given to write to and that autograd has saved before: backward refuses to use it (GPU)."""
import pytest
import torch

import comm_gemm_tile_gb300 as mk
from test_paged_gpu import _problem

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from comm_gemm_tile_gb300 import build
    build.build()
    torch.cuda.init()


def ones(*shape, dtype=BF):
    return torch.ones(shape, dtype=dtype, device="cuda")


def calls():
    """name -> (the given output, the call that writes to it)."""
    x, w, logits = ones(6, 64), ones(64), torch.randn(6, 16, device="cuda")
    route = mk.moe_route(logits, 2)
    batch, q, cache = _problem([(1, 20), (1, 9)], 2, 2, 64, 16, BF, BF)
    seqs = batch.cu_q, batch.kv_len, batch.pages
    k = ones(batch.tokens, 2, 64)
    freqs, _ = mk.rope_freqs(64)
    four = mk.W4Weight.quantize(torch.randn(32, 64, device="cuda"), group=32)
    E4 = mk.FP8
    y, s, h, y8 = ones(6, 64), ones(6, dtype=F32), ones(6, 64), torch.empty(6, 64, dtype=E4, device="cuda")
    dl, yw, qo, ao, ro = torch.empty_like(logits), ones(6, 32), torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    return {
        "rms_norm out": (y, lambda: mk.rms_norm(x, w, out=y)),
        "rms_norm h_out": (h, lambda: mk.rms_norm(x, w, residual=x, h_out=h)),
        "rms_norm in place": (x, lambda: mk.rms_norm(y, None, residual=x, h_out=x)),
        "rms_norm scale_out": (s, lambda: mk.rms_norm(x, w, out_dtype=E4, out=y8, scale_out=s)),
        "rms_norm_backward": (y, lambda: mk.rms_norm_backward(x, h, w, out=y)),
        "moe_route gates": (route["gates"], lambda: mk.moe_route(logits, 2, out=route)),
        "moe_route z_loss": (route["z_loss"], lambda: mk.moe_route(logits, 2, out={"z_loss": route["z_loss"]})),
        "moe_route_backward": (dl, lambda: mk.moe_route_backward(logits, route, out=dl)),
        "w4_gemm": (yw, lambda: mk.w4_gemm(x, four, out=yw)),
        "rope": (ro, lambda: mk.rope(q, freqs, out=ro)),
        "kv_append": (qo, lambda: mk.kv_append(cache, k, k, *seqs, q=q, freqs=freqs, q_out=qo)),
        "paged_attention": (ao, lambda: mk.paged_attention(q, cache, *seqs, out=ao)),
    }


NAMES = ("rms_norm out", "rms_norm h_out", "rms_norm in place", "rms_norm scale_out", "rms_norm_backward", "moe_route gates",
         "moe_route z_loss", "moe_route_backward", "w4_gemm", "rope", "kv_append", "paged_attention")


@pytest.mark.parametrize("name", NAMES)
def test_a_saved_tensor_that_was_written_is_not_used(name):
    saved, call = calls()[name]
    leaf = torch.ones_like(saved).requires_grad_()
    product = leaf * saved                      # (its gradient is saved * what comes back)
    (leaf * saved).sum().backward()             # nothing was written yet
    before = saved._version
    call()
    assert saved._version > before
    with pytest.raises(RuntimeError, match="inplace"):
        product.sum().backward()


def test_the_stream_of_a_norm_with_a_gradient():
    """The norm's own gradient reads the stream that a later call updates in place."""
    stream, w = ones(6, 64), ones(64, dtype=F32).requires_grad_()
    y = mk.rms_norm(stream, w)
    with torch.no_grad():
        mk.rms_norm(ones(6, 64), None, residual=stream, h_out=stream)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


def test_inference_tensors_and_outputs_of_the_call():
    with torch.inference_mode():
        x = ones(6, 64)
        assert mk.rms_norm(x, None, out=x) is x
    x, w = ones(6, 64), ones(64, dtype=F32).requires_grad_()
    mk.rms_norm(x, w).sum().backward()          # no output was given: nothing is marked
    assert x._version == 0 and w.grad is not None
