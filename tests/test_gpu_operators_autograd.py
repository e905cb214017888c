"""Outputs that the caller gives (in place among them) beside autograd: what a backward has saved of them cannot be
overwritten unnoticed."""
import pytest

import bit_quantized_mat_quantize_amd as qmm

pytestmark = pytest.mark.gpu


def _lora_out(out):
    import torch
    A, B = torch.ones(1, 4, 32, device="cuda"), torch.ones(1, out.shape[1], 4, device="cuda")
    x, ids = torch.ones(out.shape[0], 32, device="cuda"), torch.zeros(out.shape[0], dtype=torch.int32, device="cuda")
    return qmm.lora_add(out, x, A, B, ids, out=out)


def _embed_out(out):
    import torch
    w = torch.zeros(4 * out.shape[1] // 32 * 18, dtype=torch.uint8, device="cuda")
    ids = torch.zeros(out.shape[0], dtype=torch.int32, device="cuda")
    return qmm.embed_rows("q4_0", w, ids, 4, out.shape[1], out=out)


@pytest.mark.parametrize("call", [_lora_out, _embed_out])
def test_a_saved_tensor_that_is_overwritten_is_noticed(call):
    import torch
    out = torch.ones(3, 64, device="cuda")
    w = torch.ones(3, 64, device="cuda", requires_grad=True)
    y = (out * w).sum()                            # w's gradient is out, which is saved
    before = out._version
    call(out)
    assert out._version > before
    with pytest.raises(RuntimeError, match="inplace operation"):
        y.backward()
    out = torch.ones(3, 64, device="cuda")
    y = (out * w).sum()
    call(out.clone())                              # another tensor: nothing is noticed, and the gradient is out
    y.backward()
    assert torch.equal(w.grad, out)


@pytest.mark.parametrize("call", [_lora_out, _embed_out])
def test_inference_mode(call):
    import torch
    with torch.inference_mode():
        out = torch.ones(3, 64, device="cuda")
        got = call(out)
        assert got.data_ptr() == out.data_ptr()
    call(out)
    assert float(out[0, 0]) in (0.0, 257.0)        # twice 4 ranks of 32 ones on 1, or rows of zeros
