"""embed_rows, lora_add and logprobs beside autograd: they have no backward, so tensors that require a gradient are
refused where gradients are recorded, before anything else is looked at (no GPU is needed)."""
import pytest
import torch

import bit_quantized_mat_quantize_amd as qmm

IDS = torch.zeros(3, dtype=torch.int32)


def _lora(**kw):
    a = dict(base=torch.zeros(3, 96), x=torch.zeros(3, 64), A=torch.zeros(4, 8, 64), B=torch.zeros(4, 96, 8),
             scales=torch.zeros(4), out=torch.zeros(3, 96))
    a.update(kw)
    return qmm.lora_add(a["base"], a["x"], a["A"], a["B"], IDS, scales=a["scales"], out=a["out"])


@pytest.mark.parametrize("which,shape", [("base", (3, 96)), ("x", (3, 64)), ("A", (4, 8, 64)), ("B", (4, 96, 8)),
                                         ("scales", (4,)), ("out", (3, 96))])
def test_lora_add(which, shape):
    t = torch.zeros(shape, requires_grad=True)
    with pytest.raises(ValueError, match="no backward"):
        _lora(**{which: t})
    with pytest.raises(ValueError, match="no backward"):
        _lora(**{which: t * 2})                     # a result that autograd tracks
    with torch.no_grad(), pytest.raises(ValueError, match="GPU tensor"):   # the next check
        _lora(**{which: t})
    with pytest.raises(ValueError, match="GPU tensor"):
        _lora(**{which: t.detach()})


def test_logprobs_and_embed_rows():
    logits = torch.zeros(3, 1000, requires_grad=True)
    with pytest.raises(ValueError, match="no backward"):
        qmm.logprobs(logits)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU tensor"):
        qmm.logprobs(logits)
    w, out = torch.zeros(8 * 144, dtype=torch.uint8), torch.zeros(3, 256, requires_grad=True)
    with pytest.raises(ValueError, match="no backward"):
        qmm.embed_rows("q4_K", w, IDS, 8, 256, out=out)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU tensor"):
        qmm.embed_rows("q4_K", w, IDS, 8, 256, out=out)
