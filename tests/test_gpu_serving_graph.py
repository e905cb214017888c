"""The whole step of a served model captured into a graph: token ids -> embed_rows -> a projection with each request's
adapter in place -> the head -> log probabilities, once as two calls and once joined.  New ids, adapters and tokens are
copied into the captured buffers, and every replay, with eager work between, equals the eager step bit for bit.  What
each stage computes is tested in test_gpu_serving_path.py."""
import numpy as np
import pytest

import oracle
import bit_quantized_mat_quantize_amd as qmm
from bit_quantized_mat_quantize_amd.inputs import weights_t4_skewed
from gpu_helpers import to_dev, upload_weights
from test_gpu_lora import _pool
from test_gpu_logprobs import _pack

pytestmark = pytest.mark.gpu

ACT = {"q4_0": "q8_0", "q4_K": "q8_K", "q6_K": "q8_K"}


@pytest.mark.parametrize("table,proj,adapters", [("q6_K", "q4_K", "f16"), ("q4_K", "q4_0", "bf16")])
@pytest.mark.parametrize("M,V", [(1, 700), (6, 40000), (70, 700)])
def test_step_in_a_graph(M, V, table, proj, adapters):
    import torch
    D, R, E, k = 512, 8, 5, 6
    print(table, proj, adapters, M, V, flush=True)
    rng = np.random.default_rng(M + V)
    td = upload_weights(table, oracle.quantize(table, weights_t4_skewed([740, M], V, D)), V, D, "repacked")
    pd = upload_weights(proj, oracle.quantize(proj, weights_t4_skewed([741, M], D, D)), D, D, "repacked")
    A, B, _, _ = _pool(rng, E, R, D, D, adapters)
    scales = to_dev(rng.uniform(0.5, 2, E).astype(np.float32))
    mask = to_dev(_pack(rng.random((M, V)) < 0.5))
    sets = [(to_dev(rng.integers(0, V, M).astype(np.int32)), to_dev(rng.integers(-1, E, M).astype(np.int32)),
             to_dev(rng.integers(0, V, (M, 2)).astype(np.int32))) for _ in range(3)]

    def step(ids, adapter, tokens):
        h = qmm.embed_rows(table, td, ids, V, D, layout="repacked", scale=8.0)
        out, _ = qmm.quantize_mul_mat(proj, pd, h, D, layout="repacked")
        qmm.lora_add(out, h, A, B, adapter, scales=scales, out=out)
        y = qmm.quantize_row_q8(out, ACT[table])
        logits = qmm.mul_mat(table, td, y, M, V, D, layout="repacked")
        two = qmm.logprobs(logits, tokens=tokens, k=k, scale=1.25, mask=mask)
        one = qmm.mul_mat_logprobs(table, td, y, M, V, D, tokens=tokens, k=k, scale=1.25, mask=mask, layout="repacked",
                                   rows=M)
        return (out, *two, *one)

    eager = [[t.clone() for t in step(*s)] for s in sets]
    for a, b in zip(eager[0][1:5], eager[0][5:]):
        assert torch.equal(a, b)
    held = [t.clone() for t in sets[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*held)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step(*held)
    for rep in range(5):
        s = sets[rep % 3]
        for h, t in zip(held, s):
            h.copy_(t)
        for t in got:
            t.fill_(3)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, eager[rep % 3]):
            assert torch.equal(a, b), rep
        step(*s)
