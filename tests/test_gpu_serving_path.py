"""The operators beside the projections together with them, as a served model uses them: token ids -> rows of the
packed table -> a projection with each request's adapter -> the head (the same table) -> log probabilities.

Every stage is compared with its formula in 64 bits on what the stage before it gave, so that each keeps its own
tolerance: embed_rows two roundings, the products 1e-4 of sum|terms| (the library's), lora_add and logprobs as
derived in their own tests.  The chunked head equals the two calls bit for bit where its parts take the same
kernel."""
import numpy as np
import pytest

import oracle
import bit_quantized_mat_quantize_amd as qmm
from bit_quantized_mat_quantize_amd.inputs import weights_t4_skewed
from gpu_helpers import assert_close, full_reference, to_dev, to_host, upload_weights
from test_gpu_logprobs import Reference, _pack
from test_gpu_lora import _check as check_lora
from test_gpu_lora import _formula, _pool

pytestmark = pytest.mark.gpu

ACT = {"q4_0": "q8_0", "q4_K": "q8_K", "q6_K": "q8_K", "q2_K": "q8_K"}


@pytest.mark.parametrize("table,proj", [("q6_K", "q4_K"), ("q4_0", "q2_K"), ("q4_K", "q4_0")])
@pytest.mark.parametrize("M", [1, 6, 70])
def test_token_to_alternatives(M, table, proj):
    V, D, R, E, k = 700, 512, 8, 5, 6
    print(table, proj, M, flush=True)
    rng = np.random.default_rng(M)
    tw = oracle.quantize(table, weights_t4_skewed([720, M], V, D))
    pw = oracle.quantize(proj, weights_t4_skewed([721, M], D, D))
    td, pd = upload_weights(table, tw, V, D, "repacked"), upload_weights(proj, pw, D, D, "repacked")
    ids = rng.integers(0, V, M).astype(np.int32)
    A, B, A64, B64 = _pool(rng, E, R, D, D, "bf16")
    adapter = rng.integers(-1, E, M).astype(np.int32)
    scales = rng.uniform(0.5, 2, E).astype(np.float32)

    h = qmm.embed_rows(table, td, to_dev(ids), V, D, layout="repacked", scale=8.0)
    want = oracle.dequantize(table, tw, V, D)[ids] * 8.0
    h64 = to_host(h).astype(np.float64)
    assert (np.abs(h64 - want) <= 2 * 2.0 ** -24 * (1 + 1e-6) * np.abs(want)).all()

    out, y = qmm.quantize_mul_mat(proj, pd, h, D, layout="repacked")
    y_host = to_host(y).reshape(M, -1)
    assert np.array_equal(y_host, oracle.quantize(ACT[proj], to_host(h)))
    assert_close(to_host(out), *full_reference(proj, pw, y_host, M, D, D), f"{proj} projection")

    before = to_host(out).copy()
    got = qmm.lora_add(out, h, A, B, to_dev(adapter), scales=to_dev(scales), out=out)   # in place on the projection
    check_lora(to_host(got), *_formula(before, to_host(h), A64, B64, adapter, scales))

    yh = qmm.quantize_row_q8(out, ACT[table])
    logits = qmm.mul_mat(table, td, yh, M, V, D, layout="repacked")
    assert_close(to_host(logits), *full_reference(table, tw, to_host(yh).reshape(M, -1), M, V, D), "head")

    tokens = rng.integers(0, V, (M, 2)).astype(np.int32)
    allowed = rng.random((M, V)) < 0.5
    mask = to_dev(_pack(allowed))
    res = qmm.logprobs(logits, tokens=to_dev(tokens), k=k, scale=1.25, mask=mask)
    Reference(to_host(logits).astype(np.float64), 1.25, allowed).check(res, tokens, k)

    # the head and its statistics in one call, all rows at once
    one = qmm.mul_mat_logprobs(table, td, yh, M, V, D, tokens=to_dev(tokens), k=k, scale=1.25, mask=mask,
                               layout="repacked", rows=M)
    for a, b in zip(one, res):
        assert np.array_equal(to_host(a), to_host(b))


@pytest.mark.parametrize("fmt", ["q4_0", "q4_K", "q6_K", "q2_K"])
@pytest.mark.parametrize("M,rows", [(1, 1), (5, 8), (37, 8), (37, 21), (300, 64)])
def test_head_in_parts(fmt, M, rows):
    """Parts of `rows` rows (rounded down to a multiple of 8) with a remainder: each row's results are those of the
    two calls on its part, bit for bit; nothing is written past the workspace."""
    import torch
    V, D, k = 515, 512, 9
    print(fmt, M, rows, flush=True)
    rng = np.random.default_rng(M + rows)
    w = upload_weights(fmt, oracle.quantize(fmt, weights_t4_skewed([722, 1], V, D)), V, D, "repacked")
    x = to_dev(rng.standard_normal((M, D)).astype(np.float32))
    y = qmm.quantize_row_q8(x, ACT[fmt])
    tokens = to_dev(rng.integers(0, V, (M, 3)).astype(np.int32))
    mask = to_dev(_pack(rng.random((M, V)) < 0.7))
    need = qmm.mul_mat_logprobs_workspace_bytes(min(M, max(rows, 8)), V, k)
    ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
    got = qmm.mul_mat_logprobs(fmt, w, y, M, V, D, tokens=tokens, k=k, mask=mask, layout="repacked", workspace=ws[:need])
    assert (to_host(ws[need:]) == 77).all()
    step = M if rows >= M else rows // 8 * 8
    yb = y[:qmm.act_bytes(ACT[fmt], M, D)].view(M, -1)
    for m in range(0, M, step):
        n = min(step, M - m)
        logits = qmm.mul_mat(fmt, w, yb[m:m + n].contiguous(), n, V, D, layout="repacked")
        part = qmm.logprobs(logits, tokens=tokens[m:m + n].contiguous(), k=k, mask=mask[m:m + n].contiguous())
        for a, b in zip(got, part):
            assert torch.equal(a[m:m + n], b), (fmt, m)


def test_head_in_parts_split_rows_and_graph():
    """A vocabulary long enough that a row is cut over workgroups (the workspace holds logits and partial results),
    captured and replayed among eager work."""
    import torch
    V, D, M, k = 40000, 256, 11, 5
    rng = np.random.default_rng(8)
    w = upload_weights("q4_K", oracle.quantize("q4_K", weights_t4_skewed([723, 1], V, D)), V, D, "repacked")
    xs = [to_dev(rng.standard_normal((M, D)).astype(np.float32)) for _ in range(2)]
    y = torch.empty(qmm.act_bytes("q8_K", M, D), dtype=torch.uint8, device="cuda")
    tokens = to_dev(rng.integers(0, V, M).astype(np.int32))
    ws = torch.empty(qmm.mul_mat_logprobs_workspace_bytes(8, V, k), dtype=torch.uint8, device="cuda")

    def step(x):
        qmm.quantize_row_q8(x, "q8_K", out=y)
        return qmm.mul_mat_logprobs("q4_K", w, y, M, V, D, tokens=tokens, k=k, layout="repacked", workspace=ws)

    eager = [[t.clone() for t in step(x)] for x in xs]
    logits = qmm.mul_mat("q4_K", w, qmm.quantize_row_q8(xs[0][:8], "q8_K"), 8, V, D, layout="repacked")
    Reference(to_host(logits).astype(np.float64)).check([t[:8] for t in eager[0]], to_host(tokens)[:8], k)
    xin = torch.empty_like(xs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        xin.copy_(xs[0])
        step(xin)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step(xin)
    for rep in range(4):
        xin.copy_(xs[rep % 2])
        for t in got:
            t.fill_(3)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, eager[rep % 2]):
            assert torch.equal(a, b), rep
