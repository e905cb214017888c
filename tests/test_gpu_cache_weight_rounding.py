"""cache_attention of fp16 rows, few of a sequence: weights are not rounded to 11 bits.  Values whose products with their
codes are exact in fp16 (scales that are powers of two) and that cancel in the sum show a weight's rounding alone."""
import numpy as np
import pytest

from kv_reference import qmm, to_host, tolerance
from test_gpu_cache_attention import queries
from test_gpu_cache_many_steps import batch_of, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("rows,group,lens", [(1, 4, [2, 3, 39, 700]), (1, 33, [50]), (5, 8, [17, 300]), (3, 2, [90, 3])])
@pytest.mark.parametrize("kind", ["f16", "f32"])
def test_weights_of_values_that_cancel(kind, rows, group, lens, D):
    rng = np.random.default_rng([90, D, rows])
    b = batch_of(rng, lens, [rows] * len(lens), 2, D, 16)
    v = b.cache.h[:, 1]
    v[np.isfinite(v)] = np.float16(0.25) * np.sign(v[np.isfinite(v)])
    qd, q = queries(rng, b.T, 2 * group, D, kind, 0.05)       # flat weights: no entry takes all
    print(kind, rows, group, lens, D, flush=True)
    out, _, _, slack = ref = reference(b, q, D ** -0.5)
    # as fp32 rows, whose weights are held to 2^-21, but for the rounding of the result
    tol, _ = tolerance("f32", D, max(lens), slack, out)
    tol = tol + (2.0 ** -11 * np.abs(out) + 2.0 ** -25 if kind == "f16" else 0.0)
    cache, table, ln, st = b.dev()
    got = qmm.cache_attention(qd.cuda(), cache, table, ln, st)
    err = np.abs(to_host(got).astype(np.float64) - out)
    assert (err <= tol).all(), (err / tol).max()
