"""cache_attention of long runs of fp16 rows: keys are not rounded, whatever is asked for.  With scores of hundreds a key
rounded to fp16 would move a weight by per cents; the tolerance has no room for that."""
import numpy as np
import pytest
import torch

from kv_reference import qmm, to_host, tolerance
from test_gpu_cache_attention import queries
from test_gpu_cache_many_steps import batch_of, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("heads,group,tokens", [(128, 1, 300), (2, 4, 80), (1, 33, 70)])
@pytest.mark.parametrize("scale", [0.0, 1.0, -2.0])
def test_fp16_rows_see_keys_as_they_are(scale, heads, group, tokens, D):
    rng = np.random.default_rng([80, D, heads])
    b = batch_of(rng, [tokens + 400], [tokens], heads, D, 32)
    qd, q = queries(rng, tokens, heads * group, D, "f16", 1.5)
    scale = scale or D ** -0.5
    print(scale, heads, group, D, flush=True)
    out, lse, _, slack = ref = reference(b, q, scale)
    tol, ds = tolerance("f16", D, tokens + 400, slack, out)
    cache, table, lens, st = b.dev()
    alone = qmm.cache_attention(qd.cuda(), cache, table, lens, st, scale=scale)
    got, sums = qmm.cache_attention(qd.cuda(), cache, table, lens, st, scale=scale, lse=True)
    for o in (alone, got):
        err = np.abs(to_host(o).astype(np.float64) - out)
        assert (err <= tol).all(), (err / tol).max()
    assert (np.abs(to_host(sums) - lse) <= (ds + 2.0 ** -22 * (2 + np.abs(lse))) * 1.01).all()
    assert torch.equal(alone, got)      # whether lse is asked for changes nothing
