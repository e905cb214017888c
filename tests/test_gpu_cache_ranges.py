"""cache_attention where numbers of very different size stand beside one another in a call: what a row is off by then.

Keys and values are scaled by powers of two that fit the largest block that rows of the call see, queries by one that fits
their row's largest element, so that fp16 pieces hold them; what is far below it keeps a step of its own:
  * an element of a query is held to 2^-33 of its row's largest (the pieces' last step is 2^-24, rounded to half of it,
    beside a largest of 2^8 or more);
  * a block scale to half of 2^-24 beside a largest of 2^7: 2^-32 of it, and so a key or value to 2^-32 of eight times the largest
    scale; the products with the codes, rounded in 16 bits, to 2^-25 once more: 2^-31 covers both."""
import numpy as np
import pytest
import torch

from kv_reference import qmm, to_host, tolerance
from test_gpu_cache_attention import queries
from test_gpu_cache_many_steps import RUN, batch_of, reference

pytestmark = pytest.mark.gpu


def check(kind, b, q, qd, long, **kw):
    D, scale = b.D, b.D ** -0.5
    ref = reference(b, q, scale, **kw)
    out_ref, lse_ref, _, slack = ref
    tol, ds = tolerance(kind, D, max(b.lens), slack, out_ref, rounded_keys=long)
    d = np.abs(b.cache.h.astype(np.float64))
    kmax, vmax = 8 * np.nanmax(d[:, 0]), 8 * np.nanmax(d[:, 1])
    absq = np.abs(q.astype(np.float64))
    # each score's further error, which a weight has twice (its own and the sum's)
    k_sum = D * kmax if long else 0.0
    k_all = max(np.abs(np.nan_to_num(b.cache.get(p, t, 0))).sum(-1).max() for p in range(b.cache.pages) for t in range(b.page))
    more = scale * (2.0 ** -33 * absq.max(-1) * k_all + 2.0 ** -31 * kmax * (absq.sum(-1) if k_sum else 0.0))
    bound = tol + 2.02 * more[..., None] * slack[1] + 2.0 ** -31 * vmax
    cache, table, lens, st = b.dev()
    got = to_host(qmm.cache_attention(qd.cuda(), cache, table, lens, st, **kw)).astype(np.float64)
    err = np.abs(got - out_ref)
    assert np.isfinite(got).all() and (err <= bound).all(), (err.max(), (err / bound).max())
    return err, tol


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("part", [0, 1])
def test_a_large_entry_that_few_rows_see(part, many, kind):
    """The last two entries are 2^14 to 2^26 times the others, which most rows do not see."""
    rng = np.random.default_rng([70, part])
    n, heads = (RUN[kind][0], RUN[kind][1]) if many else (40, 2)
    L = n + 60
    for power in (14, 20, 26):
        b = batch_of(rng, [L], [n], heads, 64, 64)
        small = 2.0 ** (-10 if part == 1 else -2)
        b.cache.h[:, part] = (b.cache.h[:, part].astype(np.float64) * small).astype(np.float16)
        for p in (L - 2, L - 1):
            at = b.table[0, p // 64], part, slice(None), p % 64
            b.cache.h[at] = np.clip(b.cache.h[at].astype(np.float64) * 2.0 ** power, -60000, 60000).astype(np.float16)
        qd, q = queries(rng, n, heads, 64, kind, 0.5)
        if part == 0:         # so that scores of the large keys stay within thousands
            qd = (qd.float() * 2.0 ** -12).to(qd.dtype)
            q = qd.float().numpy()
        print(kind, many, part, power, flush=True)
        err, tol = check(kind, b, q, qd, many)
        print("of the ordinary tolerance:", (err / tol).max(), flush=True)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_a_large_element_of_a_query(kind):
    """One element of a row 2^12 to 2^24 times the others, where the keys hold zeros."""
    rng = np.random.default_rng(71)
    for power in (12, 18, 24) if kind != "f16" else (12,):
        b = batch_of(rng, [150], [30], 2, 64, 32)
        b.cache.q[:, 0, ..., 5] = 8       # element 5 of every key is 0
        b.cache.q[:, 0, ..., 38] = 8
        qd, q = queries(rng, 30, 4, 64, kind)
        for e in (5, 38):
            qd[..., e] *= 2.0 ** power
        q = qd.float().numpy()
        print(kind, power, flush=True)
        err, tol = check(kind, b, q, qd, False)
        print("of the ordinary tolerance:", (err / tol).max(), flush=True)
