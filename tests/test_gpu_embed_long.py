"""embed_rows for outputs of 32 MiB and more, which take a kernel of their own (two quads per thread, other stores):
every format and layout, rows that end inside the second quad's range and rows of several pieces, bad ids among them.
Tolerance and exactness as in test_gpu_embed.py; all rows are compared, on the GPU."""
import numpy as np
import pytest

import oracle
import bit_quantized_mat_quantize_amd as qmm
from bit_quantized_mat_quantize_amd.inputs import weights_t4_skewed
from gpu_helpers import to_dev, upload_weights

pytestmark = pytest.mark.gpu

LONG = 32 << 20


@pytest.mark.parametrize("scale", [1.0, 0.3])
@pytest.mark.parametrize("K", [256, 1280, 5120])
@pytest.mark.parametrize("layout", ["canonical", "repacked"])
@pytest.mark.parametrize("fmt", ["q4_0", "q4_K", "q6_K", "q2_K"])
def test_every_row(fmt, layout, K, scale):
    import torch
    N, T = 41, LONG // (4 * K) + 7
    print(fmt, layout, K, T, flush=True)
    w = oracle.quantize(fmt, weights_t4_skewed([730, K], N, K))
    rng = np.random.default_rng(K)
    ids = rng.integers(0, N, T).astype(np.int32)
    bad = np.array([0, 5, T // 2, T - 1])
    ids[bad] = [-1, N, 2**31 - 1, -2**31]
    out = torch.full((T + 1, K), -7.0, device="cuda")
    got = qmm.embed_rows(fmt, upload_weights(fmt, w, N, K, layout), to_dev(ids), N, K, layout=layout, scale=scale,
                         out=out[:T])
    assert got.numel() * 4 >= LONG
    table = to_dev(oracle.dequantize(fmt, w, N, K) * np.float64(np.float32(scale)))
    fine = torch.from_numpy((ids >= 0) & (ids < N)).cuda()
    want = table[torch.from_numpy(np.clip(ids, 0, N - 1)).cuda().long()]
    err = (got.double() - want).abs()
    bound = 0.0 if scale == 1.0 and fmt in ("q4_0", "q6_K") else 2 * 2.0 ** -24 * (1 + 1e-6)
    assert bool((err[fine] <= bound * want[fine].abs()).all())
    assert bool(got[~fine].isnan().all()) and bool((out[T] == -7.0).all())
