"""lora_add from one column range of a wide matrix to another one of it."""
import numpy as np
import pytest

import bit_quantized_mat_quantize_amd as qmm
from gpu_helpers import to_dev, to_host
from test_gpu_lora import _check, _formula, _inputs, _pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,at,to", [(1, 64, 0, 64), (7, 100, 0, 100), (50, 61, 64, 0), (300, 128, 300, 172), (40, 250, 0, 252)])
def test_from_columns_to_columns(M, N, at, to):
    """out holds the formula's result, base and all other columns what they held."""
    rng = np.random.default_rng(N)
    K, R, E, wide = 256, 12, 3, 512
    A, B, A64, B64 = _pool(rng, E, R, N, K, "bf16")
    x, _, ids = _inputs(rng, M, N, K, E=E)
    whole = rng.standard_normal((M, wide)).astype(np.float32)
    d = to_dev(whole.copy())
    got = qmm.lora_add(d[:, at:at + N], to_dev(x), A, B, to_dev(ids), out=d[:, to:to + N])
    assert got.data_ptr() == d[:, to:to + N].data_ptr()
    after = to_host(d)
    _check(after[:, to:to + N], *_formula(whole[:, at:at + N], x, A64, B64, ids))
    rest = np.ones(wide, bool)
    rest[to:to + N] = False
    assert np.array_equal(after[:, rest].view(np.uint32), whole[:, rest].view(np.uint32))


def test_shared_columns_are_refused():
    rng = np.random.default_rng(2)
    A, B, _, _ = _pool(rng, 2, 4, 64, 32, "f16")
    d, x, ids = to_dev(np.zeros((5, 500), np.float32)), to_dev(np.zeros((5, 32), np.float32)), to_dev(np.zeros(5, np.int32))
    for at, to in ((0, 60), (436, 408), (100, 40)):
        with pytest.raises(qmm.QmmError, match="overlaps base"):
            qmm.lora_add(d[:, at:at + 64], x, A, B, ids, out=d[:, to:to + 64])
