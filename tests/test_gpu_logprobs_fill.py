"""Places of the top list that no token takes, in rows that a NaN or +inf makes NaN otherwise."""
import numpy as np
import pytest

import bit_quantized_mat_quantize_amd as qmm
from gpu_helpers import to_dev, to_host
from test_gpu_logprobs import _pack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V", [70, 5001, 50001])
@pytest.mark.parametrize("poison", [np.nan, np.inf])
def test_unused_places_of_a_poisoned_row(poison, V):
    """Three tokens are allowed and one of them poisons its row; k = 6.  A NaN is no candidate, +inf is the first one;
    the candidates' log probabilities are NaN as the row's are, and the other places hold -1 and -inf."""
    rng = np.random.default_rng(V)
    x = rng.standard_normal((3, V)).astype(np.float32)
    at = np.array([4, V // 2, V - 1])
    allowed = np.zeros((3, V), bool)
    allowed[:, at] = True
    x[1, V // 2] = poison
    lp, H, ids, tl = (to_host(t) for t in qmm.logprobs(to_dev(x), tokens=to_dev(np.full((3, 1), 4, np.int32)), k=6,
                                                       mask=to_dev(_pack(allowed))))
    assert np.isnan(lp[1]).all() and np.isnan(H[1])
    some = 2 if np.isnan(poison) else 3
    assert set(ids[1, :some]) <= set(at) and (poison != np.inf or ids[1, 0] == V // 2)
    assert np.isnan(tl[1, :some]).all()
    assert (ids[1, some:] == -1).all() and (tl[1, some:] == -np.inf).all()
    for m in (0, 2):
        assert (np.sort(ids[m, :3]) == at).all() and np.isfinite(tl[m, :3]).all()
        assert (ids[m, 3:] == -1).all() and (tl[m, 3:] == -np.inf).all()
