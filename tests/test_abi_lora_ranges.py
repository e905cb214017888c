"""lora_add from one column range of a wide matrix to another: accepted where no row shares an element, refused
elsewhere.  Without a GPU: a call that passes the checks fails at the launch with QMM_EDEVICE, the pointers are
placeholders."""
import os

import pytest

from test_abi import EINVAL, _last, lib  # noqa: F401
from test_abi_operators import BIG, _far

pytestmark = pytest.mark.skipif(os.path.exists("/dev/kfd"),
                                reason="placeholder pointers are only passed where no GPU exists")
EDEVICE = 4


def test_column_ranges(lib):  # noqa: F811
    def call(offset, M=5, N=96, ldb=400, ldo=400, x=_far(2), ws=_far(6)):
        """out `offset` floats behind base."""
        return lib.qmm_lora_add(1, _far(0), BIG, _far(1), BIG, 4, 8, None, None, x, BIG, _far(3), _far(4), BIG, ldb,
                                _far(4) + 4 * offset, BIG, ldo, M, N, 64, ws, BIG, None)

    # beside base in the same rows, on either side, to the last column, and rows further on
    for offset in (96, 100, 304, -96, -304, 400 + 96, 400 + 304, -400 - 96, 3 * 400 + 200, 5 * 400, 6 * 400):
        assert call(offset) == EDEVICE, (offset, _last(lib))
    # shared columns, in the same row or in another one, on either side of the wrap to the next row
    for offset in (4, 92, 308, 396, 400, 404, 400 + 92, 400 + 308, -4, -92, -308, -396, -400, 4 * 400, 4 * 400 + 92):
        assert call(offset) == EINVAL and "overlaps base" in _last(lib), offset
    # ranges that fill the rows between them, and ones too wide for it
    assert call(200, N=200) == EDEVICE and call(200, N=204) == EINVAL and call(-200, N=204) == EINVAL
    # another row stride: the whole ranges must be apart
    assert call(96, ldo=404) == EINVAL and call(4 * 400 + 96, ldo=404) == EDEVICE
    assert call(0) == EDEVICE and call(0, ldo=404) == EINVAL
    # x, ids and the workspace may not lie between the rows
    assert call(96, x=_far(4) + 4 * 200) == EINVAL and call(96, ws=_far(4) + 4 * 200) == EINVAL
