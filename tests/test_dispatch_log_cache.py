"""What cache_evict launches and refuses near the limit of a launch's workgroups, and which calls of cache_attention have
the kernel of long runs of rows.  As in test_dispatch_log.py: a valid call
is logged after the argument checks and before the launch, which fails with QMM_EDEVICE where there is no GPU; the
pointers are placeholders."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(os.path.exists("/dev/kfd"),
                                reason="placeholder pointers are only passed where no GPU exists")

CHILD = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
from bit_quantized_mat_quantize_amd import _binding
lib = _binding.load()
hip = ctypes.CDLL("libamdhip64.so")
n = ctypes.c_int(0)
if hip.hipGetDeviceCount(ctypes.byref(n)) == 0 and n.value > 0:
    sys.exit(3)                      # a device exists: placeholder pointers must not be launched
p = lambda i: 65536 + (i << 52)
SEQS, HEADS = 4096, 64               # 2 * SEQS * HEADS = 2^19 workgroups for each chunk of entries: 31 chunks at most


def evict(dim, budget, same=False):
    c = _binding._Cache(p(0), 1 << 50, 8, 16, HEADS, dim, p(1), SEQS, 1024, p(2), None, 0)
    return lib.qmm_cache_evict(ctypes.byref(c), p(3), 1024 * 16, budget, 5, p(1) if same else p(4), 1024, p(5), p(6),
                               1024 * 16, p(7), None)


# entries of a chunk: 256 threads over the blocks of an entry, in fours
for dim, chunk in ((64, 128), (96, 84), (128, 64), (192, 40), (256, 32)):
    print(dim, evict(dim, 31 * chunk), evict(dim, 31 * chunk + 1), evict(dim, 31 * chunk + 1, True))
"""


def test_evict_up_to_the_largest_launch():
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True,
                       env=dict(os.environ, QMM_LOG="1"), timeout=300)
    if r.returncode == 3:
        pytest.skip("a GPU is present")
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.split("\n")[:5] == [f"{dim} 4 3 4" for dim in (64, 96, 128, 192, 256)]


ATTEND_HEAD = r"""
import ctypes, sys
sys.path.insert(0, sys.argv[1])
from bit_quantized_mat_quantize_amd import _binding
lib = _binding.load()
hip = ctypes.CDLL("libamdhip64.so")
n = ctypes.c_int(0)
if hip.hipGetDeviceCount(ctypes.byref(n)) == 0 and n.value > 0:
    sys.exit(3)
p = lambda i: 65536 + (i << 52)
"""
ATTEND = ATTEND_HEAD + r"""
for t in (0, 1, 2):
    for dim in (64, 96, 128, 192, 256):
        for lse, mass in ((0, 0), (1, 0), (0, 1), (1, 1)):
            c = _binding._Cache(p(0), 1 << 50, 8, 64, 8, dim, p(1), 2, 128, p(2), p(3), 4096)
            assert lib.qmm_cache_attention(ctypes.byref(c), t, p(4), 1 << 50, 32 * dim, 32, p(5), 1 << 50, 32 * dim, 0.1, 1, 0,
                                           p(6) if lse else None, p(7) if mass else None, 8192, p(8), 1 << 50, None) == 4
"""


def test_long_runs_have_their_kernel_whatever_is_asked_for():
    """Two prompts of 2048 rows: 256 rows share a tile's entries, with lse or mass or without."""
    r = subprocess.run([sys.executable, "-c", ATTEND, ROOT], capture_output=True, text=True,
                       env=dict(os.environ, QMM_LOG="1"), timeout=300)
    if r.returncode == 3:
        pytest.skip("a GPU is present")
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [l for l in r.stderr.splitlines() if l.startswith("qmm: cache_attention")]
    got = [(l.split()[2], int(l.split("dim=")[1].split()[0]), int(l.split(" of long runs")[0].split()[-1]) > 0) for l in lines]
    assert got == [(t, dim, dim <= (128 if t == "fp32" else 192)) for t in ("fp32", "fp16", "bf16")
                   for dim in (64, 96, 128, 192, 256) for _ in range(4)]


BORDERS = ATTEND_HEAD + r"""
for t, rows in ((0, 768), (0, 769), (1, 256), (1, 257), (2, 256), (2, 257)):
    c = _binding._Cache(p(0), 1 << 50, 8, 64, 8, 128, p(1), 2, 128, p(2), p(3), rows)
    assert lib.qmm_cache_attention(ctypes.byref(c), t, p(4), 1 << 50, 1024, 8, p(5), 1 << 50, 1024, 0.1, 1, 0, None, None, 0,
                                   p(8), 1 << 50, None) == 4
"""


def test_from_how_many_rows_on():
    """The kernel of long runs begins where it was measured to pay: above 256 rows in 16 bits, 768 in fp32."""
    r = subprocess.run([sys.executable, "-c", BORDERS, ROOT], capture_output=True, text=True,
                       env=dict(os.environ, QMM_LOG="1"), timeout=300)
    if r.returncode == 3:
        pytest.skip("a GPU is present")
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [l for l in r.stderr.splitlines() if l.startswith("qmm: cache_attention")]
    assert [int(l.split(" of long runs")[0].split()[-1]) > 0 for l in lines] == [False, True] * 3
