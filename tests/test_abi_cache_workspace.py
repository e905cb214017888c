"""The workspace of cache_attention, without a GPU: one of the largest call that a program makes serves its smaller ones.
Which calls take it is tried in a child process where no GPU exists: a valid call ends with QMM_EDEVICE there (the pointers
are placeholders), one whose workspace is too small with QMM_EINVAL."""
import os
import random
import subprocess
import sys

import pytest

from test_abi import lib  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def shapes(n):
    """Random calls: (type, heads, group, dim, page, width, sequences, rows, ragged)."""
    rng = random.Random(5)
    for _ in range(n):
        heads, group = rng.choice((1, 2, 3, 4, 8, 16, 64)), rng.choice((1, 2, 3, 4, 5, 8, 16))
        seqs, ragged = rng.choice((1, 2, 3, 9, 16, 32, 100, 255, 256, 257, 400)), rng.random() < 0.8
        rows = int(2 ** rng.uniform(0, 13)) if ragged else seqs
        yield (rng.choice((0, 1, 2)), heads, group, rng.choice((64, 96, 128, 192, 256)), rng.choice((16, 64, 256)),
               rng.choice((1, 2, 4, 8, 64, 256, 1000)), seqs, rows, ragged)


def test_no_smaller_call_needs_more(lib):  # noqa: F811
    def need(t, heads, group, dim, page, width, seqs, rows, ragged, mass):
        return lib.qmm_cache_attention_workspace_bytes(t, rows, heads * group, heads, dim, seqs, width, page, ragged, mass)

    rng = random.Random(6)
    for s in shapes(20000):
        t, heads, group, dim, page, width, seqs, rows, ragged = s
        for mass in (0, 1):
            n = need(*s, mass)
            assert n <= need(*s, 1), (s, "mass")
            assert n <= need(*s[:5], 2 * width, *s[6:], mass), (s, mass, "width")
            if ragged:
                more = rng.choice((1, 2, 10, 200, 5000))
                assert n <= need(*s[:7], rows + more, ragged, mass), (s, mass, more, "rows")
                assert n <= need(*s[:6], seqs + more, *s[7:], mass), (s, mass, more, "sequences")
            else:
                more = rng.choice((1, 2, 10, 200))
                assert n <= need(*s[:8], 1, mass), (s, mass, "starts")
                assert n <= need(*s[:6], seqs + more, rows + more, 1, mass), (s, mass, more, "both")


CHILD = r"""
import ctypes, random, sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
from bit_quantized_mat_quantize_amd import _binding
from test_abi_cache_workspace import shapes
lib = _binding.load()
hip = ctypes.CDLL("libamdhip64.so")
n = ctypes.c_int(0)
if hip.hipGetDeviceCount(ctypes.byref(n)) == 0 and n.value > 0:
    sys.exit(3)                      # a device exists: placeholder pointers must not be launched
p = lambda i: 65536 + (i << 52)
rng = random.Random(7)


def attend(s, lse, mass, size):
    t, heads, group, dim, page, width, seqs, rows, ragged = s
    c = _binding._Cache(p(0), 1 << 50, 8, page, heads, dim, p(1), seqs, width, p(2), p(3) if ragged else None, rows)
    ld = heads * group * dim
    return lib.qmm_cache_attention(ctypes.byref(c), t, p(4), 1 << 50, ld, heads * group, p(5), 1 << 50, ld, 0.1, 1, 0,
                                   p(6) if lse else None, p(7) if mass else None, width * page, p(8), size, None)


for s in shapes(1500):
    t, heads, group, dim, page, width, seqs, rows, ragged = s
    # weights of the entries: workgroups for whole tables, half as many as a launch has at most
    for mass in (0, 1) if seqs * heads * -(-width * page // 128) < 2**23 else (0,):
        # of this call with starts and mass, of a call of more rows and sequences: each serves this one
        size = lib.qmm_cache_attention_workspace_bytes
        sizes = [size(t, rows, heads * group, heads, dim, seqs, width, page, ragged, mass),
                 size(t, rows, heads * group, heads, dim, seqs, width, page, 1, 1),
                 size(t, rows + 300, heads * group, heads, dim, seqs + 300, 2 * width, page, 1, mass)]
        for lse in (0, 1):
            for i, n in enumerate(sizes):
                got = attend(s, lse, mass, n)
                assert got == 4, (s, lse, mass, i, n, got, lib.qmm_last_error())
"""


@pytest.mark.skipif(os.path.exists("/dev/kfd"), reason="placeholder pointers are only passed where no GPU exists")
def test_calls_take_the_workspace_of_a_larger_one():
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True, timeout=300)
    if r.returncode == 3:
        pytest.skip("a GPU is present")
    assert r.returncode == 0, r.stderr[-2000:]
