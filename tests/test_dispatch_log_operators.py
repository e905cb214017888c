"""The launch shapes of embed_rows, lora_add, logprobs and mul_mat_logprobs, read from the QMM_LOG line each call
prints.  As in test_dispatch_log.py: the shape is chosen and logged after the argument checks and before the launch,
which fails with QMM_EDEVICE where there is no GPU; the pointers are placeholders."""
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
big = 1 << 48
p = lambda i: 65536 + (i << 52)
for T, K in ((1, 4096), (2048, 4096)):
    assert lib.qmm_embed_rows(2, p(0), big, 1, p(1), T, 1.0, p(2), big, 1000, K, None) == 4
for M, N, K, R, E in ((1, 4096, 4096, 16, 8), (32, 8192, 8192, 16, 64), (2048, 28672, 8192, 16, 4), (100, 64, 256, 70, 2)):
    assert lib.qmm_lora_add(1, p(0), big, p(1), big, E, R, None, None, p(2), big, p(3), p(4), big, N, p(4), big, N, M, N, K,
                            p(5), big, None) == 4
for M, V in ((1, 32768), (1, 32769), (1, 1 << 20), (32, 128256), (513, 50257), (1024, 128256)):
    assert lib.qmm_logprobs(0, p(0), big, V, M, V, 1.0, None, 0, 0, None, 0, None, p(1), 0, None, None, p(2), big, None) == 4
row = lib.qmm_mul_mat_logprobs_workspace_bytes(1, 1000, 0)
for M, rows in ((100, 100), (100, 47), (5, 5)):
    assert lib.qmm_mul_mat_logprobs(1, p(0), big, 1, p(1), big, M, 1000, 256, 1.0, None, 0, 0, None, 0, None, p(2), 0, None,
                                    None, p(3), rows * row, None) == 4
"""

EXPECTED = [
    "embed_rows Q6_K T=1 N=1000 K=4096 layout=repacked -> plain stores",
    "embed_rows Q6_K T=2048 N=1000 K=4096 layout=repacked -> stores past the caches",
    "lora_add M=1 N=4096 K=4096 R=16 E=8 -> K in 8 parts, 1 workgroup(s) per 16-row tile, in place",
    "lora_add M=32 N=8192 K=8192 R=16 E=64 -> K in 16 parts, 16 workgroup(s) per 16-row tile, in place",
    "lora_add M=2048 N=28672 K=8192 R=16 E=4 -> K in 4 parts, 1 workgroup(s) per 16-row tile, in place",
    "lora_add M=100 N=64 K=256 R=70 E=2 -> K in 1 parts, 2 workgroup(s) per 16-row tile, in place",
    "logprobs M=1 V=32768 G=0 k=0 -> 1 workgroup(s) per row",
    "logprobs M=1 V=32769 G=0 k=0 -> 5 workgroup(s) per row",
    "logprobs M=1 V=1048576 G=0 k=0 -> 64 workgroup(s) per row",
    "logprobs M=32 V=128256 G=0 k=0 -> 16 workgroup(s) per row",
    "logprobs M=513 V=50257 G=0 k=0 -> 1 workgroup(s) per row",
    "logprobs M=1024 V=128256 G=0 k=0 -> 1 workgroup(s) per row",
    "mul_mat_logprobs Q4_K M=100 N=1000 K=256 -> 100 rows at a time",
    "mul_mat_logprobs Q4_K M=100 N=1000 K=256 -> 40 rows at a time",
    "mul_mat_logprobs Q4_K M=5 N=1000 K=256 -> 5 rows at a time",
]


def test_launch_shapes():
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True,
                       env=dict(os.environ, QMM_LOG="1"), timeout=300)
    if r.returncode == 3:
        pytest.skip("a GPU is present")
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [l[len("qmm: "):] for l in r.stderr.splitlines() if l.startswith("qmm: ") and not l.startswith("qmm: mul_mat_q")
             and " mul_mat Q" not in l]
    assert [l for l in lines if l.split()[0] in ("embed_rows", "lora_add", "logprobs", "mul_mat_logprobs")] == EXPECTED
