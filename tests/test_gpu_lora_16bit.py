"""lora_add with fp16 and bf16 adapters at the ends of their ranges: B subnormal beside normal numbers, elements of v
far below their row's largest, B large, v tiny or infinite.

Tolerance of `test_single_terms`.  A holds ones at one k each, so v is x to the bit, and each row of B has one element
that is not zero, so out = b x is one product of numbers of 24 and 11 (or 8, 24) bits.  The kernel may cut both into
pieces and add up the pieces' products, which are exact; with at most 6 of them and each addition off by at most one
step of the result (2u, u = 2^-24), |err| <= 12 u |out|, and the addition of a base of 0 is exact.  The other tests take
the bound of test_gpu_lora.py."""
import numpy as np
import pytest

import bit_quantized_mat_quantize_amd as qmm
from gpu_helpers import to_dev, to_host
from test_gpu_lora import U, _check, _formula, _torch_type

pytestmark = pytest.mark.gpu


def _run(base, x, A, B, ids, type):
    """Device result, and A, B as the 64-bit values that they hold in `type`."""
    a, b = to_dev(A).to(_torch_type(type)), to_dev(B).to(_torch_type(type))
    got = to_host(qmm.lora_add(to_dev(base), to_dev(x), a, b, to_dev(np.asarray(ids, np.int32))))
    return got, to_host(a.double()), to_host(b.double())


def _ones(R, K):
    """A [1, R, K] that takes x[k] as v[r] for r = k < R."""
    A = np.zeros((1, R, K), np.float32)
    A[0, np.arange(R), np.arange(R)] = 1.0
    return A


@pytest.mark.parametrize("M", [1, 20, 150])
@pytest.mark.parametrize("R", [5, 16, 40, 100])
@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
def test_single_terms(type, R, M):
    """Elements of v from 2^-40 to 1 of one row, normal and subnormal elements of B in every rank: each product alone
    keeps all of both factors' bits, whatever stands beside it."""
    print(type, R, M, flush=True)
    rng = np.random.default_rng(R + M)
    K, N = 128, 4 * R
    x = np.zeros((M, K), np.float32)
    x[:, :R] = rng.uniform(1, 2, (M, R)) * 2.0 ** rng.integers(-40, 1, (M, R)) * rng.choice([-1, 1], (M, R))
    x[:, 0] = 1.0
    B = np.zeros((1, N, R), np.float32)
    B[0, np.arange(N), np.arange(N) % R] = rng.uniform(1, 2, N) * 2.0 ** rng.integers(-22, 1, N)
    got, A64, B64 = _run(np.zeros((M, N), np.float32), x, _ones(R, K), B, np.zeros(M), type)
    want = x[:, :R].astype(np.float64) @ B64[0].T
    err = np.abs(got - want)
    assert (err <= 12 * U * np.abs(want)).all(), (err / np.abs(want)).max() / U


@pytest.mark.parametrize("M", [1, 40])
@pytest.mark.parametrize("type", ["f16", "bf16"])
def test_subnormal_b_beside_a_normal_number_without_effect(type, M):
    """A normal number in a row of B whose rank has v = 0 (an unused rank whose A is zero) changes nothing in how the
    subnormal numbers beside it are taken."""
    rng = np.random.default_rng(21)
    N, K, R = 70, 64, 16
    A = (rng.standard_normal((1, R, K)) / 8).astype(np.float32)
    A[0, 0] = 0.0
    B = (rng.standard_normal((1, N, R)) * 2e-6).astype(np.float32)
    B[0, :, 0] = 1.0
    x = rng.standard_normal((M, K)).astype(np.float32)
    base, ids = np.zeros((M, N), np.float32), np.zeros(M, np.int32)
    got, A64, B64 = _run(base, x, A, B, ids, type)
    _check(got, *_formula(base, x, A64, B64, ids))


@pytest.mark.parametrize("M", [2, 40])
@pytest.mark.parametrize("type", ["f16", "bf16"])
def test_ranks_far_apart(type, M):
    """The ranks with large v have no part in the odd columns of out, those with v 2^-30 of it have."""
    rng = np.random.default_rng(22)
    N, K, R = 65, 96, 12
    A = (rng.standard_normal((1, R, K)) / 10).astype(np.float32)
    A[0, 1::2] *= np.float32(2.0 ** -12)
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, K // 2:] *= np.float32(2.0 ** -18)
    A[0, 1::2, :K // 2] = 0.0
    B = rng.standard_normal((1, N, R)).astype(np.float32)
    B[0, 1::2, 0::2] = 0.0
    base, ids = np.zeros((M, N), np.float32), np.zeros(M, np.int32)
    got, A64, B64 = _run(base, x, A, B, ids, type)
    _check(got, *_formula(base, x, A64, B64, ids))


@pytest.mark.parametrize("M", [3, 40])
def test_large_finite_b(M):
    """bf16 reaches 2^127: products with a small v that fp32 holds come out."""
    rng = np.random.default_rng(23)
    N, K, R = 66, 64, 8
    A = (rng.standard_normal((1, R, K)) * 1e-6).astype(np.float32)
    B = (rng.uniform(0.5, 3, (1, N, R)) * rng.choice([-1e38, 1e35, 1e30], (1, N, R))).astype(np.float32)
    x = rng.standard_normal((M, K)).astype(np.float32)
    base, ids = np.zeros((M, N), np.float32), np.zeros(M, np.int32)
    got, A64, B64 = _run(base, x, A, B, ids, "bf16")
    assert np.isfinite(B64).all()
    _check(got, *_formula(base, x, A64, B64, ids))


@pytest.mark.parametrize("M", [1, 40])
@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
def test_tiny_v(type, M):
    """Rows of v between 2^-110 and 2^-80: as in test_single_terms (no result is subnormal)."""
    rng = np.random.default_rng(24)
    K, R = 64, 12
    N = 5 * R
    x = np.zeros((M, K), np.float32)
    x[:, :R] = rng.uniform(1, 2, (M, R)) * 2.0 ** rng.integers(-110, -80, (M, R)) * rng.choice([-1, 1], (M, R))
    B = np.zeros((1, N, R), np.float32)
    B[0, np.arange(N), np.arange(N) % R] = rng.uniform(1, 2, N) * 2.0 ** rng.integers(0, 10, N)
    got, A64, B64 = _run(np.zeros((M, N), np.float32), x, _ones(R, K), B, np.zeros(M), type)
    want = x[:, :R].astype(np.float64) @ B64[0].T
    err = np.abs(got - want)
    assert (err <= 12 * U * np.abs(want)).all(), (err / np.abs(want)).max() / U


@pytest.mark.parametrize("M", [1, 40])
@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
def test_infinite_v(type, M):
    """v past the largest fp32 number is infinite and so are the results it enters, also beside large elements of the
    other sign; a row that does not have it stays finite."""
    N, K, R = 20, 32, 3
    A = np.zeros((1, R, K), np.float32)
    A[0, 0, 0], A[0, 1, 1], A[0, 2, 2] = 10.0, 1.0, 1.0
    x = np.zeros((M, K), np.float32)
    x[:, 0], x[:, 1], x[:, 2] = 3e38, -1e6, 2.0
    if M > 1:
        x[M - 1, 0] = 0.0
    B = np.ones((1, N, R), np.float32)
    B[0, 1] = -1.0
    B[0, 2:, 1] = np.linspace(-2, 2, N - 2)
    got, A64, B64 = _run(np.zeros((M, N), np.float32), x, A, B, np.zeros(M), type)
    hit = slice(0, M - 1 if M > 1 else M)
    assert (got[hit, 0] == np.inf).all() and (got[hit, 1] == -np.inf).all() and (got[hit, 2:] == np.inf).all()
    if M > 1:
        assert np.isfinite(got[M - 1]).all() and got[M - 1, 0] == -1e6 + 2.0
