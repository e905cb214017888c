"""lora_add against the formula in 64 bits.

Tolerance.  u = 2^-24.  v = sum_k A x is a sum of K exact-operand products: at
most K roundings of the partial sums and one of each product, |dv| <= (K + 1) u *
sum|A x|; the scale rounds once more.  The second product adds R + 1, the
addition of the base one (of the result).  With T = s * sum_r |B| sum_k |A x|:
|d out| <= (K + R + 4) u T + u |out|, to first order; 1.01 covers the rest.
Integer inputs whose sums stay below 2^24 are exact in any order."""
import numpy as np
import pytest

import bit_quantized_mat_quantize_amd as qmm
from gpu_helpers import to_dev, to_host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _torch_type(name):
    import torch
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def _pool(rng, E, R, N, K, type):
    """A, B as device tensors of `type` and as the 64-bit values they hold."""
    A = to_dev((rng.standard_normal((E, R, K)) / np.sqrt(K)).astype(np.float32)).to(_torch_type(type))
    B = to_dev((rng.standard_normal((E, N, R)) * 0.2).astype(np.float32)).to(_torch_type(type))
    return A, B, to_host(A.double()), to_host(B.double())


def _formula(base, x, A, B, ids, scales=None, ranks=None):
    """out and the bound of its error, rows with an id that names no adapter left out (NaN)."""
    M, N = base.shape
    E, R, K = A.shape
    out, tol = base.astype(np.float64), np.zeros((M, N))
    for m, e in enumerate(ids):
        if e == -1:
            continue
        if not 0 <= e < E:
            out[m] = np.nan
            continue
        r = R if ranks is None else min(max(int(ranks[e]), 0), R)
        s = 1.0 if scales is None else np.float64(scales[e])
        a, b = A[e, :r], B[e, :, :r]
        xm = x[m].astype(np.float64)
        out[m] += s * (b @ (a @ xm))
        tol[m] = 1.01 * ((K + R + 4) * U * abs(s) * (np.abs(b) @ (np.abs(a) @ np.abs(xm))) + U * np.abs(out[m]))
    return out, tol


def _check(got, out, tol, what=""):
    got = got.astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(out)), what
    fine = ~np.isnan(out)
    err = np.abs(got - out)[fine]
    assert (err <= tol[fine]).all(), (what, (err - tol[fine]).max())


def _inputs(rng, M, N, K, ids=None, E=1):
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[:, rng.integers(0, K)] *= 20
    base = rng.standard_normal((M, N)).astype(np.float32)
    if ids is None:
        ids = rng.integers(-1, E, M).astype(np.int32)
    return x, base, np.asarray(ids, np.int32)


@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,K,R,E", [(1, 1, 32, 1, 1), (1, 4096, 1024, 16, 3), (2, 70, 64, 3, 2), (5, 257, 96, 7, 8),
                                       (16, 512, 256, 8, 16), (17, 300, 2080, 24, 4), (33, 129, 320, 64, 64),
                                       (65, 1030, 512, 33, 5), (130, 260, 128, 100, 3), (530, 36, 4096, 12, 9),
                                       (40, 64, 32, 256, 2), (70, 260, 96, 4, 5), (200, 131, 64, 6, 4),
                                       (33, 516, 160, 10, 7), (12, 300, 2048, 20, 3), (140, 68, 4096, 34, 6),
                                       (9, 5, 64, 60, 2), (300, 1028, 64, 130, 2)])
def test_formula(M, N, K, R, E, type):
    print(M, N, K, R, E, type, flush=True)
    rng = np.random.default_rng(M * 1000 + N + K + R)
    A, B, A64, B64 = _pool(rng, E, R, N, K, type)
    x, base, ids = _inputs(rng, M, N, K, E=E)
    if M == 1:
        ids[:] = E - 1
    scales = rng.uniform(-2, 2, E).astype(np.float32)
    ranks = rng.integers(-1, R + 3, E).astype(np.int32)       # 0, below 0 and above R among them
    got = to_host(qmm.lora_add(to_dev(base), to_dev(x), A, B, to_dev(ids), scales=to_dev(scales),
                               ranks=to_dev(ranks)))
    _check(got, *_formula(base, x, A64, B64, ids, scales, ranks))
    got = to_host(qmm.lora_add(to_dev(base), to_dev(x), A, B, to_dev(ids)))
    _check(got, *_formula(base, x, A64, B64, ids))


@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,R", [(3, 50, 5), (48, 200, 16), (700, 96, 40)])
def test_integers_are_exact(M, N, R, type):
    """Small integers: any order of the sums gives the integer result; wrong elements of any tile would show."""
    import torch
    rng = np.random.default_rng(R)
    K, E = 160, 6
    A = rng.integers(-3, 4, (E, R, K)).astype(np.float32)
    B = rng.integers(-3, 4, (E, N, R)).astype(np.float32)
    x = rng.integers(-5, 6, (M, K)).astype(np.float32)
    base = rng.integers(-100, 101, (M, N)).astype(np.float32)
    ids = rng.integers(-1, E, M).astype(np.int32)
    dt = _torch_type(type)
    got = to_host(qmm.lora_add(to_dev(base), to_dev(x), to_dev(A).to(dt), to_dev(B).to(dt), to_dev(ids)))
    want, _ = _formula(base, x, A.astype(np.float64), B.astype(np.float64), ids)
    assert np.abs(want).max() < 2 ** 24
    assert np.array_equal(got.astype(np.float64), want)


@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("M,N,R", [(100, 19200, 12), (100, 19001, 20), (144, 60000, 16), (300, 28001, 40),
                                   (20, 70001, 4), (520, 17000, 6)])
def test_wide_outputs_are_exact(M, N, R, type):
    """Several column groups per workgroup, outputs past the caches, K in five parts: integers as above.
    |v| <= 5 * 3 * 2560 and |out| <= 100 + 3 * 40 * 38400 < 2^24, so every sum is exact in fp32."""
    rng = np.random.default_rng(M + N + R)
    K, E = 2560, 5
    A = rng.integers(-3, 4, (E, R, K)).astype(np.float32)
    B = rng.integers(-3, 4, (E, N, R)).astype(np.float32)
    x = rng.integers(-5, 6, (M, K)).astype(np.float32)
    base = rng.integers(-100, 101, (M, N)).astype(np.float32)
    ids = np.repeat(rng.integers(-1, E, (M + 6) // 7), 7)[:M].astype(np.int32)  # runs of seven rows
    dt = _torch_type(type)
    got = to_host(qmm.lora_add(to_dev(base), to_dev(x), to_dev(A).to(dt), to_dev(B).to(dt), to_dev(ids)))
    want = base.astype(np.float64)
    for e in range(E):
        rows = ids == e
        v = x[rows].astype(np.float64) @ A[e].astype(np.float64).T
        want[rows] += v @ B[e].astype(np.float64).T
    assert np.array_equal(got.astype(np.float64), want)


@pytest.mark.parametrize("M", [7, 64, 600])
def test_routing(M):
    """All rows one adapter, each row its own, none at all, sorted and shuffled: the same rows give the same bits."""
    rng = np.random.default_rng(M)
    N, K, R, E = 96, 128, 16, 64
    A, B, A64, B64 = _pool(rng, E, R, N, K, "bf16")
    x, base, _ = _inputs(rng, M, N, K, E=E)
    for ids in (np.full(M, 5), np.arange(M) % E, np.sort(rng.integers(0, E, M)), np.full(M, -1),
                np.where(np.arange(M) % 3 == 0, -1, 9)):
        ids = ids.astype(np.int32)
        got = to_host(qmm.lora_add(to_dev(base), to_dev(x), A, B, to_dev(ids)))
        _check(got, *_formula(base, x, A64, B64, ids))
        assert np.array_equal(got[ids == -1].view(np.uint32), base[ids == -1].view(np.uint32))
        order = rng.permutation(M)
        mixed = to_host(qmm.lora_add(to_dev(base[order]), to_dev(x[order]), A, B, to_dev(ids[order])))
        assert np.array_equal(mixed.view(np.uint32), got[order].view(np.uint32))


@pytest.mark.parametrize("M", [5, 100])
def test_bad_ids_and_unused_values(M):
    """Ids that name no adapter give NaN rows and nothing else; what lies behind an adapter's rank, in adapters
    that no row asks for and in rows without an adapter may be NaN or infinite."""
    rng = np.random.default_rng(M)
    N, K, R, E = 70, 96, 12, 5
    A, B, A64, B64 = _pool(rng, E, R, N, K, "f16")
    ranks = np.array([12, 5, 0, 7, 12], np.int32)
    for e in range(E):
        A[e, ranks[e]:], B[e, :, ranks[e]:] = float("nan"), float("inf")
    A[4], B[4] = float("inf"), float("nan")
    x, base, _ = _inputs(rng, M, N, K, E=E)
    ids = rng.integers(0, 4, M).astype(np.int32)
    ids[0], ids[1], ids[2], ids[-1] = E, -2, -1, 2**31 - 1
    x[:3], x[-1] = np.nan, np.inf
    got = to_host(qmm.lora_add(to_dev(base), to_dev(x), A, B, to_dev(ids), ranks=to_dev(ranks)))
    want, tol = _formula(base, np.where(np.isfinite(x), x, 0), np.nan_to_num(A64), np.nan_to_num(B64), ids, None, ranks)
    _check(got, want, tol)
    assert np.isnan(got[[0, 1, -1]]).all() and np.array_equal(got[2], base[2])


@pytest.mark.parametrize("M,N", [(3, 64), (50, 61), (600, 256)])
def test_in_place_and_column_ranges(M, N):
    """Two adapters' outputs on the halves of one concatenated projection, in place; nothing around them changes."""
    import torch
    rng = np.random.default_rng(N)
    K, R, E, wide = 256, 8, 3, 1000
    x, _, ids = _inputs(rng, M, N, K, E=E)
    ids[0] = E + 1                              # a bad row stays inside its columns too
    whole = rng.standard_normal((M, wide)).astype(np.float32)
    out = to_dev(whole.copy())
    want, tol = whole.astype(np.float64), np.zeros(whole.shape)
    for at, type in ((0, "f16"), (wide - 400, "bf16")):
        A, B, A64, B64 = _pool(rng, E, R, N, K, type)
        view = out[:, at:at + N]
        got = qmm.lora_add(view, to_dev(x), A, B, to_dev(ids), out=view)
        assert got.data_ptr() == view.data_ptr()
        want[:, at:at + N], tol[:, at:at + N] = _formula(whole[:, at:at + N], x, A64, B64, ids)
        # the same out of place, from and to other strides
        dst = torch.full((M, N + 3), -7.0, device="cuda")
        qmm.lora_add(to_dev(whole)[:, at:at + N], to_dev(x), A, B, to_dev(ids), out=dst[:, :N])
        dst = to_host(dst)
        assert np.array_equal(dst[:, :N].view(np.uint32), to_host(view).view(np.uint32)) and (dst[:, N:] == -7).all()
    got = to_host(out)
    _check(got, want, tol)
    free = np.ones(wide, bool)
    free[:N] = free[wide - 400:wide - 400 + N] = False
    assert np.array_equal(got[:, free], whole[:, free])


@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("scale_x,scale_b", [(1.0, 1e-6), (1e30, 1e-5), (1e-30, 1.0), (3e4, 100.0)])
@pytest.mark.parametrize("M", [2, 40])
def test_magnitudes(M, scale_x, scale_b, type):
    """B subnormal in fp16, x far outside its range, rows of v whose elements lie far apart."""
    print(M, scale_x, scale_b, type, flush=True)
    rng = np.random.default_rng(11)
    N, K, R, E = 65, 64, 20, 2
    A, B, _, _ = _pool(rng, E, R, N, K, "f32")
    A = (A * to_dev((10.0 ** rng.uniform(-6, 0, (E, R, 1))).astype(np.float32))).to(_torch_type(type))
    B = B * scale_b
    B[:, 3::5] *= 1e-4                                  # rows far below their neighbours
    B = B.to(_torch_type(type))
    x, _, ids = _inputs(rng, M, N, K, E=E)
    x = (x * scale_x).astype(np.float32)
    base = np.zeros((M, N), np.float32)
    ids[0] = 1
    got = to_host(qmm.lora_add(to_dev(base), to_dev(x), A, B, to_dev(ids)))
    out, tol = _formula(base, x, to_host(A.double()), to_host(B.double()), ids)
    # what fp16 pieces leave: below 2^-33 of the row's largest v, times sum|B|
    for m, e in enumerate(ids):
        if e >= 0:
            v = np.abs(to_host(A[e].double()) @ x[m].astype(np.float64)).max()
            tol[m] += 2.0 ** -33 * v * np.abs(to_host(B[e].double())).sum(1)
    _check(got, out, tol)


def test_out_past_4_gib():
    """Rows of base and out that lie past 2^32 bytes, sampled."""
    import torch
    M, N, K, R, E = 40000, 28672, 32, 4, 3
    rng = np.random.default_rng(12)
    A, B, A64, B64 = _pool(rng, E, R, N, K, "bf16")
    x, _, ids = _inputs(rng, M, 1, K, E=E)
    base = torch.zeros(M, N, device="cuda")
    base += torch.arange(M, device="cuda", dtype=torch.float32).unsqueeze(1)
    assert base.numel() * 4 > 1 << 32
    rows = np.array([0, 1, 17, M // 2, 37449, 37450, M - 1])          # row 37449 holds byte 2^32
    qmm.lora_add(base, to_dev(x), A, B, to_dev(ids), out=base)
    got = to_host(base[torch.from_numpy(rows).cuda()])
    want, tol = _formula(np.tile(rows[:, None], (1, N)).astype(np.float32), x[rows], A64, B64, ids[rows])
    _check(got, want, tol)


def test_unaligned_column_range_is_refused():
    rng = np.random.default_rng(1)
    A, B, _, _ = _pool(rng, 2, 4, 8, 32, "f16")
    base = to_dev(np.zeros((2, 16), np.float32))
    with pytest.raises(qmm.QmmError, match="16-byte"):
        qmm.lora_add(base[:, 1:9], to_dev(np.zeros((2, 32), np.float32)), A, B, to_dev(np.zeros(2, np.int32)))


def test_streams_and_graphs_with_a_workspace_each():
    """Two captured calls that may overlap, each with its own workspace, replayed among eager work: every replay
    equals the eager result bit for bit."""
    import torch
    rng = np.random.default_rng(9)
    N, K, R, E = 300, 1024, 16, 4
    A, B, A64, B64 = _pool(rng, E, R, N, K, "bf16")
    calls = []
    for M in (3, 200):
        x, base, ids = _inputs(rng, M, N, K, E=E)
        d = [to_dev(v) for v in (base, x, ids)]
        ws = torch.empty(qmm.lora_workspace_bytes(M, R, K, E), dtype=torch.uint8, device="cuda")
        out = torch.zeros(M, N, device="cuda")
        want, tol = _formula(base, x, A64, B64, ids)
        eager = to_host(qmm.lora_add(d[0], d[1], A, B, d[2]))
        _check(eager, want, tol)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = qmm.lora_add(d[0], d[1], A, B, d[2], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert np.array_equal(to_host(other).view(np.uint32), eager.view(np.uint32))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            qmm.lora_add(d[0], d[1], A, B, d[2], out=out, workspace=ws)
        calls.append((g, (d, ws), out, eager, side))   # what a graph reads lives as long as it does
    for rep in range(4):
        for g, _, out, eager, side in calls:
            out.fill_(-1.0)
        torch.cuda.synchronize()
        for g, _, out, eager, side in calls:
            with torch.cuda.stream(side):
                g.replay()
        torch.cuda.synchronize()
        for g, _, out, eager, side in calls:
            assert np.array_equal(to_host(out).view(np.uint32), eager.view(np.uint32)), rep


def test_empty():
    import torch
    A, B = torch.zeros(2, 4, 32, device="cuda"), torch.zeros(2, 8, 4, device="cuda")
    x, ids = torch.zeros(0, 32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    assert qmm.lora_add(torch.zeros(0, 8, device="cuda"), x, A, B, ids).shape == (0, 8)
