"""logprobs against log-softmax in 64 bits; the top list exactly.

Tolerance.  u = 2^-24, z_i = scale (x_i - m) <= 0.  Each exponent carries up to
four roundings (the difference, the scale times log2 e (2), the product): 4u|z_i|
absolutely, and the base-2 exponential one unit (2u) of its own; S and T add
L = V / 256 + 64 roundings (a thread's terms, its rescales, the joins).  So
|d log S| <= u (L + 2 + 4 sum p|z|), and log p = (z_i - log S) rounds its parts
three more times: |d log p| <= u (8 (|z_i| + log S) + L + 8 + 4 W), W = sum p (|z|
+ z^2); the entropy is log S + |T|/S, both >= 0: u ((L + 8)(1 + H) + 8 W)."""
import numpy as np
import pytest

import bit_quantized_mat_quantize_amd as qmm
from gpu_helpers import to_dev, to_host

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = ["f32", "f16", "bf16"]


def _dev_type(x, type):
    """x rounded to `type` on the GPU, and the 64-bit values it then holds."""
    import torch
    d = to_dev(x.astype(np.float32)).to({"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[type])
    return d, to_host(d.double())


def _pack(allowed):
    """[rows, V] truth values -> int32 words."""
    rows, V = allowed.shape
    b = np.zeros((rows, (V + 31) // 32 * 32), np.uint8)
    b[:, :V] = allowed
    return np.packbits(b, axis=1, bitorder="little").view(np.int32).copy()


class Reference:
    def __init__(self, x, scale=1.0, allowed=None):
        x = np.array(x, np.float64)
        if allowed is not None:
            x[~np.broadcast_to(allowed, x.shape)] = -np.inf
        self.x, V = x, x.shape[1]
        scale = np.float64(np.float32(scale))
        m = x.max(1, keepdims=True)
        with np.errstate(invalid="ignore", divide="ignore"):
            z = np.where(x == -np.inf, -np.inf, scale * (x - np.where(np.isfinite(m), m, 0)))
            e = np.exp(z)
            S = e.sum(1, keepdims=True)
            p = np.where(S > 0, e / S, 0)
            zz = np.where(p > 0, z, 0)
            self.lp = np.where(S > 0, z - np.log(S), -np.inf)
            self.lp[self.lp < np.finfo(np.float32).min] = -np.inf      # what fp32 cannot hold
            self.H = np.where(S > 0, np.log(S) - (p * zz).sum(1, keepdims=True), 0)[:, 0]
            L = V / 256 + 64
            W = (p * (np.abs(zz) + zz * zz)).sum(1, keepdims=True)
            logS = np.where(S > 0, np.log(S), 0)
            fin = np.where(np.isfinite(z), np.abs(z), 0)
            self.tol = U * (8 * (fin + logS) + L + 8 + 4 * W)
            self.tol_H = (U * ((L + 8) * (1 + self.H[:, None]) + 8 * W))[:, 0]

    def top(self, k):
        order = np.argsort(-self.x, axis=1, kind="stable")[:, :k]
        ids = np.full((self.x.shape[0], k), -1, np.int64)
        ids[:, :order.shape[1]] = order
        rows = np.arange(len(ids))[:, None]
        ids[self.x[rows, ids] == -np.inf] = -1
        return ids

    def check(self, got, tokens=None, k=0, what=""):
        lp, H, ids, tl = (None if t is None else to_host(t) for t in got)
        assert (np.abs(H - self.H) <= self.tol_H).all(), (what, np.abs(H - self.H).max())
        rows = np.arange(len(self.x))[:, None]
        if tokens is not None:
            t = tokens.reshape(len(tokens), -1)
            self._close(lp.reshape(t.shape), self.lp[rows, t], self.tol[rows, t], what)
        if k:
            want = self.top(k)
            assert np.array_equal(ids, want), (what, np.argwhere(ids != want)[:5])
            none = want < 0
            self._close(np.where(none, 0, tl), np.where(none, 0, self.lp[rows, want]), self.tol[rows, want], what)
            assert (tl[none] == -np.inf).all(), what

    @staticmethod
    def _close(got, want, tol, what):
        inf = want == -np.inf
        assert np.array_equal(got == -np.inf, inf), what
        err = np.abs(got - np.where(inf, 0, want))[~inf]
        assert (err <= tol[~inf]).all(), (what, (err - tol[~inf]).max())


def _logits(rng, M, V):
    x = 2.0 * rng.standard_normal((M, V)) - 4.0
    for m in range(M):
        at = rng.integers(0, V, 5)
        x[m, at] = 4.0 + 5.0 * rng.standard_normal(5)
    return x


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("M,V,G,k,scale", [(1, 1, 1, 1, 1.0), (1, 2, 2, 5, 0.5), (3, 63, 1, 64, 1.0),
                                           (2, 257, 3, 20, 1.25), (1, 4097, 1, 5, 1.0), (7, 5000, 1, 40, 0.7),
                                           (1, 32000, 1, 20, 1.0), (1, 40961, 1, 33, 1.0), (2, 100003, 2, 64, 1.0), (40, 9001, 1, 8, 2.0),
                                           (1030, 333, 1, 3, 1.0), (1025, 4100, 2, 1, 1.0)])
def test_against_64_bits(M, V, G, k, scale, type):
    print(M, V, G, k, scale, type, flush=True)
    rng = np.random.default_rng(M * 7 + V)
    x, x64 = _dev_type(_logits(rng, M, V), type)
    tokens = rng.integers(0, V, (M, G)).astype(np.int32)
    got = qmm.logprobs(x, tokens=to_dev(tokens), k=k, scale=scale)
    Reference(x64, scale).check(got, tokens, k)
    lp, H, ids, tl = qmm.logprobs(x, tokens=to_dev(tokens[:, 0].copy()), scale=scale, entropy=False)
    assert H is None and ids is None and tl is None and lp.shape == (M,)
    assert np.array_equal(to_host(lp), to_host(got[0])[:, 0])


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("pad", [0, 1, 5, 8])
def test_row_strides(pad, type):
    """Rows that start at every alignment; NaN between the rows is not read."""
    import torch
    rng = np.random.default_rng(pad)
    M, V, k = 11, 2055, 9
    x, x64 = _dev_type(_logits(rng, M, V), type)
    wide = torch.full((M, V + pad), float("nan"), dtype=x.dtype, device="cuda")
    wide[:, :V] = x
    tokens = rng.integers(0, V, (M, 1)).astype(np.int32)
    Reference(x64).check(qmm.logprobs(wide[:, :V], tokens=to_dev(tokens), k=k), tokens, k)


@pytest.mark.parametrize("type", TYPES)
@pytest.mark.parametrize("M,V", [(1, 40), (3, 1000), (2, 20011), (2, 70003), (1030, 97)])
@pytest.mark.parametrize("shared", [False, True])
def test_masks(M, V, shared, type):
    """Masked places may hold anything; rows that allow one token or none; bits behind V do not matter."""
    rng = np.random.default_rng(V)
    k = 12
    allowed = rng.random((1 if shared else M, V)) < 0.3
    allowed[:, V // 2] = True
    if not shared and M > 1:
        allowed[-1] = np.arange(V) == V // 2
        allowed[0] = False
    x = _logits(rng, M, V)
    wild = ~np.broadcast_to(allowed, x.shape)
    x[wild] = rng.choice([np.nan, np.inf, -np.inf, 6e4, -6e4], wild.sum())
    d, x64 = _dev_type(x, type)
    words = _pack(allowed)
    if V % 32:
        words[:, -1] |= np.int32(-(1 << (V % 32))) if V % 32 < 31 else np.int32(-2**31)
    tokens = rng.integers(0, V, (M, 3)).astype(np.int32)
    tokens[:, 1] = V // 2
    mask = to_dev(words[0].copy() if shared and M > 2 else words)
    got = qmm.logprobs(d, tokens=to_dev(tokens), k=k, mask=mask)
    Reference(np.where(wild, 0, x64), 1.0, allowed).check(got, tokens, k)
    if not shared and M > 1:                    # the row that allows nothing
        assert (to_host(got[0])[0] == -np.inf).all() and to_host(got[1])[0] == 0
        assert (to_host(got[2])[0] == -1).all() and (to_host(got[3])[0] == -np.inf).all()


@pytest.mark.parametrize("M", [2, 1030])
@pytest.mark.parametrize("V", [900, 9000, 40000])
def test_ties_and_orders(M, V):
    """Equal logits (all of them, two values, 0 and -0), ascending and descending rows: ties go to the lowest
    index, and rows on which every logit enters the list come out right."""
    rng = np.random.default_rng(V)
    k = 33
    up = np.linspace(-3, 3, V)
    for name, row in (("constant", np.full(V, 1.5)), ("two values", rng.integers(0, 2, V).astype(float)),
                      ("zeros", np.where(rng.random(V) < 0.5, 0.0, -0.0)), ("ascending", up), ("descending", up[::-1]),
                      ("steps", np.floor(up * 10))):
        print(name, flush=True)
        x, x64 = _dev_type(np.tile(row, (M, 1)), "f32")
        tokens = np.full((M, 1), V - 1, np.int32)
        Reference(x64).check(qmm.logprobs(x, tokens=to_dev(tokens), k=k), tokens, k, name)


@pytest.mark.parametrize("V", [70, 5001, 50001])
def test_extreme_values(V):
    """Rows of the lowest finite number, of -inf, with one finite logit, with a range that overflows a difference."""
    rng = np.random.default_rng(V)
    low = np.float64(np.finfo(np.float32).min)
    rows = {"lowest": np.full(V, low), "lowest and one": np.where(np.arange(V) == 7, 2.0, low),
            "-inf": np.full(V, -np.inf), "-inf and one": np.where(np.arange(V) == 7, -3.0, -np.inf),
            "both ends": np.where(np.arange(V) % 2 == 0, low, -low), "far below": np.where(np.arange(V) == 3, 0.0, -1e4),
            "large": 1e4 + rng.standard_normal(V), "tiny": rng.standard_normal(V) * 1e-38}
    x, x64 = _dev_type(np.stack(list(rows.values())), "f32")
    tokens = np.tile(np.array([7, 0, 1], np.int32), (len(rows), 1))
    Reference(x64).check(qmm.logprobs(x, tokens=to_dev(tokens), k=4), tokens, 4)


@pytest.mark.parametrize("V", [70, 5001, 50001])
def test_nan_and_inf_poison_their_row_only(V):
    rng = np.random.default_rng(V)
    x = rng.standard_normal((4, V)).astype(np.float32)
    x[1, V // 2], x[2, V - 1] = np.nan, np.inf
    tokens = np.full((4, 1), 2, np.int32)
    lp, H, ids, tl = (to_host(t) for t in qmm.logprobs(to_dev(x), tokens=to_dev(tokens), k=5))
    for m in (1, 2):
        assert np.isnan(lp[m]).all() and np.isnan(H[m]) and np.isnan(tl[m]).all()
    assert ids[2, 0] == V - 1 and V // 2 not in ids[1]
    fine = [0, 3]
    ref = Reference(x[fine].astype(np.float64))
    assert np.array_equal(ids[fine], ref.top(5))
    assert (np.abs(H[fine] - ref.H) <= ref.tol_H).all()


def test_bad_tokens_give_nan():
    rng = np.random.default_rng(3)
    x, x64 = _dev_type(_logits(rng, 2, 300), "f32")
    tokens = np.array([[-1, 5, 300], [299, 2**31 - 1, -2**31]], np.int32)
    got = to_host(qmm.logprobs(x, tokens=to_dev(tokens))[0])
    good = (tokens >= 0) & (tokens < 300)
    assert np.isnan(got[~good]).all()
    ref = Reference(x64)
    m, g = np.nonzero(good)
    assert (np.abs(got[m, g] - ref.lp[m, tokens[m, g]]) <= ref.tol[m, tokens[m, g]]).all()


def test_logits_past_4_gib():
    """Rows that lie past 2^32 bytes; every row is the same one shifted, so its results are known."""
    import torch
    M, V, k = 9000, 120000, 4
    rng = np.random.default_rng(13)
    row, row64 = _dev_type(_logits(rng, 1, V), "f32")
    x = torch.empty(M, V, device="cuda")
    assert x.numel() * 4 > 1 << 32
    x.copy_(row.expand(M, V))
    at = np.array([0, 8946, 8947, 8948, M - 1])                        # row 8947 holds byte 2^32
    x[8947, 77], x[M - 1, V - 1] = 30.0, 31.0
    lp, H, ids, tl = qmm.logprobs(x, tokens=torch.full((M,), 77, dtype=torch.int32, device="cuda"), k=k)
    x64 = np.tile(row64, (len(at), 1))
    x64[2, 77], x64[4, V - 1] = 30.0, 31.0
    pick = torch.from_numpy(at).cuda()
    Reference(x64).check([t[pick] for t in (lp, H, ids, tl)], np.full((len(at), 1), 77), k)


def test_more_tokens_than_threads_and_empty():
    import torch
    rng = np.random.default_rng(4)
    x, x64 = _dev_type(_logits(rng, 2, 700), "bf16")
    tokens = rng.integers(0, 700, (2, 700)).astype(np.int32)
    Reference(x64).check(qmm.logprobs(x, tokens=to_dev(tokens)), tokens)
    lp, H, ids, tl = qmm.logprobs(torch.zeros(0, 700, device="cuda"), k=3)
    assert lp is None and H.shape == (0,) and ids.shape == (0, 3) and tl.shape == (0, 3)


def test_streams_and_graphs_with_a_workspace_each():
    """Split rows (a workspace) captured twice, replayed among eager work: every replay equals the eager result."""
    import torch
    rng = np.random.default_rng(5)
    side = torch.cuda.Stream()
    calls = []
    for M, V, k in ((1, 60000, 20), (5, 40000, 3)):
        x, x64 = _dev_type(_logits(rng, M, V), "f32")
        tokens = rng.integers(0, V, (M, 1)).astype(np.int32)
        dt = to_dev(tokens)
        ws = torch.empty(qmm.logprobs_workspace_bytes(M, V, k), dtype=torch.uint8, device="cuda")
        assert ws.numel() > 0
        eager = qmm.logprobs(x, tokens=dt, k=k)
        Reference(x64).check(eager, tokens, k)
        side.wait_stream(torch.cuda.current_stream())
        other = qmm.logprobs(x, tokens=dt, k=k, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for a, b in zip(eager, other):
            assert torch.equal(a, b)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            got = qmm.logprobs(x, tokens=dt, k=k, workspace=ws)
        calls.append((g, got, eager, (x, dt, ws)))     # what a graph reads lives as long as it does
    for rep in range(4):
        for g, got, eager, _ in calls:
            for t in got:
                t.fill_(7)
        torch.cuda.synchronize()
        for g, got, eager, _ in calls:
            with torch.cuda.stream(side):
                g.replay()
        torch.cuda.synchronize()
        for g, got, eager, _ in calls:
            for a, b in zip(got, eager):
                assert torch.equal(a, b), rep
