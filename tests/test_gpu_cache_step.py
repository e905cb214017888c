"""A layer's steps with the cache as a program runs them: the quantized product of queries, keys and values, rope over
its columns, cache_write, cache_attention with mass, the product behind, and cache_evict once a sequence passed its
budget.  Each operator's result is held against its definition on the operands it was given."""
import numpy as np
import pytest
import torch

from kv_reference import TYPES, Batch, Cache, attention, encode, evict, qmm, to_host, tolerance
from test_gpu_rope import check as check_rope, reference as rope_reference

pytestmark = pytest.mark.gpu

HEADS, GROUP, D, PAGE, K = 2, 4, 64, 16, 256
N = (HEADS * GROUP + 2 * HEADS) * D
TABLE, POOL = 6, 20          # pages of a sequence and of the cache


class Layer:
    def __init__(self, kind, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.kind = kind
        self.qkv = qmm.quantize_weights(torch.randn(N, K, generator=g, device="cuda") / 16, "q4_K")
        self.back = qmm.quantize_weights(torch.randn(K, HEADS * GROUP * D, generator=g, device="cuda") / 16, "q4_K")
        self.cache = qmm.cache_new(POOL, HEADS, D, PAGE)
        self.cache.zero_()
        self.table = torch.from_numpy(np.random.default_rng(seed).permutation(POOL)[:3 * TABLE].reshape(3, TABLE).astype(np.int32)).cuda()
        self.lens = torch.zeros(3, dtype=torch.int32).cuda()
        self.mass = torch.zeros(3, HEADS, TABLE * PAGE, device="cuda")

    def step(self, x, positions, starts):
        """out [T, K], and what the operators made of it."""
        T = x.shape[0]
        rows = qmm.mul_mat("q4_K", self.qkv, qmm.quantize_row_q8(x, "q8_K"), T, N, K).to(TYPES[self.kind]).view(T, -1, D)
        turned = rows.clone()
        qk = turned[:, :HEADS * (GROUP + 1)]
        qmm.rope(qk, positions, out=qk)
        q, k, v = turned.split((HEADS * GROUP, HEADS, HEADS), 1)
        qmm.cache_write(self.cache, k, v, self.table, self.lens, starts)
        out, lse = qmm.cache_attention(q, self.cache, self.table, self.lens, starts, mass=self.mass, lse=True)
        y = qmm.mul_mat("q4_K", self.back, qmm.quantize_row_q8(out.reshape(T, -1).float(), "q8_K"), T, K, HEADS * GROUP * D)
        return y, rows, turned, out


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_steps_against_the_definitions(kind):
    rng = np.random.default_rng(60)
    layer = Layer(kind, 61)
    host = Cache(POOL, HEADS, D, PAGE)
    host.h[:], host.q[:] = 0, 0   # the bytes of an empty cache
    table, lens = layer.table.cpu().numpy(), np.zeros(3, int)
    total = np.zeros((3, HEADS, TABLE * PAGE))
    place = np.zeros(3, int)     # positions given so far: eviction frees entries, not positions
    budget, recent, evicted, off = 40, 6, 0, 0.0
    for n in ((50, 3, 17), (1, 1, 1), (1, 30, 1), (2, 1, 40), (1, 1, 1)):
        lens += n
        place += n
        layer.lens.copy_(torch.from_numpy(lens.astype(np.int32)))
        starts = torch.from_numpy(np.concatenate(([0], np.cumsum(n))).astype(np.int32)).cuda()
        pos = np.concatenate([np.arange(p - m, p) for p, m in zip(place, n)]).astype(np.int32)
        x = torch.randn(sum(n), K, device="cuda")
        _, rows, turned, out = layer.step(x, torch.from_numpy(pos).cuda(), starts)
        print(kind, n, lens, flush=True)
        raw, t = to_host(rows).astype(np.float64), to_host(turned)
        want, slack = rope_reference(raw[:, :HEADS * (GROUP + 1)], pos, D, "half", 10000.0)
        check_rope(kind, turned[:, :HEADS * (GROUP + 1)], want, slack)
        assert np.array_equal(t[:, HEADS * (GROUP + 1):], raw[:, HEADS * (GROUP + 1):])
        # the entries that the rows became
        at = 0
        for b, m in enumerate(n):
            for i in range(m):
                p = lens[b] - m + i
                for part, first in ((0, HEADS * GROUP), (1, HEADS * (GROUP + 1))):
                    host.put(table[b, p // PAGE], p % PAGE, part, t[at + i, first:first + HEADS])
            at += m
        assert np.array_equal(to_host(layer.cache).reshape(POOL, 2, HEADS, -1), host.bytes())
        batch = Batch.__new__(Batch)
        batch.lens, batch.rows, batch.heads, batch.D, batch.page = lens.tolist(), list(n), HEADS, D, PAGE
        batch.width, batch.table, batch.cache = TABLE, table, host
        ref, lse_ref, mass, room = attention(batch, t[:, :HEADS * GROUP], D ** -0.5)
        tol, ds = tolerance(kind, D, max(lens), room, ref, rounded_keys=True)
        assert (np.abs(to_host(out) - ref) <= tol).all()
        total += mass
        got = to_host(layer.mass)
        off = max(off, 2 * (ds.max() + 2.0 ** -21 * (2 + np.abs(lse_ref).max())))
        assert (np.abs(got - total) <= (off + 4 * 2.0 ** -24 * sum(n) * GROUP) * (total + 1)).all()
        if (lens > budget).any():
            ids, kept, left = evict(lens.tolist(), got, budget, recent)
            after, m, moved = qmm.cache_evict(layer.cache, layer.table, layer.lens, layer.mass, budget, recent)
            assert np.array_equal(to_host(moved), ids) and np.array_equal(to_host(m)[..., :budget], kept)
            assert np.array_equal(to_host(after), left)
            h, c = host.h.copy(), host.q.copy()
            for b in range(3):
                for hd in range(HEADS):
                    for i, p in enumerate(ids[b, hd][: left[b]]):
                        src, dst = table[b, p // PAGE], table[b, i // PAGE]
                        host.h[dst, :, hd, i % PAGE], host.q[dst, :, hd, i % PAGE] = h[src, :, hd, p % PAGE], c[src, :, hd, p % PAGE]
            lens[:] = left
            layer.mass.copy_(m)
            total = to_host(m).astype(np.float64)
            at = torch.from_numpy(np.concatenate(([0], np.cumsum(left))).astype(np.int32)).cuda()
            for part, got in enumerate(qmm.cache_read(layer.cache, int(left.sum()), layer.table, after, at)):
                want = np.concatenate([np.stack([host.get(table[b, p // PAGE], p % PAGE, part) for p in range(left[b])])
                                       for b in range(3)])
                assert np.array_equal(to_host(got), want.astype(np.float32))
            layer.cache.copy_(host.to_dev())   # what is behind the entries that stay is nobody's
            evicted += 1
    assert evicted >= 2


@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_a_captured_step(kind):
    """The whole step of single tokens, eviction included, captured once and replayed while lengths grow to the budget
    and past it, against eager steps of a second layer."""
    a, b = Layer(kind, 70), Layer(kind, 70)
    x, pos = torch.randn(3, K, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    budget, recent = 24, 4

    def step(layer):
        y = layer.step(x, pos, None)[0]
        lens, mass, ids = qmm.cache_evict(layer.cache, layer.table, layer.lens, layer.mass, budget, recent)
        layer.lens.copy_(lens)
        layer.mass.copy_(mass)
        layer.lens.add_(1)
        return y, ids

    for layer in (a, b):
        layer.lens.copy_(torch.tensor([1, 20, 9], dtype=torch.int32))
    start = [t.clone() for t in (a.cache, a.mass, a.lens)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a)
    torch.cuda.synchronize()
    for t, s in zip((a.cache, a.mass, a.lens), start):
        t.copy_(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        y, ids = step(a)
    for i in range(12):
        x.copy_(torch.randn(3, K, device="cuda"))
        pos.fill_(i)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, ids, a.lens, a.mass, a.cache)]
        want = [*step(b), b.lens, b.mass, b.cache]
        torch.cuda.synchronize()
        for u, w in zip(got, want):
            assert torch.equal(u, w), i
    assert (a.lens == torch.tensor([13, 25, 21], dtype=torch.int32).cuda()).all()


def test_versions_and_recorded_gradients():
    """What is written counts as changed: a backward pass that saved it refuses.  Nothing is written through a tensor
    that records its gradient."""
    layer = Layer("f32", 80)
    layer.lens.fill_(1)
    x = torch.randn(3, HEADS, D, device="cuda")
    q = torch.randn(3, HEADS * GROUP, D, device="cuda")
    out, pos = torch.zeros_like(q), torch.zeros(3, dtype=torch.int32, device="cuda")
    before = [t._version for t in (layer.cache, layer.mass, out, q)]
    qmm.cache_write(layer.cache, x, x, layer.table, layer.lens)
    assert layer.cache._version > before[0]
    qmm.cache_attention(q, layer.cache, layer.table, layer.lens, mass=layer.mass, out=out)
    assert layer.mass._version > before[1] and out._version > before[2]
    qmm.rope(q, pos, out=q)
    assert q._version > before[3]
    at = layer.cache._version
    qmm.cache_evict(layer.cache, layer.table, layer.lens, layer.mass, 4)
    assert layer.cache._version > at
    g = q.clone().requires_grad_()
    for call in (lambda: qmm.rope(g, pos), lambda: qmm.cache_attention(g, layer.cache, layer.table, layer.lens),
                 lambda: qmm.cache_write(layer.cache, g[:, :HEADS], x, layer.table, layer.lens)):
        with pytest.raises(ValueError, match="no backward"):
            call()
    with torch.no_grad():
        qmm.rope(g, pos)
        qmm.cache_attention(g, layer.cache, layer.table, layer.lens)
    with torch.inference_mode():
        qmm.cache_attention(q, layer.cache, layer.table, layer.lens)
    torch.cuda.synchronize()
