"""cache_attention's kernel for long runs of rows over contexts of many steps: 64 entries a step, twelve steps and more one
after another in one split, so that its rings wrap several times; and what 16-bit calls of long runs return as lse and mass.
The reference is attention in 64 bits over the numbers that the cache holds, formed for whole heads at a time."""
import numpy as np
import pytest
import torch

from kv_reference import DIMS, TYPES, Batch, decode, qmm, seen, to_host, tolerance
from test_gpu_cache_attention import queries

pytestmark = pytest.mark.gpu

# Rows of a sequence and cache head that the kernel takes begin above 256 in 16 bits and 768 in fp32; heads up to 192 and
# 128.  The splits are those that fill 256 workgroups over the tiles of 256 rows and the heads: none with these heads.
RUN = {"f32": (1100, 64), "f16": (300, 128), "bf16": (300, 128)}


def entries(batch, b, part):
    """[len, heads, D] in 64 bits."""
    p = np.arange(batch.lens[b])
    at = batch.table[b, p // batch.page], part, slice(None), p % batch.page
    h, q = batch.cache.h[at], batch.cache.q[at]
    return decode(h, q).reshape(len(p), batch.heads, batch.D)


def reference(batch, q, scale, **kw):
    """(out, lse, mass, slack) as kv_reference.attention gives them, head by head."""
    T, HQ, D = q.shape
    G = HQ // batch.heads
    out, lse = np.zeros((T, HQ, D)), np.full((T, HQ), -np.inf)
    terms, weight, total = np.zeros((T, HQ)), np.zeros((T, HQ, D)), np.zeros((T, HQ, D))
    mass = np.zeros((len(batch.lens), batch.heads, batch.width * batch.page))
    at = 0
    for b, n in enumerate(batch.rows):
        L = batch.lens[b]
        k, v = entries(batch, b, 0), entries(batch, b, 1)
        see = seen(n, L, kw.get("causal", True), kw.get("window", 0))
        some = see.any(1)
        for hq in range(HQ):
            h, x = hq // G, q[at:at + n, hq].astype(np.float64)
            s = np.where(see, x @ k[:, h].T * scale, -np.inf)
            m = np.where(some, s.max(1, initial=-np.inf), 0.0)[:, None]
            e = np.exp(s - m)
            p = e / np.where(some, e.sum(1), 1.0)[:, None]
            out[at:at + n, hq] = p @ v[:, h]
            lse[at:at + n, hq] = np.where(some, m[:, 0] + np.log(np.where(some, e.sum(1), 1.0)), -np.inf)
            terms[at:at + n, hq] = np.where(see, np.abs(x) @ np.abs(k[:, h]).T, 0.0).max(1, initial=0.0) * abs(scale)
            weight[at:at + n, hq] = p @ np.abs(v[:, h])
            total[at:at + n, hq] = see @ np.abs(v[:, h])
            mass[b, h, :L] += p.sum(0)
        at += n
    return out, lse, mass, (terms, weight, total)


def batch_of(rng, lens, rows, heads, D, page, width=None):
    """A batch whose entries are numbers of about one, all blocks at once."""
    b = Batch(rng, [0] * len(lens), [0] * len(lens), 1, D, page, width=1, spare=1)
    b.lens, b.rows, b.heads = list(lens), list(rows), heads
    need = [-(-n // page) for n in lens]
    b.width = width or max(need)
    order = rng.permutation(sum(need) + 2)
    b.table = np.full((len(lens), b.width), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        b.table[i, :n] = order[at:at + n]
        at += n
    c = b.cache
    c.pages, c.heads = len(order), heads
    shape = (c.pages, 2, heads, page)
    # scales of either sign from 1/16 to 3/8, as rows of the normal distribution leave them
    c.h = (rng.uniform(0.0625, 0.375, (*shape, D // 32)) * rng.choice([-1, 1], (*shape, D // 32))).astype(np.float16)
    c.q = rng.integers(0, 16, (*shape, D), dtype=np.uint8)
    for i, n in enumerate(lens):      # behind the length: anything
        for t in range(n, need[i] * page):
            c.h[b.table[i, t // page], :, :, t % page] = np.nan
    return b


def compare(kind, b, q, got, ref, keys_rounded):
    """out within its tolerance."""
    out, _, _, slack = ref
    tol, _ = tolerance(kind, b.D, max(b.lens), slack, out, rounded_keys=keys_rounded)
    err = np.abs(to_host(got).astype(np.float64) - out)
    assert (err <= tol).all(), (err.max(), (err - tol).max())


@pytest.mark.parametrize("kw", [{}, dict(window=500), dict(causal=False)])
@pytest.mark.parametrize("kind,D", [("f32", 64), ("f32", 96), ("f32", 128), ("f16", 64), ("f16", 96), ("bf16", 128),
                                    ("f16", 192), ("bf16", 192)])
def test_many_steps_of_one_split(kind, D, kw):
    n, heads = RUN[kind]
    rng = np.random.default_rng([60, D])
    b = batch_of(rng, [n + 471], [n], heads, D, 32)
    qd, q = queries(rng, n, heads, D, kind, 1.5)
    print(kind, D, kw, flush=True)
    ref = reference(b, q, D ** -0.5, **kw)
    cache, table, lens, st = b.dev()
    compare(kind, b, q, qmm.cache_attention(qd.cuda(), cache, table, lens, st, **kw), ref, True)


@pytest.mark.parametrize("kind,D", [("f32", 64), ("f32", 128), ("f16", 64), ("bf16", 96), ("bf16", 192)])
def test_many_steps_of_several_splits(kind, D):
    """One head, so that the entries are split to what 512 of them to a split allow; a short run and a token beside it."""
    n = RUN[kind][0] // 4 + 1
    rng = np.random.default_rng([61, D])
    b = batch_of(rng, [1700, 900, 77], [n, 3, 1], 1, D, 64)
    qd, q = queries(rng, b.T, 4, D, kind, 1.5)
    print(kind, D, flush=True)
    ref = reference(b, q, D ** -0.5)
    cache, table, lens, st = b.dev()
    compare(kind, b, q, qmm.cache_attention(qd.cuda(), cache, table, lens, st), ref, True)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_scales_that_grow_along_many_steps(kind):
    """Larger scales of keys and values every few steps: what is in LDS is decoded again, what was summed is rescaled."""
    n, heads = RUN[kind]
    D, L = 64, n + 500
    rng = np.random.default_rng(62)
    b = batch_of(rng, [L], [n], heads, D, 64)
    for p in range(L):
        page, t = b.table[0, p // 64], p % 64
        b.cache.h[page, 0, :, t] *= np.float16(2.0 ** (p // 190 - 4))
        b.cache.h[page, 1, :, t] *= np.float16(2.0 ** (p // 130))
    qd, q = queries(rng, n, heads, D, kind, 1.5)
    print(kind, flush=True)
    ref = reference(b, q, D ** -0.5)
    cache, table, lens, st = b.dev()
    compare(kind, b, q, qmm.cache_attention(qd.cuda(), cache, table, lens, st), ref, True)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", DIMS)
def test_sums_of_long_runs(D, kind):
    """lse and mass of long runs over many steps: fp32 results of scores from keys that are not rounded, 16-bit calls'
    too, in whichever kernel.

    A weight is off by its score's error and the lse's (ds each, three roundings of the exponent's size and of 2^x: 2^-22
    times 2 + |lse|), by what two fp16 pieces leave of the keys (2^-22 of the sum of magnitudes) beside ds, relative to itself, and by
    fp32 sums of up to 2 + rows numbers; a weight below 2^-126 is 0."""
    n, group = RUN[kind][0] // 4 + 1, 4
    rng = np.random.default_rng([63, D])
    b = batch_of(rng, [n + 600, 300, 77], [n, 9, 1], 2, D, 32)
    qd, q = queries(rng, b.T, 2 * group, D, kind, 1.5)
    print(D, kind, flush=True)
    ref = reference(b, q, D ** -0.5)
    out_ref, lse_ref, mass_ref, slack = ref
    cache, table, lens, st = b.dev()
    mass = torch.zeros(mass_ref.shape, device="cuda")
    got, lse = qmm.cache_attention(qd.cuda(), cache, table, lens, st, lse=True, mass=mass)
    compare(kind, b, q, got, ref, False)
    ds = tolerance(kind, D, max(b.lens), slack, out_ref)[1]
    off = ds + 2.0 ** -22 * (2 + np.abs(lse_ref))
    assert (np.abs(to_host(lse) - lse_ref) <= off * 1.01).all()
    per, rows = 2 * (off + 2.0 ** -22 * slack[0]).max(), n * group + 2
    assert (np.abs(to_host(mass) - mass_ref) <= (per + rows * 2.0 ** -24) * mass_ref + rows * 2.0 ** -126).all()
    # each of the two alone gives the same bits
    only = torch.zeros_like(mass)
    assert torch.equal(got, qmm.cache_attention(qd.cuda(), cache, table, lens, st, mass=only)) and torch.equal(mass, only)
    again, alone = qmm.cache_attention(qd.cuda(), cache, table, lens, st, lse=True)
    assert torch.equal(got, again) and torch.equal(lse, alone)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("ask", ["out", "lse", "mass"])
def test_long_runs_in_a_graph(ask, kind):
    """Long and short runs captured and replayed with other lengths and starts, between eager calls; out alone, so that
    16-bit calls too reach the kernel of long runs, and with lse or mass."""
    rng = np.random.default_rng(64)
    n, heads, group, D = (1100 if kind == "f32" else 300) // 16 + 20, 2, 16, 64
    b = batch_of(rng, [512] * 4, [0] * 4, heads, D, 32)
    cache, table, lens, starts = b.dev()
    q = torch.from_numpy(rng.standard_normal((n, heads * group, D)).astype(np.float32)).to(TYPES[kind]).cuda()
    out = torch.zeros_like(q)
    masses = [torch.zeros(4, heads, 512, device="cuda") if ask == "mass" else None for _ in range(2)]

    def step(m):
        got = qmm.cache_attention(q, cache, table, lens, starts, mass=m, out=out, lse=ask == "lse")
        return [t.clone() for t in (got if ask == "lse" else (got,))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(None if masses[0] is None else masses[0].clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step(masses[0])
    run = n - 15
    for rows, length in (((1, 1, 1, 1), (5, 80, 512, 33)), ((run, 1, 10, 1), (500, 80, 256, 33)), ((0, n, 0, 0), (7, 512, 1, 0)),
                         ((2, run, 0, 9), (20, 300, 100, 9)), ((run, 1, 10, 1), (500, 80, 256, 33))):
        lens.copy_(torch.tensor(length, dtype=torch.int32))
        starts.copy_(torch.tensor(np.concatenate(([0], np.cumsum(rows))), dtype=torch.int32))
        used = sum(rows)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in got]
        want = step(masses[1])
        torch.cuda.synchronize()
        print(ask, kind, rows, flush=True)
        for a, w in zip(replayed, want):
            assert torch.equal(a[:used], w[:used]) and torch.isfinite(a[:used].float()).any()
        if ask == "mass":
            assert torch.equal(masses[0], masses[1]) and masses[0].any()


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
def test_a_sequence_alone_and_beside_others(kind):
    """The bits of a sequence's rows do not depend on the others of the call where they are in as many splits: tables of
    128 entries are not split, and of 512 long runs are not and short ones are in four."""
    rng = np.random.default_rng(65)
    n, heads, group, D = RUN[kind][0] // 8 + 2, 2, 8, 128
    for capacity, rows in ((128, [1, 4, 128, 1, 20]), (512, [1, n, 9, n + 3, 0])):
        b = batch_of(rng, [min(capacity, r + 90) for r in rows], rows, heads, D, 32, width=capacity // 32)
        qd, _ = queries(rng, b.T, heads * group, D, kind)
        cache, table, lens, st = b.dev()
        for ask in (False, True):
            print(kind, capacity, ask, flush=True)
            got = qmm.cache_attention(qd.cuda(), cache, table, lens, st, lse=ask)
            at = 0
            for i, r in enumerate(rows):
                if r:
                    one = qmm.cache_attention(qd[at:at + r].cuda(), cache, table[i:i + 1].clone(), lens[i:i + 1].clone(),
                                              torch.tensor([0, r], dtype=torch.int32).cuda(), lse=ask)
                    for a, w in zip(one if ask else (one,), got if ask else (got,)):
                        assert torch.equal(a, w[at:at + r]), (i, r)
                at += r


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("group,heads,width", [(16, 1, 1500), (16, 3, 300), (33, 2, 500)])
def test_same_bits_of_split_runs_of_16_bits(group, heads, width, kind):
    """Long runs in several splits, out alone: the same bits again, on another stream and into a given out."""
    rng = np.random.default_rng([66, group])
    n = 300 // group + 1
    b = batch_of(rng, [n + 1200, 90, 3], [n, 7, 1], heads, 64, 32, width=width)
    qd, q = queries(rng, b.T, heads * group, 64, kind)
    cache, table, lens, st = b.dev()
    print(group, heads, width, kind, flush=True)
    first = qmm.cache_attention(qd.cuda(), cache, table, lens, st)
    compare(kind, b, q, first, reference(b, q, 64 ** -0.5), True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = qmm.cache_attention(qd.cuda(), cache, table, lens, st, stream=side)
    out = torch.full_like(first, 7.0)
    qmm.cache_attention(qd.cuda(), cache, table, lens, st, out=out)
    torch.cuda.synchronize()
    assert torch.equal(first, again) and torch.equal(first, out)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("B", [3, 300])
@pytest.mark.parametrize("order", ["down", "beyond", "again"])
def test_starts_that_make_no_sense_in_16_bits(order, B, kind):
    """As the test of that name of fp32 and mass: any starts and lens, out alone, which the kernel of long runs forms."""
    rng = np.random.default_rng(67)
    T, W, page, group = 400, 3, 16, 16
    starts = {"down": np.linspace(T, 0, B + 1), "beyond": rng.integers(-2**31, 2**31, B + 1),
              "again": np.arange(B + 1) % 2 * T}[order].astype(np.int32)
    lens = rng.choice(np.array([-5, 0, 30, 48, 1000, 2**31 - 1], np.int64), B).astype(np.int32)
    cache = qmm.cache_new(20, 2, 64, page)
    cache.zero_()
    table = torch.from_numpy(rng.integers(-2, 22, (B, W)).astype(np.int32)).cuda()
    s, n = torch.from_numpy(starts).cuda(), torch.from_numpy(lens).cuda()
    q = torch.ones(T, 2 * group, 64, dtype=TYPES[kind], device="cuda")
    need = qmm.cache_attention_workspace_bytes(q, 2, B, W, page, True)
    room = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    wide = torch.full((T + 8, 2 * group, 64), 7.0, dtype=TYPES[kind], device="cuda")
    print(order, B, kind, flush=True)
    qmm.cache_attention(q, cache, table, n, s, out=wide[4:T + 4], workspace=room[:need])
    torch.cuda.synchronize()
    assert (room[need:] == 0x5A).all() and (wide[:4] == 7).all() and (wide[T + 4:] == 7).all()


@pytest.mark.parametrize("kind,rows", [("f32", 767), ("f32", 768), ("f32", 769), ("f32", 1024), ("f32", 1025), ("f16", 256),
                                       ("f16", 257), ("bf16", 256), ("bf16", 257)])
def test_borders_of_who_takes_the_rows(kind, rows):
    rng = np.random.default_rng([68, rows])
    b = batch_of(rng, [rows + 33, rows - 1], [rows, rows - 1], 2, 128, 32)
    qd, q = queries(rng, b.T, 2, 128, kind)
    print(kind, rows, flush=True)
    ref = reference(b, q, 128 ** -0.5)
    cache, table, lens, st = b.dev()
    compare(kind, b, q, qmm.cache_attention(qd.cuda(), cache, table, lens, st), ref, kind == "bf16")
    got, lse = qmm.cache_attention(qd.cuda(), cache, table, lens, st, lse=True)
    compare(kind, b, q, got, ref, False)
    ds = tolerance(kind, 128, max(b.lens), ref[3], ref[0])[1]
    assert (np.abs(to_host(lse) - ref[1]) <= (ds + 2.0 ** -22 * (2 + np.abs(ref[1]))) * 1.01).all()
