"""cache_attention against attention in 64 bits over the numbers that the cache holds; the tolerance is derived in
kv_reference.tolerance."""
import numpy as np
import pytest
import torch

from kv_reference import DIMS, TYPES, Batch, attention, qmm, to_host, tolerance

pytestmark = pytest.mark.gpu


def queries(rng, T, heads, D, kind, scale=1.0):
    t = torch.from_numpy((rng.standard_normal((T, heads, D)) * scale).astype(np.float32)).to(TYPES[kind])
    return t, t.float().numpy()


def check(kind, batch, q, qd, dev=None, starts="own", mass=True, **kw):
    """out, lse and mass of one call against the reference; returns out."""
    cache, table, lens, st = dev or batch.dev()
    if starts is None:
        st = None
    scale = kw.pop("scale", batch.D ** -0.5)
    out_ref, lse_ref, mass_ref, slack = attention(batch, q, scale, **kw)
    tol, ds = tolerance(kind, batch.D, max(batch.lens, default=0), slack, out_ref, rounded_keys=True)
    m0 = torch.rand(mass_ref.shape, device="cuda") if mass else None
    m1 = None if m0 is None else m0.clone()
    got, lse = qmm.cache_attention(qd.cuda(), cache, table, lens, st, scale=scale, lse=True, mass=m1, **kw)
    alone = qmm.cache_attention(qd.cuda(), cache, table, lens, st, scale=scale, **kw)   # may round keys in 16 bits
    for out in (to_host(alone).astype(np.float64), to_host(got).astype(np.float64)):
        err = np.abs(out - out_ref)
        assert np.isfinite(out).all() and (err <= tol).all(), (err.max(), (err - tol).max())
    l = to_host(lse).astype(np.float64)
    none = np.isneginf(lse_ref)
    assert np.array_equal(np.isneginf(l), none) and not out[none].any()
    # a sum of weights off by ds each, its logarithm, two roundings
    assert (np.abs(l[~none] - lse_ref[~none]) <= (ds + 2.0 ** -22 * (2 + np.abs(lse_ref)))[~none] * 1.01).all()
    if mass:
        # every weight off by its score's and the lse's error, and fp32 sums of all rows on top of what was there
        add = to_host(m1).astype(np.float64) - to_host(m0)
        off = 2 * (ds.max(initial=0.0) + 2.0 ** -21 * (2 + np.abs(lse_ref[~none]).max(initial=0.0)))
        n = batch.T * q.shape[1] + 2
        assert (np.abs(add - mass_ref) <= off * mass_ref + n * 2.0 ** -24 * (mass_ref + 1)).all()
    return got


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("lens,heads,group,page", [([1], 1, 1, 16), ([7, 16, 33], 2, 4, 16), ([300, 1, 129], 3, 7, 32),
                                                   ([65], 1, 16, 64), ([50, 20], 2, 24, 1024)])
def test_one_row_each(lens, heads, group, page, D, kind):
    print(lens, heads, group, page, D, kind, flush=True)
    rng = np.random.default_rng([20, D, page])
    b = Batch(rng, lens, [1] * len(lens), heads, D, page)
    qd, q = queries(rng, b.T, heads * group, D, kind, 1.5)
    one = check(kind, b, q, qd, starts=None)
    assert torch.equal(one, check(kind, b, q, qd, mass=False).to(one.dtype)) or len(lens) > 1


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("kw", [{}, dict(window=1), dict(window=20), dict(causal=False)])
@pytest.mark.parametrize("lens,rows,heads,group,D,page", [
    ([40, 0, 17, 90], [40, 0, 3, 1], 2, 2, 64, 16), ([130, 3, 61], [65, 3, 61], 1, 5, 128, 32),
    ([5, 20, 4], [9, 20, 2], 2, 3, 96, 64), ([150], [150], 1, 1, 256, 16), ([33, 200], [16, 17], 3, 1, 192, 128)])
def test_ragged_rows(lens, rows, heads, group, D, page, kw, kind):
    """Prompts, drafts and single tokens side by side; sequences without rows or entries, rows before position 0."""
    print(lens, rows, heads, group, D, page, kw, kind, flush=True)
    rng = np.random.default_rng([21, D, page])
    b = Batch(rng, lens, rows, heads, D, page, width=-(-max(lens) // page) + 2)
    qd, q = queries(rng, b.T, heads * group, D, kind)
    check(kind, b, q, qd, **kw)


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("rows,group", [(1, 8), (5, 2), (300, 2)])
def test_long_contexts_split(rows, group, kind):
    """Tables with room for far more entries than there are: many splits, most of them empty."""
    rng = np.random.default_rng(22)
    b = Batch(rng, [1500, 700], [rows, rows], 2, 64, 16, width=1000)
    qd, q = queries(rng, b.T, 2 * group, 64, kind, 2.0)
    print(rows, group, kind, flush=True)
    check(kind, b, q, qd)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 90])
@pytest.mark.parametrize("scale", [3.0, -0.5, 0.0, 1e-6])
def test_peaked_and_flat_weights(scale, rows, kind):
    """Scores of hundreds, of either sign, and none at all."""
    rng = np.random.default_rng(23)
    b = Batch(rng, [180], [rows], 2, 128, 32)
    qd, q = queries(rng, b.T, 4, 128, kind, 2.0)
    print(scale, rows, kind, flush=True)
    check(kind, b, q, qd, scale=scale)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [1, 70])
@pytest.mark.parametrize("size", [2.0 ** -9, 1.0, 2.0 ** 12])
def test_magnitudes(size, rows, kind):
    """Values and keys far from one, rising along the sequence, and scales of zero; queries the other way."""
    rng = np.random.default_rng(24)
    b = Batch(rng, [140], [rows], 1, 64, 16, scale=size)
    b.cache.h[:] = b.cache.h * np.exp2(rng.integers(-2, 3, b.cache.h.shape)).astype(np.float16)
    b.cache.h[0, :, :, 3] = 0
    for p in range(140):   # later values are larger
        page = b.table[0, p // 16]
        b.cache.h[page, 1, :, p % 16] *= np.float16(2.0 ** (p // 40))
    qd, q = queries(rng, b.T, 3, 64, kind, 1.0 / size)
    print(size, rows, kind, flush=True)
    check(kind, b, q, qd)


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("rows", [1, 3, 100])
def test_nan_reaches_those_that_see_it(rows, kind):
    """A NaN scale of a key or value makes NaN of the rows that see the entry, and of no other; entries behind the
    length, outside the window or on pages of others may hold anything."""
    rng = np.random.default_rng(25)
    L, page, window = 120, 16, 50
    b = Batch(rng, [L], [rows], 2, 64, page, spare=3)
    for t in range(L, b.width * page):
        b.cache.h[b.table[0, t // page], :, :, t % page] = rng.choice([np.nan, np.inf, 60000.0], (2, 2, 2))
    qd, q = queries(rng, b.T, 4, 64, kind)
    print(rows, kind, flush=True)
    clean = {w: check(kind, b, q, qd, window=w) for w in (0, window)}
    # entry 20: out of the window of the last rows; entry L - 2: seen by the last two
    for at, part, head in ((20, 1, 0), (20, 0, 1), (L - 2, 1, 1), (L - 2, 0, 0)):
        pg = b.table[0, at // page]
        keep = b.cache.h[pg, part, head, at % page].copy()
        b.cache.h[pg, part, head, at % page, 1] = np.nan
        dev = b.dev()
        for w in (0, window):
            got, lse = qmm.cache_attention(qd.cuda(), *dev, window=w, lse=True)
            pos = np.arange(L - rows, L)
            sees = (pos >= at) & ((pos - at < w) if w else True)
            bad = torch.zeros(got.shape[:2], dtype=torch.bool)
            bad[torch.from_numpy(sees), 2 * head:2 * head + 2] = True
            got, lse = got.cpu(), lse.cpu()
            assert torch.equal(torch.isnan(got), bad.unsqueeze(2).expand_as(got)), (at, part, head, w)
            assert torch.equal(torch.isnan(lse), bad)
            ok = ~bad.unsqueeze(2).expand_as(got)
            assert torch.allclose(got[ok].float(), clean[w].cpu()[ok].float(), atol=1e-3)
        b.cache.h[pg, part, head, at % page] = keep


@pytest.mark.parametrize("rows", [1, 60])
def test_pages_outside_the_pool(rows):
    rng = np.random.default_rng(26)
    b = Batch(rng, [100, 100], [rows, rows], 1, 64, 16)
    qd, q = queries(rng, b.T, 2, 64, "f32")
    want = check("f32", b, q, qd).cpu()
    for bad in (-1, b.cache.pages, 2**31 - 1, -2**31):
        table = b.table.copy()
        table[1, 4] = bad           # entries 64 .. 79 of sequence 1
        cache, _, lens, st = b.dev()
        got = qmm.cache_attention(qd.cuda(), cache, torch.from_numpy(table).cuda(), lens, st).cpu()
        pos = np.arange(100 - rows, 100)
        nan = torch.from_numpy(np.concatenate((np.zeros(rows, bool), pos >= 64)))
        assert torch.isnan(got[nan]).all() and torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("rows", [1, 40])
def test_queries_that_are_not_numbers(rows):
    rng = np.random.default_rng(27)
    b = Batch(rng, [90], [rows], 1, 128, 16)
    qd, q = queries(rng, b.T, 4, 128, "f32")
    want = check("f32", b, q, qd).cpu()
    y = qd.clone()
    y[0, 1, 7], y[-1, 2, 100], y[-1, 3, 0] = float("inf"), float("nan"), -float("inf")
    got = qmm.cache_attention(y.cuda(), *b.dev()).cpu()
    bad = torch.zeros(rows, 4, dtype=torch.bool)
    bad[0, 1] = bad[-1, 2] = bad[-1, 3] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


def test_rows_of_no_sequence_and_strides():
    """out and q as column ranges of one matrix; rows before, between and behind the sequences keep what they hold."""
    rng = np.random.default_rng(28)
    heads, group, D = 2, 3, 64
    b = Batch(rng, [50, 30], [4, 20], heads, D, 16)
    n = heads * group * D
    wide = torch.randn(30, 3 * n + 64, device="cuda")
    q, out = wide[:, :n].unflatten(1, (heads * group, D)), wide[:, n + 64:2 * n + 64].unflatten(1, (heads * group, D))
    cache, table, lens, _ = b.dev()
    before = wide.clone()
    starts = torch.tensor([3, 7, 27], dtype=torch.int32).cuda()
    assert qmm.cache_attention(q, cache, table, lens, starts, out=out) is out
    want = attention(b, q[3:27].cpu().numpy(), D ** -0.5)[0]
    assert np.abs(to_host(out)[3:27] - want).max() < 1e-4
    out[3:27] = before[3:27, n + 64:2 * n + 64].unflatten(1, (heads * group, D))
    assert torch.equal(wide, before)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_same_bits_every_time_and_beside_others(kind):
    """A call again, on another stream, among others; a sequence alone in its tables' width gives the bits it gives in a
    batch with the same number of splits."""
    rng = np.random.default_rng(29)
    b = Batch(rng, [400, 77, 260], [1, 30, 200], 2, 128, 32)
    qd, _ = queries(rng, b.T, 8, 128, kind)
    dev, q = b.dev(), qd.cuda()
    ref = qmm.cache_attention(q, *dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [qmm.cache_attention(q, *dev, stream=s) for s in (side, None, side, None)]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, ref)


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("ragged", [False, True])
def test_graph_that_grows(kind, ragged):
    """A captured step (write, attend with mass) replayed while lengths, tables and queries change, with eager work
    between; two graphs that share no workspace do not disturb one another."""
    rng = np.random.default_rng(30)
    heads, group, D, page, B = 2, 4, 64, 16, 3
    cache = torch.zeros(40, 2, heads, page, 36, dtype=torch.uint8, device="cuda")
    table = torch.from_numpy(rng.permutation(39)[:36].reshape(3, 12).astype(np.int32)).cuda()
    lens = torch.tensor([1, 1, 1], dtype=torch.int32).cuda()
    starts = torch.arange(4, dtype=torch.int32).cuda() if ragged else None
    k, v = (torch.randn(B, heads, D, device="cuda").to(TYPES[kind]) for _ in range(2))
    q = torch.randn(B, heads * group, D, device="cuda").to(TYPES[kind])
    mass = torch.zeros(B, heads, 192, device="cuda")

    def step(c, m):
        qmm.cache_write(c, k, v, table, lens, starts)
        return qmm.cache_attention(q, c, table, lens, starts, mass=m)

    eager_cache, eager_mass = cache.clone(), mass.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache.clone(), mass.clone())
    torch.cuda.synchronize()
    graphs, outs, state = [], [], []
    for _ in range(2):
        state.append((cache.clone(), mass.clone()))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(step(*state[-1]))
        graphs.append(g)
    for i in range(1, 190, 27):
        lens.copy_(torch.tensor([i, min(190, i + 2), 1 + i // 2], dtype=torch.int32))
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, device="cuda"))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        want = step(eager_cache, eager_mass)
        torch.cuda.synchronize()
        for o, (c, m) in zip(outs, state):
            assert torch.equal(o, want) and torch.equal(c, eager_cache) and torch.equal(m, eager_mass), i


def test_empty_calls():
    cache = qmm.cache_new(2, 2, 64, page=16)
    i32 = dict(dtype=torch.int32, device="cuda")
    table, lens, starts = torch.zeros(3, 1, **i32), torch.zeros(3, **i32), torch.zeros(4, **i32)
    assert qmm.cache_attention(torch.zeros(0, 4, 64, device="cuda"), cache, table, lens, starts).shape == (0, 4, 64)
    assert qmm.cache_attention(torch.zeros(0, 4, 64, device="cuda"), cache, table[:0], lens[:0]).shape == (0, 4, 64)
    out, lse = qmm.cache_attention(torch.ones(3, 4, 64, device="cuda"), cache, table, lens, lse=True)
    assert not out.any() and torch.isneginf(lse).all()


def test_pool_past_4_gib():
    """Pages whose bytes lie past 2^32."""
    rng = np.random.default_rng(31)
    heads, D, page = 8, 128, 256
    b = Batch(rng, [300], [1], heads, D, page, spare=0)
    pages = (5 << 30) // (2 * heads * page * 72)
    cache = torch.zeros(pages, 2, heads, page, 72, dtype=torch.uint8, device="cuda")
    small = b.cache.to_dev()
    table = b.table.copy()
    for i, p in enumerate((pages - 1, pages - 3)):
        cache[p] = small[b.table[0, i]]
        table[0, i] = p
    qd, q = queries(rng, 1, 16, D, "f32")
    _, _, lens, _ = b.dev()
    got = qmm.cache_attention(qd.cuda(), cache, torch.from_numpy(table).cuda(), lens)
    assert torch.equal(got, qmm.cache_attention(qd.cuda(), small, *b.dev()[1:3]))
    assert np.abs(to_host(got) - attention(b, q, D ** -0.5)[0]).max() < 1e-4
