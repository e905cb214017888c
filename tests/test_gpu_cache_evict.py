"""cache_evict against a sort of every entry; all results exact."""
import numpy as np
import pytest
import torch

from kv_reference import DIMS, Batch, evict, qmm, to_host

pytestmark = pytest.mark.gpu


def weights(rng, B, heads, n, how):
    m = rng.random((B, heads, n)).astype(np.float32) ** 4 * 8
    if how == "ties":
        m = np.round(m * 2) / 2
    elif how == "equal":
        m[:] = 1.5
    elif how == "odd":
        m = rng.choice(np.array([0.0, -0.0, -1.0, np.inf, -np.inf, np.nan, 1e-40, 3.0, 3.0000002], np.float32), m.shape)
    return m.astype(np.float32)


def run(b, mass, budget, recent, to=None, table=None):
    cache, tab, lens, _ = b.dev()
    to_d = None if to is None else torch.from_numpy(to).cuda()
    before = cache.clone()
    n, m, ids = qmm.cache_evict(cache, tab if table is None else table, lens, torch.from_numpy(mass).cuda(), budget, recent, to=to_d)
    return cache, before, to_host(n), to_host(m), to_host(ids)


def check(b, mass, budget, recent, to=None):
    want_ids, want_mass, want_lens = evict(b.lens, mass, budget, recent)
    cache, before, n, m, ids = run(b, mass, budget, recent, to)
    assert np.array_equal(ids, want_ids) and np.array_equal(n, want_lens)
    assert np.array_equal(m[..., :budget], want_mass, equal_nan=True) and not m[..., budget:].any()
    at = b.table if to is None else to
    # every entry's bytes, through the scales and codes of a host copy
    for s in range(len(b.lens)):
        for h in range(b.heads):
            for i in range(want_lens[s]):
                p = want_ids[s, h, i]
                src, dst = b.table[s, p // b.page], at[s, i // b.page]
                yield (s, h, i, src, p % b.page, dst, i % b.page)
    got = to_host(cache)
    hc = b.cache
    h0, q0 = hc.h.copy(), hc.q.copy()
    for s in range(len(b.lens)):
        for h in range(b.heads):
            for i in range(want_lens[s]):
                p = want_ids[s, h, i]
                src, dst = b.table[s, p // b.page], at[s, i // b.page]
                hc.h[dst, :, h, i % b.page], hc.q[dst, :, h, i % b.page] = h0[src, :, h, p % b.page], q0[src, :, h, p % b.page]
    want = hc.bytes()
    hc.h, hc.q = h0, q0
    if to is None:  # what is behind the entries that stay is nobody's
        got, want = got.copy().reshape(want.shape), want
        mask = entry_mask(b, want_lens)
        assert np.array_equal(got[mask], want[mask])
    else:
        assert np.array_equal(got.reshape(want.shape), want)


def entry_mask(b, lens):
    """The bytes of the first entries of each sequence, and of all pages that are no sequence's."""
    from kv_reference import Cache
    c = Cache(b.cache.pages, b.heads, b.D, b.page)
    c.q[:] = 15
    c.h.view(np.uint16)[:] = 0xFFFF
    for s, L in enumerate(b.lens):
        for p in range(lens[s], L):
            page = b.table[s, p // b.page]
            c.q[page, :, :, p % b.page] = 0
            c.h.view(np.uint16)[page, :, :, p % b.page] = 0
    return c.bytes() == 255


def checked(*a, **kw):
    for _ in check(*a, **kw):
        pass


@pytest.mark.parametrize("own", [True, False])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("lens,budget,recent,heads,page", [([40, 17, 0, 100], 24, 5, 2, 16), ([130], 64, 64, 1, 32),
                                                           ([70, 70, 71], 70, 0, 3, 64), ([300, 5], 1, 0, 2, 16),
                                                           ([33, 200], 150, 149, 1, 128)])
def test_what_stays(lens, budget, recent, heads, page, D, own):
    print(lens, budget, recent, heads, page, D, own, flush=True)
    rng = np.random.default_rng([40, D, page])
    need = -(-budget // page)
    b = Batch(rng, lens, [0] * len(lens), heads, D, page, width=max(-(-max(lens) // page), need),
              spare=2 + (0 if own else need * len(lens)))
    for s, n in enumerate(lens):   # pages for the budget where a sequence has fewer
        b.table[s, -(-n // page):] = -1
    to = None
    if not own:
        free = np.setdiff1d(np.arange(b.cache.pages), b.table[b.table >= 0])
        to = rng.permutation(free)[:need * len(lens)].reshape(len(lens), need).astype(np.int32)
    checked(b, weights(rng, len(lens), heads, b.width * page, "plain"), budget, recent, to)


@pytest.mark.parametrize("how", ["ties", "equal", "odd"])
@pytest.mark.parametrize("recent", [0, 30])
def test_ties_and_odd_weights(how, recent):
    rng = np.random.default_rng(41)
    b = Batch(rng, [150, 90, 64], [0] * 3, 2, 64, 16)
    print(how, recent, flush=True)
    checked(b, weights(rng, 3, 2, b.width * 16, how), 60, recent)


@pytest.mark.parametrize("how", ["plain", "ties", "equal"])
@pytest.mark.parametrize("L,budget,recent", [(5000, 3000, 100), (9001, 8999, 0), (20000, 1, 1), (70000, 33333, 77)])
def test_long(L, budget, recent, how):
    """More entries than the selection has threads, chunks that depend on one another; the order by torch's sort."""
    print(L, budget, recent, how, flush=True)
    rng = np.random.default_rng(L)
    page, heads = 256, 2
    W = -(-L // page)
    cache = torch.randint(0, 256, (W, 2, heads, page, 36), dtype=torch.uint8, device="cuda")
    cache.view(W, 2, heads, -1)[..., page * 32:] &= 0x3B   # finite scales
    table = torch.from_numpy(rng.permutation(W).astype(np.int32)).view(1, W).cuda()
    lens = torch.tensor([L], dtype=torch.int32).cuda()
    mass = torch.from_numpy(weights(rng, 1, heads, W * page, how)).cuda()
    whole = torch.tensor([0, L], dtype=torch.int32).cuda()
    k, v = qmm.cache_read(cache, L, table, lens, whole)
    n, m, ids = qmm.cache_evict(cache, table, lens, mass, budget, recent)
    order = mass[..., :L - recent].sort(dim=-1, descending=True, stable=True).indices[..., :budget - recent]
    want = torch.cat((order.sort(-1).values, torch.arange(L - recent, L, device="cuda").expand(1, heads, recent)), -1)
    assert torch.equal(ids.long(), want) and int(n) == budget
    assert torch.equal(m[..., :budget], mass.gather(2, want)) and not m[..., budget:].any()
    kept = torch.tensor([0, budget], dtype=torch.int32).cuda()
    k2, v2 = qmm.cache_read(cache, budget, table, n, kept)
    for h in range(heads):
        assert torch.equal(k2[:, h], k[want[0, h], h]) and torch.equal(v2[:, h], v[want[0, h], h])


def test_pages_that_are_not_there():
    """Entries of a missing page come out NaN; nothing is written for a missing page; all else is as it should be."""
    rng = np.random.default_rng(42)
    b = Batch(rng, [64], [0], 1, 64, 16, spare=3)
    mass = weights(rng, 1, 1, 64, "plain")
    free = np.setdiff1d(np.arange(b.cache.pages), b.table)
    to = free[:3].reshape(1, 3).astype(np.int32)
    table = b.table.copy()
    table[0, 1] = 2**31 - 1
    to[0, 2] = -7
    cache, _, lens, _ = b.dev()
    before = to_host(cache)
    n, m, ids = qmm.cache_evict(cache, torch.from_numpy(table).cuda(), lens, torch.from_numpy(mass).cuda(), 40, 8,
                                to=torch.from_numpy(to).cuda())
    ids = to_host(ids)[0, 0]
    k, v = qmm.cache_read(cache, 40, torch.from_numpy(to).cuda(), n, torch.tensor([0, 40], dtype=torch.int32).cuda())
    k, v = to_host(k), to_host(v)
    for i, p in enumerate(ids):
        if i >= 32 or 16 <= p < 32:
            assert np.isnan(k[i]).all() and np.isnan(v[i]).all(), i
        else:
            assert np.array_equal(k[i], b.cache.get(b.table[0, p // 16], p % 16, 0).astype(np.float32)), i
            assert np.array_equal(v[i], b.cache.get(b.table[0, p // 16], p % 16, 1).astype(np.float32)), i
    others = np.setdiff1d(np.arange(b.cache.pages), to[0, :2])
    assert np.array_equal(to_host(cache)[others], before[others])


def test_again_and_in_a_graph():
    """Evict, append, evict: a captured eviction in place gives what the eager one does, replay after replay."""
    rng = np.random.default_rng(43)
    heads, D, page, B, budget = 3, 128, 16, 4, 40
    W = 6
    start = torch.randint(0, 120, (B * W, 2, heads, page, 72), dtype=torch.uint8, device="cuda")
    table = torch.from_numpy(rng.permutation(B * W).reshape(B, W).astype(np.int32)).cuda()
    cache, eager = start.clone(), start.clone()
    lens = torch.tensor([90, 41, 40, 7], dtype=torch.int32).cuda()
    mass = torch.rand(B, heads, W * page, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = qmm.cache_evict(cache, table, lens, mass, budget, 6)
    for rep in range(4):
        lens.copy_(torch.from_numpy(rng.integers(0, W * page + 1, B).astype(np.int32)))
        mass.copy_(torch.rand(mass.shape, device="cuda"))
        torch.cuda.synchronize()
        g.replay()
        want = qmm.cache_evict(eager, table, lens, mass, budget, 6)
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y), rep
        assert torch.equal(cache, eager), rep
