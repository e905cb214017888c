"""cache_attention with runs of rows that are long for their type (more than 256 query rows of a cache head in 16 bits,
1024 in fp32), and with many sequences: the reference and tolerances of test_gpu_cache_attention."""
import numpy as np
import pytest
import torch

from kv_reference import DIMS, TYPES, Batch, attention, qmm, to_host, tolerance
from test_gpu_cache_attention import check, queries

pytestmark = pytest.mark.gpu

GROUP = 16
TOKENS = {"f32": 70, "f16": 20, "bf16": 20}   # times GROUP: 1120 and 320 rows


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("kw", [{}, dict(window=13), dict(causal=False)])
def test_beside_short_ones(kw, D, kind):
    """A long run of rows, a short one, a single token, one of rows before position 0 and a sequence without rows."""
    rng = np.random.default_rng([40, D])
    n = TOKENS[kind]
    b = Batch(rng, [n + 37, 50, 19, n - 5, 12], [n, 5, 1, n, 0], 1, D, 16, width=9)
    qd, q = queries(rng, b.T, GROUP, D, kind)
    print(kw, D, kind, flush=True)
    check(kind, b, q, qd, **kw)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("group,heads,width", [(16, 1, 4000), (16, 3, 300), (5, 2, 40), (33, 2, 500)])
def test_splits(group, heads, width, kind):
    """Tables with room for more entries than there are, so that the entries are split, into up to all that fit."""
    rng = np.random.default_rng([41, group])
    n = (1100 if kind == "f32" else 300) // group + 1
    b = Batch(rng, [n + 200, 90, 3], [n, 7, 1], heads, 64, 32, width=width)
    qd, q = queries(rng, b.T, heads * group, 64, kind)
    print(group, heads, width, kind, flush=True)
    a = check(kind, b, q, qd)
    assert torch.equal(a, check(kind, b, q, qd, mass=False))


@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_two_tiles_and_edges(kind):
    """Rows one below, at and above the borders of tiles and of who takes them."""
    rng = np.random.default_rng(42)
    for rows in ((1024, 1025, 1279, 1280, 1281) if kind == "f32" else (256, 257, 511, 512, 513)):
        b = Batch(rng, [rows], [rows], 1, 64, 256)
        qd, q = queries(rng, b.T, 1, 64, kind)
        print(rows, kind, flush=True)
        check(kind, b, q, qd, window=40)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale", [3.0, -0.5, 0.0])
def test_peaked_and_flat_weights(scale, kind):
    rng = np.random.default_rng(43)
    n = TOKENS[kind]
    b = Batch(rng, [180], [n], 1, 128, 32)
    qd, q = queries(rng, b.T, GROUP, 128, kind, 2.0)
    print(scale, kind, flush=True)
    check(kind, b, q, qd, scale=scale)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("size", [2.0 ** -9, 1.0, 2.0 ** 12])
def test_magnitudes(size, kind):
    """Values and keys far from one, rising along the sequence; queries the other way."""
    rng = np.random.default_rng(44)
    n = TOKENS[kind]
    b = Batch(rng, [140], [n], 1, 64, 16, scale=size)
    b.cache.h[:] = b.cache.h * np.exp2(rng.integers(-2, 3, b.cache.h.shape)).astype(np.float16)
    for p in range(140):
        b.cache.h[b.table[0, p // 16], 1, :, p % 16] *= np.float16(2.0 ** (p // 40))
    qd, q = queries(rng, b.T, GROUP, 64, kind, 1.0 / size)
    print(size, kind, flush=True)
    check(kind, b, q, qd)


@pytest.mark.parametrize("kind", ["f32", "f16"])
def test_nan_reaches_those_that_see_it(kind):
    rng = np.random.default_rng(45)
    n, page, window = TOKENS[kind], 16, 30
    L = n + 50
    b = Batch(rng, [L], [n], 1, 64, page, spare=3)
    for t in range(L, b.width * page):
        b.cache.h[b.table[0, t // page], :, :, t % page] = rng.choice([np.nan, np.inf, 60000.0], (2, 1, 2))
    qd, q = queries(rng, b.T, GROUP, 64, kind)
    clean = {w: check(kind, b, q, qd, window=w) for w in (0, window)}
    pos = np.arange(L - n, L)
    for at, part in ((20, 1), (20, 0), (L - 2, 1), (L - 2, 0), (L - 20, 1)):
        pg = b.table[0, at // page]
        keep = b.cache.h[pg, part, 0, at % page].copy()
        b.cache.h[pg, part, 0, at % page, 1] = np.nan
        dev = b.dev()
        for w in (0, window):
            mass = torch.zeros(1, 1, b.width * page, device="cuda")
            got, lse = qmm.cache_attention(qd.cuda(), *dev, window=w, lse=True, mass=mass)
            sees = torch.from_numpy((pos >= at) & ((pos - at < w) if w else True))
            alone = qmm.cache_attention(qd.cuda(), *dev, window=w).cpu()
            assert torch.equal(torch.isnan(alone), sees[:, None, None].expand_as(alone))
            got, lse = got.cpu(), lse.cpu()
            print(kind, at, part, w, flush=True)
            assert torch.equal(torch.isnan(got), sees[:, None, None].expand_as(got))
            assert torch.equal(torch.isnan(lse), sees[:, None].expand_as(lse))
            ok = ~sees[:, None, None].expand_as(got)
            assert torch.allclose(got[ok].float(), clean[w].cpu()[ok].float(), atol=1e-3)
            # entries that a row of NaN sees get NaN, the others and what is behind the length do not
            hit = np.zeros(b.width * page, bool)
            for p in pos[sees.numpy()]:
                hit[max(0, p - w + 1) if w else 0:p + 1] = True
            assert np.array_equal(np.isnan(to_host(mass)[0, 0]), hit)
        b.cache.h[pg, part, 0, at % page] = keep


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_pages_and_queries_that_are_not_there(kind):
    rng = np.random.default_rng(46)
    n = TOKENS[kind]
    L = n + 30
    b = Batch(rng, [L, L], [n, n], 1, 96, 16)
    qd, q = queries(rng, b.T, GROUP, 96, kind)
    check(kind, b, q, qd)
    at = L // 32 * 16
    for bad in (-1, b.cache.pages, 2**31 - 1, -2**31):
        table = b.table.copy()
        table[1, at // 16] = bad
        cache, _, lens, st = b.dev()
        got = qmm.cache_attention(qd.cuda(), cache, torch.from_numpy(table).cuda(), lens, st).cpu()
        want = qmm.cache_attention(qd.cuda(), *b.dev()).cpu()
        pos = np.arange(L - n, L)
        nan = torch.from_numpy(np.concatenate((np.zeros(n, bool), pos >= at)))
        assert torch.isnan(got[nan]).all() and torch.equal(got[~nan], want[~nan])
    y = qd.clone()
    y[0, 1, 7], y[-1, 2, 90], y[n, 3, 0] = float("inf"), float("nan"), -float("inf")
    got, want = qmm.cache_attention(y.cuda(), *b.dev()).cpu(), qmm.cache_attention(qd.cuda(), *b.dev()).cpu()
    bad = torch.zeros(b.T, GROUP, dtype=torch.bool)
    bad[0, 1] = bad[-1, 2] = bad[n, 3] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("ask", ["lse", "mass", "both"])
def test_sums_of_16_bit_calls(ask, D, kind):
    """lse and mass are fp32 results: their scores come from keys that are not rounded (`rounded_keys` left out of the
    tolerance; a weight is off by its score's and the lse's error, relative to itself)."""
    rng = np.random.default_rng([51, D])
    b = Batch(rng, [60, 45, 30], [40, 3, 1], 1, D, 16)
    qd, q = queries(rng, b.T, GROUP, D, kind, 2.0)
    out_ref, lse_ref, mass_ref, slack = attention(b, q, D ** -0.5)
    ds = tolerance(kind, D, 60, slack, out_ref)[1]
    print(ask, D, kind, flush=True)
    cache, table, lens, st = b.dev()
    mass = torch.zeros(mass_ref.shape, device="cuda") if ask != "lse" else None
    got = qmm.cache_attention(qd.cuda(), cache, table, lens, st, lse=ask != "mass", mass=mass)
    off = ds + 2.0 ** -22 * (2 + np.abs(lse_ref))
    if ask != "mass":
        assert (np.abs(to_host(got[1]) - lse_ref) <= off * 1.01).all()
    if mass is not None:
        # fp32 queries' pieces are not needed, the keys' two hold 22 bits: 2^-22 of the sum of magnitudes beside ds
        per = 2 * (off + 2.0 ** -22 * slack[0]).max()
        n = b.T * GROUP + 2
        assert (np.abs(to_host(mass) - mass_ref) <= (per + n * 2.0 ** -24) * mass_ref + n * 2.0 ** -40).all()


@pytest.mark.parametrize("kind", ["f32", "f16"])
@pytest.mark.parametrize("B", [63, 65, 200, 256, 257, 700])
def test_many_sequences(B, kind):
    """Around the borders of how sequences are counted, one of them with a long run of rows, many with none."""
    rng = np.random.default_rng([47, B])
    rows = rng.choice([0, 0, 1, 1, 2, 5], B)
    rows[B // 2] = TOKENS[kind]
    lens = rows + rng.integers(0, 20, B)
    b = Batch(rng, lens.tolist(), rows.tolist(), 1, 64, 16)
    qd, q = queries(rng, b.T, GROUP, 64, kind)
    print(B, kind, flush=True)
    check(kind, b, q, qd)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("B", [3, 300])
@pytest.mark.parametrize("order", ["down", "beyond", "again"])
def test_starts_that_make_no_sense(order, B, kind):
    """Any starts and lens: nothing outside out, mass and the workspace is written, and the call ends."""
    rng = np.random.default_rng(48)
    T, W, page = 400, 3, 16
    starts = {"down": np.linspace(T, 0, B + 1), "beyond": rng.integers(-2**31, 2**31, B + 1),
              "again": np.arange(B + 1) % 2 * T}[order].astype(np.int32)
    lens = rng.choice(np.array([-5, 0, 30, 48, 1000, 2**31 - 1], np.int64), B).astype(np.int32)
    cache = qmm.cache_new(20, 2, 64, page)
    cache.zero_()
    table = torch.from_numpy(rng.integers(-2, 22, (B, W)).astype(np.int32)).cuda()
    s, n = torch.from_numpy(starts).cuda(), torch.from_numpy(lens).cuda()
    q = torch.ones(T, 2 * GROUP, 64, dtype=TYPES[kind], device="cuda")
    need = qmm.cache_attention_workspace_bytes(q, 2, B, W, page, True, True)
    room = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    wide = torch.full((T + 8, 2 * GROUP, 64), 7.0, dtype=TYPES[kind], device="cuda")
    mass = torch.zeros(B + 1, 2, W * page, device="cuda")
    print(order, B, kind, flush=True)
    qmm.cache_attention(q, cache, table, n, s, out=wide[4:T + 4], mass=mass[:B], workspace=room[:need])
    torch.cuda.synchronize()
    assert (room[need:] == 0x5A).all() and (wide[:4] == 7).all() and (wide[T + 4:] == 7).all() and not mass[B].any()


def test_same_bits_in_a_graph():
    """Long and short runs, captured and replayed with other lengths and starts between eager calls."""
    rng = np.random.default_rng(49)
    T, heads, D, page, W = 60, 2, 128, 32, 8
    cache = torch.randint(0, 255, (40, 2, heads, page, 72), dtype=torch.uint8, device="cuda")
    cache.view(40, 2, heads, -1)[..., page * D // 2:] = 0x2C     # scales of 2^-4 or so
    table = torch.from_numpy(rng.permutation(40)[:32].reshape(4, 8).astype(np.int32)).cuda()
    lens, starts = torch.zeros(4, dtype=torch.int32).cuda(), torch.zeros(5, dtype=torch.int32).cuda()
    q = torch.randn(T, heads * GROUP, D, device="cuda").bfloat16()
    mass = torch.zeros(4, heads, W * page, device="cuda")
    out = torch.zeros_like(q)

    def step(m):
        return qmm.cache_attention(q, cache, table, lens, starts, mass=m, out=out).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(mass.clone())
    torch.cuda.synchronize()
    inside = mass.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = step(inside)
    for rows, n in (((1, 1, 1, 1), (5, 80, 256, 33)), ((40, 1, 18, 1), (200, 80, 256, 33)), ((0, 60, 0, 0), (7, 90, 1, 0)),
                    ((20, 20, 20, 0), (20, 256, 100, 3))):
        lens.copy_(torch.tensor(n, dtype=torch.int32))
        starts.copy_(torch.tensor(np.concatenate(([0], np.cumsum(rows))), dtype=torch.int32))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        replayed, m = got.clone(), inside.clone()
        out.zero_()
        want = step(mass)
        torch.cuda.synchronize()
        assert torch.equal(replayed, want) and torch.equal(m, mass), rows
