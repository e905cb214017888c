"""cache_write and cache_read: the bytes of the pages and the numbers read back, both exact."""
import numpy as np
import pytest
import torch

from kv_reference import DIMS, TYPES, Batch, Cache, decode, encode, qmm, to_host

pytestmark = pytest.mark.gpu


def host_write(cache, batch_rows, lens, table, k, v):
    at = 0
    for b, n in enumerate(batch_rows):
        for i in range(n):
            pos = lens[b] - n + i
            page = table[b, pos // cache.page] if 0 <= pos < table.shape[1] * cache.page else -1
            if 0 <= page < cache.pages:
                cache.put(page, pos % cache.page, 0, k[at + i])
                cache.put(page, pos % cache.page, 1, v[at + i])
        at += n


def rows_of(rng, T, heads, D, kind):
    """Numbers of very different sizes, ties, zeros, blocks of one sign."""
    x = rng.standard_normal((2, T, heads, D)).astype(np.float32)
    x *= np.exp2(rng.integers(-12, 12, (2, T, heads, D // 32, 1)).astype(np.float32)).repeat(32, -1).reshape(x.shape)
    x[rng.random(x.shape) < 0.02] *= 8
    x[rng.random(x.shape) < 0.05] = 0
    x.reshape(-1, 32)[::7] = np.round(x.reshape(-1, 32)[::7])  # ties in magnitude, codes between two steps
    x.reshape(-1, 32)[3::11] = 0
    t = torch.from_numpy(x).to(TYPES[kind])
    return t, t.float().numpy()


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", DIMS)
@pytest.mark.parametrize("lens,rows,heads,page", [([1], [1], 1, 16), ([5, 40, 17], [5, 33, 0], 3, 16),
                                                  ([70, 64, 65, 130], [1, 1, 1, 1], 8, 64), ([200, 9], [150, 2], 5, 128),
                                                  ([3], [3], 17, 1024)])
def test_bytes_and_numbers(lens, rows, heads, page, D, kind):
    print(lens, rows, heads, page, D, kind, flush=True)
    rng = np.random.default_rng([10, D, page])
    b = Batch(rng, [0] * len(lens), [0] * len(lens), heads, D, page, width=max(-(-n // page) for n in lens) + 1,
              spare=sum(-(-n // page) for n in lens) + 3)
    order, at = rng.permutation(b.cache.pages), 0
    for i, n in enumerate(lens):
        m = -(-n // page)
        b.table[i, :m] = order[at:at + m]
        at += m
    T = sum(rows)
    dev, host = rows_of(rng, T, heads, D, kind)
    cache = b.cache.to_dev()
    table, ln = torch.from_numpy(b.table).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    one = all(n == 1 for n in rows)
    starts = None if one else torch.tensor(np.concatenate(([0], np.cumsum(rows))), dtype=torch.int32).cuda()
    host_write(b.cache, rows, lens, b.table, host[0], host[1])
    qmm.cache_write(cache, dev[0].cuda(), dev[1].cuda(), table, ln, starts)
    assert np.array_equal(to_host(cache).reshape(b.cache.bytes().shape), b.cache.bytes())
    for out in ("f32", "f16", "bf16"):
        k, v = qmm.cache_read(cache, T, table, ln, starts, dtype=TYPES[out])
        for x, got in zip(host, (k, v)):
            want = torch.from_numpy(decode(*encode(x)).reshape(x.shape)).to(TYPES[out])
            assert torch.equal(got.cpu(), want)


def test_matches_the_weight_encoder():
    """The numbers are those of the library's own Q4_0 blocks."""
    rng = np.random.default_rng(11)
    heads, D, T, page = 4, 128, 32, 32
    _, host = rows_of(rng, T, heads, D, "f32")
    cache = qmm.cache_new(2, heads, D, page=page)
    table, lens = torch.tensor([[1]], dtype=torch.int32).cuda(), torch.tensor([T], dtype=torch.int32).cuda()
    starts = torch.tensor([0, T], dtype=torch.int32).cuda()
    k = torch.from_numpy(host[0]).cuda()
    qmm.cache_write(cache, k, k, table, lens, starts)
    got, same = qmm.cache_read(cache, T, table, lens, starts)
    w = qmm.quantize_weights(k.view(T, heads * D), "q4_0")
    want = qmm.embed_rows("q4_0", w, torch.arange(T, dtype=torch.int32, device="cuda"), T, heads * D)
    assert torch.equal(got.view(T, -1), want) and torch.equal(same, got)


def test_what_is_not_a_number():
    """Infinities, NaN and scales past fp16 make their block NaN and no other; scales below fp16 make it 0."""
    heads, D = 1, 64
    x = np.random.default_rng(12).standard_normal((8, heads, D)).astype(np.float32)
    x[0, 0, 3] = np.inf
    x[1, 0, 40] = -np.inf
    x[2, 0, 31] = np.nan
    x[3, 0, 32] = 8 * 65520.0      # d rounds to infinity
    x[4, 0, 32] = 8 * 65519.0      # and this one not
    x[5, 0, :32] *= 1e-9           # d is 0 in fp16
    x[6, 0, :32] = 1e-40           # subnormal
    x[7, 0, :] = 0.0
    cache = qmm.cache_new(1, heads, D, page=16)
    table, lens = torch.tensor([[0]], dtype=torch.int32).cuda(), torch.tensor([8], dtype=torch.int32).cuda()
    starts = torch.tensor([0, 8], dtype=torch.int32).cuda()
    v = np.zeros_like(x)
    qmm.cache_write(cache, torch.from_numpy(x).cuda(), torch.from_numpy(v).cuda(), table, lens, starts)
    k, zero = (to_host(t) for t in qmm.cache_read(cache, 8, table, lens, starts))
    want = decode(*encode(x)).reshape(x.shape)
    assert np.array_equal(k, want.astype(np.float32), equal_nan=True) and not zero.any()
    assert np.isnan(want).reshape(8, 2, 32).any(-1).tolist() == [[True, False], [False, True], [True, False], [False, True],
                                                               [False, False], [False, False], [False, False], [False, False]]
    assert not k[5, 0, :32].any() and not k[6, 0, :32].any()


def test_rows_and_pages_that_are_not_there():
    """Rows of no sequence, positions below 0, pages outside the pool: nothing is written for them, they read as NaN, and
    all else is as it was."""
    heads, D, page, T = 2, 64, 16, 40
    rng = np.random.default_rng(13)
    _, host = rows_of(rng, T, heads, D, "f32")
    c = Cache(5, heads, D, page)
    table = np.array([[0, 7, 1], [-1, 2, 3], [4, -5, 2**31 - 1]], np.int32)
    lens = np.array([36, 20, 3], np.int32)
    starts = np.array([2, 22, 30, 36], np.int32)   # rows 0, 1 and 36 .. 39 are nobody's; sequence 2 has 6 rows, 3 entries
    cache = c.to_dev()
    table_d, lens_d, starts_d = (torch.from_numpy(a).cuda() for a in (table, lens, starts))
    kd, vd = (torch.from_numpy(h).cuda() for h in host)
    qmm.cache_write(cache, kd, vd, table_d, lens_d, starts_d)
    host_write(c, np.diff(starts), lens, table, host[0][2:], host[1][2:])
    assert np.array_equal(to_host(cache).reshape(c.bytes().shape), c.bytes())
    got = to_host(qmm.cache_read(cache, T, table_d, lens_d, starts_d)[0])
    at = 2
    for b, n in enumerate(np.diff(starts)):
        for i in range(n):
            pos = lens[b] - n + i
            there = pos >= 0 and 0 <= table[b, pos // page] < 5
            assert np.isnan(got[at]).all() != there, (b, i)
            at += 1


@pytest.mark.parametrize("starts", [[0, -5, 100, 3], [9, 4, 2, 1], [2**31 - 1, -2**31, 5, 5], [50, 60, 70, 80]])
@pytest.mark.parametrize("lens", [[5, 5, 5], [-7, 2**31 - 1, -2**31]])
def test_arrays_that_make_no_sense(starts, lens):
    """Whatever starts and lens hold, nothing outside the arrays is touched: the pool's neighbours keep their bytes."""
    heads, D, page, T = 2, 64, 16, 12
    pool = torch.full((3 * 2 * heads * page * 36 + 512,), 77, dtype=torch.uint8, device="cuda")
    cache = pool[256:-256].view(3, 2, heads, page, 36)
    table = torch.tensor([[0, 1], [2, 9], [-1, 0]], dtype=torch.int32).cuda()
    ln, st = torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(starts, dtype=torch.int32).cuda()
    k = torch.randn(T, heads, D, device="cuda")
    qmm.cache_write(cache, k, k, table, ln, st)
    a, b = qmm.cache_read(cache, T, table, ln, st)
    out = qmm.cache_attention(torch.randn(T, 4, D, device="cuda"), cache, table, ln, st,
                              mass=torch.zeros(3, heads, 32, device="cuda"))
    torch.cuda.synchronize()
    assert (pool[:256] == 77).all() and (pool[-256:] == 77).all() and a.shape == b.shape and out.shape == (T, 4, D)


@pytest.mark.parametrize("B", [63, 64, 65, 700, 5000])
def test_many_sequences(B):
    """The search for a row's sequence takes more than one step; empty sequences among them."""
    rng = np.random.default_rng(B)
    rows = rng.integers(0, 3, B)
    rows[rng.random(B) < 0.3] = 0
    rows[-1] = 1
    T, page = int(rows.sum()), 16
    table = torch.arange(B, dtype=torch.int32).view(B, 1).cuda()
    lens = torch.from_numpy((rows + 2).astype(np.int32)).cuda()
    starts = torch.from_numpy(np.concatenate(([0], np.cumsum(rows))).astype(np.int32)).cuda()
    k = torch.from_numpy(rng.integers(-7, 8, (T, 1, 64)).astype(np.float32))
    k.view(T, 2, 32)[..., 0] = -8
    cache = torch.zeros(B, 2, 1, page, 36, dtype=torch.uint8, device="cuda")
    qmm.cache_write(cache, k.cuda(), -k.cuda(), table, lens, starts)
    a, b = qmm.cache_read(cache, T, table, lens, starts)
    assert torch.equal(a.cpu(), k) and torch.equal(b.cpu(), torch.from_numpy(decode(*encode(-k.numpy())).reshape(T, 1, 64)).float())


def test_strides_stream_graph_and_growth():
    """Rows from column ranges; a captured step appends at the lengths that its buffers hold when it is replayed."""
    heads, D, page, B, steps = 2, 96, 16, 3, 20
    rng = np.random.default_rng(14)
    wide = torch.from_numpy(rng.standard_normal((B, 5 * heads * D)).astype(np.float32)).cuda()
    k, v = (wide[:, i * heads * D:(i + 1) * heads * D].unflatten(1, (heads, D)) for i in (1, 3))
    cache = torch.zeros(8, 2, heads, page, D * 9 // 16, dtype=torch.uint8, device="cuda")
    want = torch.zeros_like(cache)
    table = torch.tensor([[3, 0], [6, 1], [2, 7]], dtype=torch.int32).cuda()
    lens = torch.tensor([1, 1, 1], dtype=torch.int32).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qmm.cache_write(cache, k, v, table, lens, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    qmm.cache_write(want, k.contiguous(), v.contiguous(), table, lens)
    assert torch.equal(cache, want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        qmm.cache_write(cache, k, v, table, lens)
    for i in range(2, steps):
        wide.copy_(torch.randn(wide.shape, device="cuda"))
        lens.fill_(i)
        torch.cuda.synchronize()
        g.replay()
        qmm.cache_write(want, k, v, table, lens)
        torch.cuda.synchronize()
        assert torch.equal(cache, want), i


def test_pool_past_4_gib():
    heads, D, page = 8, 128, 256
    pages = (5 << 30) // (2 * heads * page * 72)
    cache = torch.zeros(pages, 2, heads, page, 72, dtype=torch.uint8, device="cuda")
    assert cache.numel() > 1 << 32
    table = torch.tensor([[pages - 1], [0]], dtype=torch.int32).cuda()
    lens = torch.tensor([256, 7], dtype=torch.int32).cuda()
    k = torch.randn(2, heads, D, device="cuda")
    qmm.cache_write(cache, k, -k, table, lens)
    a, b = qmm.cache_read(cache, 2, table, lens)
    x = k.cpu().numpy()
    assert torch.equal(a.cpu(), torch.from_numpy(decode(*encode(x)).reshape(x.shape)).float())
    assert torch.equal(b.cpu(), torch.from_numpy(decode(*encode(-x)).reshape(x.shape)).float())
