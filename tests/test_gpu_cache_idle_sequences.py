"""cache_write and cache_read where most sequences of a long batch's table have no rows: the rows' places, and that a call
does not take longer by the sequences that are passed over."""
import numpy as np
import pytest
import torch

from kv_reference import decode, encode, qmm

pytestmark = pytest.mark.gpu


def setup(B, busy, heads=1, D=64, page=64):
    """(cache, table, lens, starts, rows) of B sequences of which those of `busy` (sequence: rows) have any, all new."""
    rows = np.zeros(B, np.int64)
    for b, n in busy.items():
        rows[b] = n
    need = -(-rows // page)
    W = int(need.max())
    table = np.full((B, W), -1, np.int32)
    at = 0
    for b in busy:
        table[b, :need[b]] = np.arange(at, at + need[b])
        at += int(need[b])
    starts = np.concatenate(([0], np.cumsum(rows))).astype(np.int32)
    cache = torch.zeros(at, 2, heads, page, D * 9 // 16, dtype=torch.uint8, device="cuda")
    dev = [torch.from_numpy(a).cuda() for a in (table, rows.astype(np.int32), starts)]
    return cache, *dev, int(rows.sum())


@pytest.mark.parametrize("B,busy", [
    (600, {0: 8195, 599: 1}), (600, {3: 8190, 4: 1, 5: 1, 70: 2, 71: 1, 200: 1, 599: 9}), (65536, {1: 8193, 65535: 4}),
    (65536, {17: 4100, 16000: 1, 16001: 2, 40000: 4095, 65534: 1}), (300, {b: 28 + b % 5 for b in range(0, 300)}),
    (3000, {b: 1 + 90 * (b % 3) for b in range(7, 3000, 31)})])
def test_places(B, busy):
    cache, table, lens, starts, T = setup(B, busy)
    rng = np.random.default_rng(B + len(busy))
    k = rng.standard_normal((T, 1, 64)).astype(np.float32)
    print(B, len(busy), T, flush=True)
    assert T >= 8192 or B == 3000
    qmm.cache_write(cache, torch.from_numpy(k).cuda(), torch.from_numpy(-k).cuda(), table, lens, starts)
    got = qmm.cache_read(cache, T, table, lens, starts)
    for x, g in zip((k, -k), got):
        want = torch.from_numpy(decode(*encode(x)).reshape(x.shape)).float()
        assert torch.equal(g.cpu(), want)
    # and by the reader's one row each: entry i of every busy sequence
    for i in (0, max(busy.values()) - 1):
        one = qmm.cache_read(cache, B, table, torch.full_like(lens, i + 1))[0].cpu()
        for b, n in busy.items():
            if i < n:
                assert torch.equal(one[b], got[0][int(starts[b]) + i].cpu()), (b, i)


def least_us(f, calls=20, times=7):
    f()
    best = float("inf")
    for _ in range(times):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        for _ in range(calls):
            f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / calls * 1e3)
    return best


def test_sequences_that_are_passed_over_cost_nothing():
    """The same rows in a table of two sequences and of 65536, of which 65534 have none: a row's sequence is found in a
    number of reads that grows with the logarithm (one at a time, they took 240 times as long)."""
    took = []
    for B in (2, 65536):
        cache, table, lens, starts, T = setup(B, {0: 8195, B - 1: 1}, heads=8, D=128)
        k = torch.randn(T, 8, 128, device="cuda").bfloat16()
        took.append((least_us(lambda: qmm.cache_write(cache, k, k, table, lens, starts)),
                     least_us(lambda: qmm.cache_read(cache, T, table, lens, starts, dtype=torch.bfloat16))))
        print(B, took[-1], flush=True)
    assert took[1][0] < 10 * took[0][0] and took[1][1] < 10 * took[0][1]
