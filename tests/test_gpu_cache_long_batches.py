"""cache_write and cache_read of thousands of rows, where a workgroup has eight of them and long outputs go past the
caches.  Blocks of whole numbers with a -8 first have d = 1, so that every number comes back as it was."""
import numpy as np
import pytest
import torch

from kv_reference import TYPES, qmm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("heads,D,page,rows", [(8, 128, 64, (8300, 0, 5, 1)), (8, 128, 16, (1, 4001, 99, 1)), (3, 96, 128, (9000, 1, 700, 3)),
                                               (1, 256, 16, (16389, 7, 0, 2)), (5, 64, 1024, (3000, 2999, 3001, 1))])
def test_numbers_come_back(heads, D, page, rows, kind):
    print(heads, D, page, rows, kind, flush=True)
    g = torch.Generator().manual_seed(D + heads)
    T, before = sum(rows), 11     # rows of no sequence before the first and behind the last
    k, v = (torch.randint(-7, 8, (T + 2 * before, heads, D), generator=g).float() for _ in range(2))
    for x in (k, v):
        x.view(-1, 32)[:, 0] = -8
    lens = [n + 3 if n else 0 for n in rows]
    W = max(-(-n // page) for n in lens)
    pages = 4 * W + 1
    table = torch.randperm(pages, generator=g)[:4 * W].int().view(4, W).cuda()
    starts = torch.tensor(np.concatenate(([0], np.cumsum(rows))) + before, dtype=torch.int32).cuda()
    ln = torch.tensor(lens, dtype=torch.int32).cuda()
    cache = torch.full((pages, 2, heads, page, D * 9 // 16), 0x55, dtype=torch.uint8, device="cuda")
    kd, vd = k.to(TYPES[kind]).cuda(), v.to(TYPES[kind]).cuda()
    qmm.cache_write(cache, kd, vd, table, ln, starts)
    for out in ("f32", "f16", "bf16"):
        a, b = qmm.cache_read(cache, T + 2 * before, table, ln, starts, dtype=TYPES[out])
        mine = slice(before, before + T)
        assert torch.equal(a[mine].float().cpu(), k[mine]) and torch.equal(b[mine].float().cpu(), v[mine]), out
    again = torch.full_like(cache, 0x55)
    for first in range(0, T, 1000):   # in parts, which one row a workgroup writes: the same bytes, and no others
        at = np.clip(starts.cpu().numpy(), before + first, before + min(T, first + 1000))
        left = np.array([max(0, min(starts[i + 1].item(), before + first + 1000) - starts[i].item()) for i in range(4)])
        part = torch.tensor(np.array(lens) - np.array(rows) + np.minimum(left, rows), dtype=torch.int32).cuda()
        qmm.cache_write(again, kd, vd, table, part, torch.from_numpy(at.astype(np.int32)).cuda())
    assert torch.equal(again, cache)
