"""The operators between the projections of a served model, as cases that can be timed and compared.

* ``rope``:   rotary positions of the heads of a projection's output (qmm.rope);
* ``write``:  new rows of keys and values into a paged cache of 4-bit blocks, and these rows read back as the
  values that the cache holds (qmm.cache_write, qmm.cache_read);
* ``attend``: attention over such a cache, single tokens, several and whole prompts, and the weight that each
  entry gets (qmm.cache_attention);
* ``evict``:  the entries with the most accumulated weight into fewer pages, read back as values
  (qmm.cache_evict, qmm.cache_read).

With ``own`` false, ``run`` computes a case in elementary torch operations; with ``own`` true it calls the
library.  ``exact`` computes the same outputs in 64 bits, written apart from both.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one token of a chat: query and key heads side by side in the projection's output, the smallest call
        rope("rope_token", T=1, H=40, D=128, rot=128, layout="half", base=500000.0, scaling="none", far=8192, type="f32"),
        # long prompts of a model whose context was stretched 16 times, half of each head rotated
        rope("rope_prompt", T=4099, H=40, D=128, rot=64, layout="interleaved", base=10000.0, scaling="ramp",
             far=1000000, type="bf16"),
        # a decode step of 61 requests: one new row each
        write("write_batch", B=61, rows=1, length=5000, heads=8, D=128, page=64, type="f32"),
        # four prompts of different lengths in one step, small pages
        write("write_prompt", B=4, rows=1025, length=1500, heads=8, D=128, page=16, type="bf16"),
        # one token of a chat after a thousand others
        attend("attend_token", B=1, rows=1, length=1000, heads=8, group=4, D=128, page=64, window=0, mass=False,
               lse=False, type="f32"),
        # a decode step of 32 requests of up to 8192 tokens
        attend("attend_batch", B=32, rows=1, length=8192, heads=8, group=8, D=128, page=64, window=0, mass=False,
               lse=False, type="f32"),
        # two long documents, one token each
        attend("attend_long", B=2, rows=1, length=131072, heads=8, group=4, D=128, page=256, window=0, mass=False,
               lse=True, type="bf16"),
        # drafts of a few tokens beside the rest of a prompt, a window, an odd group, small heads
        attend("attend_mixed", B=9, rows=555, length=4100, heads=8, group=3, D=64, page=16, window=1024, mass=False,
               drafts=True, lse=False, type="f16"),
        # the second part of two prompts: 2048 new rows each on top of what is there
        attend("attend_prompt", B=2, rows=2048, length=8192, heads=8, group=4, D=128, page=64, window=0, mass=False,
               lse=False, type="bf16"),
        # prompts in full precision whose weights are accumulated for the eviction
        attend("attend_mass", B=3, rows=700, length=2100, heads=4, group=7, D=128, page=32, window=0, mass=True,
               lse=False, type="f32"),
        # four requests that ran over their budget of 1024 entries
        evict("evict_step", B=4, length=1100, budget=1024, recent=128, heads=8, D=128, page=64),
        # a batch after long prompts: at most 4096 entries of each stay
        evict("evict_batch", B=16, length=9000, budget=4096, recent=512, heads=8, D=128, page=64),
    ]


def rope(name, **c):
    return {"name": name, "op": "rope", **c}


def write(name, **c):
    return {"name": name, "op": "write", **c}


def attend(name, **c):
    return {"name": name, "op": "attend", "drafts": False, **c}


def evict(name, **c):
    return {"name": name, "op": "evict", **c}


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(("rope", "write", "attend", "attend", "attend", "evict"))
    kind, page = rng.choice(sorted(TYPES)), rng.choice((16, 32, 64, 128, 256))
    heads, D = rng.choice((1, 2, 4, 8, rng.randint(1, 16))), rng.choice((64, 64, 96, 128, 128, 192, 256))
    if op == "rope":
        D = rng.choice((64, 80, 96, 128, 256))
        c = {"op": op, "T": _log(rng, 1, 4096), "H": _log(rng, 1, 72), "D": D, "rot": rng.choice((D, D, D // 2, 2 * rng.randint(8, D // 2))),
             "layout": rng.choice(("half", "interleaved")), "base": rng.choice((10000.0, 500000.0, 1000000.0)),
             "scaling": rng.choice(("none", "linear", "ramp", "factors")), "far": _log(rng, 100, 1000000), "type": kind}
    elif op == "write":
        rows = _log(rng, 1, 1024)
        c = {"op": op, "B": _log(rng, 1, max(1, 4096 // rows)), "rows": rows, "length": rows + _log(rng, 1, 1000),
             "heads": heads, "D": D, "page": page, "type": kind}
    elif op == "attend":
        rows = rng.choice((1, 1, _log(rng, 2, 16), _log(rng, 16, 2048)))
        c = {"op": op, "B": _log(rng, 1, 64), "rows": rows, "length": rows + _log(rng, 16, 32768), "heads": heads,
             "group": rng.choice((1, 2, 4, 8, rng.randint(1, 16))), "D": D, "page": page,
             "window": rng.choice((0, 0, 0, _log(rng, 16, 4096))), "mass": rng.choice((False, False, True)),
             "drafts": rows > 16 and rng.random() < 0.3, "lse": rng.choice((False, True)), "type": kind}
        while _cost(c) > 2 * 2048 * 8192 * 32 * 128 / 2 or c["B"] * c["length"] * c["heads"] * c["D"] > 2 * 131072 * 8 * 128:
            c["B"], c["length"] = (c["B"] + 1) // 2, rows + (c["length"] - rows + 1) // 2
            c["group"] = (c["group"] + 1) // 2
    else:
        budget = _log(rng, 16, 8192)
        c = {"op": op, "B": _log(rng, 1, 32), "length": budget + _log(rng, 1, 2 * budget), "budget": budget,
             "recent": rng.choice((0, budget // 8, rng.randint(0, budget))), "heads": heads, "D": D, "page": page}
        while c["B"] * budget * heads * D > 16 * 4096 * 8 * 128:
            c["B"] = c["B"] // 2 or 1
            heads = c["heads"] = (heads + 1) // 2
    return c


def _cost(c):
    """Products of a query and a key element of an attention case, with what the matrix of a small one is padded to."""
    return c["B"] * max(4, c["rows"]) * c["length"] * c["heads"] * c["group"] * c["D"]


def _plan(c):
    """Each sequence's new rows and its length with them: of different sizes, up to those of the case."""
    rows, lens = [], []
    for i in range(c["B"]):
        n = c["rows"]
        if c["op"] == "write":
            n = max(1, n * (i + 1) // c["B"])
        elif c["drafts"] and i < c["B"] - 1:
            n = 1 + 3 * i % 7  # drafts beside one prompt
        elif n > 200:
            n -= 37 * (i % 4)
        rows.append(n)
        lens.append(max(n, c["length"] - i * c["length"] // (3 * c["B"])))
    return rows, lens


# ---------------------------------------------------------------- what a program has in hand
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return {"rope": _prepare_rope, "write": _prepare_write, "attend": _prepare_attend, "evict": _prepare_evict}[case["op"]](case, g)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _prepare_rope(c, g):
    T, H, D = c["T"], c["H"], c["D"]
    qkv = (_randn(g, T, (H + 8) * D) * 2.0).to(TYPES[c["type"]])  # query and key heads, then the values'
    positions = torch.randint(0, c["far"], (T,), generator=g, device=DEV, dtype=torch.int32)
    factors = None
    if c["scaling"] == "factors":
        factors = 1.0 + 7.0 * torch.rand(c["rot"] // 2, generator=g, device=DEV)
    scaling = {"none": {}, "linear": {"freq_scale": 0.125}, "factors": {"magnitude": 1.19},
               "ramp": {"freq_scale": 1 / 16, "ramp": (0.2 * c["rot"], 0.4 * c["rot"]), "magnitude": 0.1 * math.log(16) + 1}}
    return {"case": c, "x": qkv[:, :H * D].unflatten(1, (H, D)), "positions": positions, "factors": factors,
            "scaling": scaling[c["scaling"]]}


def _tables(c, g, lens, spare=3):
    """Pages in no order, a few of them nobody's, and for each sequence its own."""
    need = [-(-n // c["page"]) for n in lens]
    order = torch.randperm(sum(need) + spare, generator=g, device=DEV).to(torch.int32)
    width = -(-max(lens) // c["page"])
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=DEV)
    at = torch.arange(width, device=DEV) < torch.tensor(need, device=DEV).unsqueeze(1)
    table[at] = order[: sum(need)]
    return table, sum(need) + spare


def _filled(c, g, table, pages, lens):
    """A cache whose entries are as rows of keys and values leave them; what nobody wrote holds anything."""
    heads, page, D, B = c["heads"], c["page"], c["D"], len(lens)
    cache = torch.randint(0, 256, (pages, 2, heads, page, D * 9 // 16), generator=g, device=DEV, dtype=torch.uint8)
    n = page * D // 2
    # block scales of values about one, either sign; some keys stand out
    d = (0.08 + 0.2 * torch.rand(pages, 2, heads, D // 32, page, generator=g, device=DEV))
    d *= 1.0 - 2.0 * (torch.rand(d.shape, generator=g, device=DEV) < 0.5).float()
    d[:, 0] *= 1.0 + 1.5 * (torch.rand(pages, heads, 1, page, generator=g, device=DEV) < 0.02).float()
    written = torch.zeros(pages, page, dtype=torch.bool, device=DEV)
    have = torch.arange(table.shape[1] * page, device=DEV) < torch.tensor(lens, device=DEV).unsqueeze(1)
    used = table >= 0
    written[table[used].long()] = have.view(B, -1, page)[used]
    d = torch.where(written.view(pages, 1, 1, 1, page), d, math.nan).half()
    cache.view(pages, 2, heads, -1)[..., n:] = d.view(torch.uint8).reshape(pages, 2, heads, -1)
    return cache


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _starts(rows):
    return _ints([sum(rows[:i]) for i in range(len(rows) + 1)])


def _prepare_write(c, g):
    rows, lens = _plan(c)
    table, pages = _tables(c, g, lens)
    T, n, t = sum(rows), c["heads"] * c["D"], TYPES[c["type"]]
    qkv = _randn(g, T, 6 * n)  # four query heads for each key head, then keys and values
    qkv[:, torch.randperm(6 * n, generator=g, device=DEV)[: 6 * n // 50]] *= 6.0  # channels that stand out
    qkv = qkv.to(t)
    cache = torch.full((pages, 2, c["heads"], c["page"], c["D"] * 9 // 16), 255, dtype=torch.uint8, device=DEV)
    k, v = (qkv[:, a * n:(a + 1) * n].unflatten(1, (c["heads"], c["D"])) for a in (4, 5))
    return {"case": c, "cache": cache, "k": k, "v": v, "table": table, "lens": _ints(lens),
            "starts": None if c["rows"] == 1 else _starts(rows), "rows": rows}


def _prepare_attend(c, g):
    rows, lens = _plan(c)
    table, pages = _tables(c, g, lens)
    T, n = sum(rows), c["heads"] * c["group"] * c["D"]
    q = (1.2 * _randn(g, T, n + 2 * c["heads"] * c["D"])).to(TYPES[c["type"]])[:, :n].unflatten(1, (-1, c["D"]))
    mass = torch.rand(c["B"], c["heads"], table.shape[1] * c["page"], generator=g, device=DEV) if c["mass"] else None
    return {"case": c, "cache": _filled(c, g, table, pages, lens), "q": q, "table": table, "lens": _ints(lens),
            "starts": None if c["rows"] == 1 else _starts(rows), "rows": rows, "mass": mass}


def _prepare_evict(c, g):
    lens = [max(1, c["length"] - i * c["length"] // (3 * c["B"])) for i in range(c["B"])]
    left = [min(n, c["budget"]) for n in lens]
    table, used = _tables(c, g, lens)
    to, more = _tables(c, g, [c["budget"]] * c["B"], spare=0)
    width = table.shape[1] * c["page"]
    # a few entries hold most of the weight, and many that nothing looked at hold none
    mass = torch.rand(c["B"], c["heads"], width, generator=g, device=DEV) ** 4 * 8.0
    mass *= (torch.rand(mass.shape, generator=g, device=DEV) < 0.9).float()
    mass *= (torch.arange(width, device=DEV) < torch.tensor(lens, device=DEV).view(-1, 1, 1)).float()
    cache = _filled(c, g, table, used + more, lens)
    return {"case": c, "cache": cache, "table": table, "lens": _ints(lens), "mass": mass, "to": to + used, "rows": left,
            "left": _starts(left)}


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        return _own(c, s)
    return {"rope": _plain_rope, "write": _plain_write, "attend": _plain_attend, "evict": _plain_evict}[c["op"]](c, s)


def _own(c, s):
    import bit_quantized_mat_quantize_amd as qmm
    if c["op"] == "rope":
        return qmm.rope(s["x"], s["positions"], rot=c["rot"], layout=c["layout"], base=c["base"], factors=s["factors"],
                        **s["scaling"])
    if c["op"] == "write":
        qmm.cache_write(s["cache"], s["k"], s["v"], s["table"], s["lens"], starts=s["starts"])
        k, v = qmm.cache_read(s["cache"], s["k"].shape[0], s["table"], s["lens"], starts=s["starts"])
        return {"k": k, "v": v}
    if c["op"] == "attend":
        mass = None if s["mass"] is None else s["mass"].clone()
        out = qmm.cache_attention(s["q"], s["cache"], s["table"], s["lens"], starts=s["starts"], window=c["window"],
                                  mass=mass, lse=c["lse"])
        return {"out": out[0] if c["lse"] else out, "lse": out[1] if c["lse"] else None, "mass": mass}
    lens, mass, ids = qmm.cache_evict(s["cache"], s["table"], s["lens"], s["mass"], c["budget"], c["recent"], to=s["to"])
    k, v = qmm.cache_read(s["cache"], sum(s["rows"]), s["to"], lens, starts=s["left"], dtype=torch.float16)
    return {"lens": lens, "mass": mass, "ids": ids, "k": k, "v": v}


def _plain_rope(c, s):
    """Angles in 64 bits, the rotation in 32."""
    x, rot, half = s["x"].float(), c["rot"], c["rot"] // 2
    p = s["scaling"]
    i = torch.arange(half, device=DEV, dtype=torch.float64)
    f = c["base"] ** (-2.0 * i / rot)
    if s["factors"] is not None:
        f = f / s["factors"].double()
    r = 1.0
    if "ramp" in p:
        low, high = p["ramp"]
        r = ((i - low) / (high - low)).clamp(0.0, 1.0)
    f = f * (1.0 - r * (1.0 - p.get("freq_scale", 1.0)))
    angle = (s["positions"].double().unsqueeze(1) * f).unsqueeze(1)
    mag = p.get("magnitude", 1.0)
    cos, sin = (angle.cos() * mag).float(), (angle.sin() * mag).float()
    if c["layout"] == "half":
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1).to(s["x"].dtype)


def _row_map(s, n):
    """For each sequence its rows as indices of the flat ones (padded to n with row 0), which are real, and their positions."""
    B = s["lens"].numel()
    i = torch.arange(n, device=DEV)
    if s["starts"] is None:
        first, count = torch.arange(B, device=DEV), torch.ones(B, dtype=torch.long, device=DEV)
    else:
        first, count = s["starts"][:-1].long(), (s["starts"][1:] - s["starts"][:-1]).long()
    real = i < count.unsqueeze(1)
    return torch.where(real, first.unsqueeze(1) + i, 0), real, s["lens"].long().unsqueeze(1) - count.unsqueeze(1) + i


def _encoded(x):
    """Blocks of 32 as the library's Q4_0 encoder leaves them: the scale's fp16 and the codes."""
    x = x.float().unflatten(-1, (-1, 32))
    a = x.abs()
    top = x.gather(-1, a.argmax(-1, keepdim=True))
    d = top / -8.0
    inv = torch.where(d != 0, 1.0 / d, 0.0)
    return d.half().squeeze(-1), (torch.round(x * inv) + 8.0).clamp(0.0, 15.0).to(torch.uint8).flatten(-2)


def _words(codes):
    """Codes as bytes, eight to a 32-bit word: the first in the lowest bits."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _plain_write(c, s):
    heads, D, page = c["heads"], c["D"], c["page"]
    at, real, pos = _row_map(s, max(s["rows"]))
    page_of = s["table"].gather(1, (pos // page).clamp(min=0, max=s["table"].shape[1] - 1))[real].long()
    t, rows = (pos % page)[real], at[real]
    k, v, d = _parts(c, s["cache"])
    dk, qk = _encoded(s["k"][rows])
    dv, qv = _encoded(s["v"][rows])
    # keys: a row per entry, word g of every block side by side; values: four entries' words side by side
    k[page_of, :, t] = _words(qk).view(-1, heads, D // 32, 4, 4).transpose(2, 3).reshape(-1, heads, D // 2)
    v[page_of, :, t // 4, :, t % 4] = _words(qv).view(-1, heads, D // 8, 4)
    d[:, 0][page_of, :, :, t] = dk
    d[:, 1][page_of, :, :, t] = dv
    return dict(zip("kv", _plain_read(c, s["cache"], s["table"], real, pos, torch.float32)))


def _gathered(c, cache, table):
    """Keys and values of whole tables in fp32 [B, heads, width * page, D]; what no page holds is zero."""
    heads, D, page, (B, W) = c["heads"], c["D"], c["page"], table.shape
    flat = cache.view(cache.shape[0], 2, heads, -1)[table.long().clamp(min=0)]
    d = flat[..., page * D // 2:].contiguous().view(torch.float16).view(B, W, 2, heads, D // 32, page)
    b = flat[..., : page * D // 2]
    q = torch.stack((b & 15, b >> 4), -1).view(B, W, 2, heads, -1)
    k = q[:, :, 0].view(B, W, heads, page, 4, D // 32, 8).transpose(4, 5).reshape(B, W, heads, page, D)
    v = q[:, :, 1].view(B, W, heads, page // 4, D // 8, 4, 8).transpose(4, 5).reshape(B, W, heads, page, D)
    out = []
    for n, codes in enumerate((k, v)):
        x = (codes.view(B, W, heads, page, D // 32, 32).float() - 8.0) * d[:, :, n].transpose(-1, -2).unsqueeze(-1).float()
        out.append(x.permute(0, 2, 1, 3, 4, 5).reshape(B, heads, W * page, D))
    return out


def _parts(c, cache):
    """Views of a cache: its keys' rows, its values' words, the block scales of both."""
    flat, n = cache.view(cache.shape[0], 2, c["heads"], -1), c["page"] * c["D"] // 2
    return (flat[:, 0, :, :n].unflatten(-1, (c["page"], c["D"] // 2)),
            flat[:, 1, :, :n].unflatten(-1, (c["page"] // 4, c["D"] // 8, 4, 4)),
            flat[..., n:].view(torch.float16).unflatten(-1, (c["D"] // 32, c["page"])))


def _plain_read(c, cache, table, real, pos, dtype):
    """The entries of the given positions, one row each."""
    heads, D, page = c["heads"], c["D"], c["page"]
    k, v, d = _parts(c, cache)
    src, t = table.gather(1, (pos // page).clamp(min=0, max=table.shape[1] - 1))[real].long(), (pos % page)[real]
    k, v = k[src, :, t].view(-1, heads, 4, D // 32, 4).transpose(2, 3), v[src, :, t // 4, :, t % 4]
    out = []
    for n, b in enumerate((k, v)):
        q = torch.stack((b & 15, b >> 4), -1).view(-1, heads, D // 32, 32)
        out.append(((q.float() - 8.0) * d[:, n][src, :, :, t].unsqueeze(-1).float()).flatten(-2).to(dtype))
    return out


def _plain_attend(c, s):
    heads, G, D, n, B = c["heads"], c["group"], c["D"], max(s["rows"]), c["B"]
    at, real, pos = _row_map(s, n)
    k, v = _gathered(c, s["cache"], s["table"])
    L = k.shape[2]
    j = torch.arange(L, device=DEV)
    have = (j < s["lens"].unsqueeze(1)).view(B, 1, L, 1)
    k, v = torch.where(have, k, 0.0), torch.where(have, v, 0.0)
    q = s["q"][at].float().view(B, n, heads, G, D).permute(0, 2, 1, 3, 4).reshape(B, heads, n * G, D)
    x = torch.matmul(q, k.transpose(2, 3).contiguous()).view(B, heads, n, G, L) * (1.0 / math.sqrt(D))
    see = real.unsqueeze(2) & (j <= pos.unsqueeze(2))
    if c["window"]:
        see &= j > pos.unsqueeze(2) - c["window"]
    x = x.masked_fill_(~see.view(B, 1, n, 1, L), -math.inf)
    m = x.max(-1, keepdim=True).values.clamp(min=-3e38)
    e = x.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e.view(B, heads, n * G, L), v).view(B, heads, n, G, D) / total.clamp(min=1e-38)
    out = out.permute(0, 2, 1, 3, 4)[real].reshape(-1, heads * G, D).to(s["q"].dtype)
    lse = mass = None
    if c["lse"]:
        lse = (m + total.log()).squeeze(-1).permute(0, 2, 1, 3)[real].reshape(-1, heads * G)
    if c["mass"]:
        mass = s["mass"] + (e / total.clamp(min=1e-38)).sum((2, 3))
    return {"out": out, "lse": lse, "mass": mass}


def _plain_evict(c, s):
    heads, D, page, budget, (B, W) = c["heads"], c["D"], c["page"], c["budget"], s["table"].shape
    L, j = s["lens"].view(-1, 1, 1).long(), torch.arange(W * page, device=DEV)
    order = torch.where(j >= L - c["recent"], math.inf, s["mass"])
    order = torch.where(j >= L, -math.inf, order)
    ids = order.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    ids = torch.where(ids < L, ids, W * page).sort(-1).values
    ids = torch.nn.functional.pad(ids, (0, budget - ids.shape[-1]), value=W * page)
    real = ids < L
    at = torch.where(real, ids, 0)
    # entries as they are: a key's row, a value's words, both scales
    h = torch.arange(heads, device=DEV).view(1, -1, 1)
    src, t = s["table"].unsqueeze(1).expand(B, heads, W).gather(2, at // page).long(), at % page
    k, v, d = _parts(c, s["cache"])
    got = k[src, h, t], v[src, h, t // 4, :, t % 4], d[src, 0, h, :, t], d[src, 1, h, :, t]
    i = torch.arange(budget, device=DEV)
    dst, u = s["to"][:, i // page].unsqueeze(1).expand(B, heads, budget).long()[real], (i % page).expand(B, heads, budget)[real]
    hh = h.expand(B, heads, budget)[real]
    k[dst, hh, u], v[dst, hh, u // 4, :, u % 4] = got[0][real], got[1][real]
    d[dst, 0, hh, :, u], d[dst, 1, hh, :, u] = got[2][real], got[3][real]
    mass = torch.zeros(B, heads, s["to"].shape[1] * page, device=DEV)
    mass[..., :budget] = torch.where(real, s["mass"].gather(2, at), 0.0)
    lens = s["lens"].clamp(max=budget)
    _, some, pos = _row_map({"lens": lens, "starts": s["left"]}, max(s["rows"]))
    k, v = _plain_read(c, s["cache"], s["to"], some, pos, torch.float16)
    return {"lens": lens, "mass": mass, "ids": torch.where(real, ids, -1).int(), "k": k, "v": v}


# ---------------------------------------------------------------- the same in 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "write": _exact_write, "attend": _exact_attend, "evict": _exact_evict}[case["op"]](case, s)


def _exact_rope(c, s):
    """Pair by pair, as a product of complex numbers."""
    x, out, p = s["x"].double(), s["x"].double().clone(), s["scaling"]
    pos = s["positions"].double()
    for i in range(c["rot"] // 2):
        f = c["base"] ** (-2.0 * i / c["rot"])
        if s["factors"] is not None:
            f = f / s["factors"][i].double()
        share = 1.0
        if "ramp" in p:
            share = min(1.0, max(0.0, (i - p["ramp"][0]) / (p["ramp"][1] - p["ramp"][0])))
        turn = pos * (f * (share * p.get("freq_scale", 1.0) + (1.0 - share)))
        a, b = (i, i + c["rot"] // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)
        z = torch.complex(x[:, :, a], x[:, :, b]) * torch.polar(torch.full_like(turn, p.get("magnitude", 1.0)), turn).unsqueeze(1)
        out[:, :, a], out[:, :, b] = z.real, z.imag
    return out


def _exact_write(c, s):
    """The values that the blocks stand for: d and the codes go through the roundings that define them."""
    out = {}
    for name in "kv":
        x = s[name].double().unflatten(-1, (-1, 32))
        first = (x.abs() == x.abs().amax(-1, keepdim=True)).int().argmax(-1, keepdim=True)  # the first of equals
        d = (-x.gather(-1, first) / 8.0).float()
        inv = (1.0 / d.double()).float()
        q = torch.round((x * inv.double()).float().double()).add(8.0).clamp(0.0, 15.0)
        out[name] = ((q - 8.0) * d.half().double()).flatten(-2)
    return out


def _entries(c, cache, pages, h, part):
    """Entries of one head in the order of the pages, in 64 bits; each element found by its address."""
    page, D = c["page"], c["D"]
    n = page * D * 9 // 16
    flat = cache.view(-1)
    base = ((pages.long() * 2 + part) * c["heads"] + h) * n
    t, i = torch.arange(page, device=DEV).view(-1, 1), torch.arange(D, device=DEV)
    if part == 0:
        at = t * (D // 2) + (((i % 32) // 8) * (D // 32) + i // 32) * 4 + (i % 8) // 2
    else:
        at = ((t // 4 * (D // 8) + i // 8) * 4 + t % 4) * 4 + (i % 8) // 2
    q = (flat[base.view(-1, 1, 1) + at].int() >> (4 * (i % 2))) & 15
    scale = (base.view(-1, 1, 1) + page * D // 2 + 2 * ((i // 32) * page + t))
    bits = flat[scale].int() | (flat[scale + 1].int() << 8)
    d = bits.to(torch.int16).view(torch.float16).double()
    return ((q - 8) * d).view(-1, D)


def _exact_attend(c, s):
    """Sequence by sequence, head by head."""
    rows, lens = s["rows"], s["lens"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device=DEV)
    mass = None if s["mass"] is None else s["mass"].double()
    at = 0
    for b, (n, L) in enumerate(zip(rows, lens)):
        pages = s["table"][b, : -(-L // c["page"])]
        j, i = torch.arange(L, device=DEV), torch.arange(L - n, L, device=DEV).unsqueeze(1)
        hidden = (j > i) | (j <= i - c["window"]) if c["window"] else j > i
        for h in range(c["heads"]):
            k, v = (_entries(c, s["cache"], pages, h, part)[:L] for part in (0, 1))
            for g in range(h * c["group"], (h + 1) * c["group"]):
                x = (s["q"][at:at + n, g].double() @ k.t()) * c["D"] ** -0.5
                x[hidden] = -math.inf
                lse[at:at + n, g] = torch.logsumexp(x, 1)
                p = torch.softmax(x, 1)
                out[at:at + n, g] = p @ v
                if mass is not None:
                    mass[b, h, :L] += p.sum(0)
        at += n
    return {"out": out, "lse": lse if c["lse"] else None, "mass": mass}


def _exact_evict(c, s):
    """Sequence by sequence, head by head: the newest, and of the others those that fewest come before."""
    B, heads, page, budget, recent = c["B"], c["heads"], c["page"], c["budget"], c["recent"]
    lens = s["lens"].tolist()
    ids = torch.full((B, heads, budget), -1, dtype=torch.int32, device=DEV)
    mass = torch.zeros(B, heads, s["to"].shape[1] * page, dtype=torch.float64, device=DEV)
    ks, vs = [], []
    for b, L in enumerate(lens):
        k, v = [], []
        for h in range(heads):
            m = s["mass"][b, h, :L].double()
            if L <= budget:
                keep = torch.arange(L, device=DEV)
            else:
                old = L - recent
                best = torch.topk(m[:old], budget - recent).values if budget > recent else m[:0]
                edge = best.min() if budget > recent else torch.tensor(math.inf, device=DEV)
                above = (m[:old] > edge).nonzero().squeeze(1)
                equal = (m[:old] == edge).nonzero().squeeze(1)[: budget - recent - above.numel()]
                keep = torch.cat((above, equal, torch.arange(old, L, device=DEV))).sort().values
            ids[b, h, : keep.numel()] = keep.int()
            mass[b, h, : keep.numel()] = m[keep]
            pages = s["table"][b, : -(-L // page)]
            k.append(_entries(c, s["cache"], pages, h, 0)[keep])
            v.append(_entries(c, s["cache"], pages, h, 1)[keep])
        ks.append(torch.stack(k, 1))
        vs.append(torch.stack(v, 1))
    return {"lens": s["lens"].clamp(max=budget), "mass": mass, "ids": ids, "k": torch.cat(ks), "v": torch.cat(vs)}


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "rope":
        n = c["T"] * c["H"] * c["D"]
        return {"bytes": 2 * n * SIZE[c["type"]] + 4 * c["T"], "flops": 3 * c["T"] * c["H"] * c["rot"]}
    row = c["heads"] * c["D"]  # elements of an entry's keys, or of its values
    if c["op"] == "write":
        rows, _ = _plan(c)
        # both inputs, the blocks written and read, both outputs
        return {"bytes": sum(rows) * 2 * row * (SIZE[c["type"]] + 2 * 9 / 16 + 4), "flops": sum(rows) * 2 * row * 4}
    if c["op"] == "attend":
        rows, lens = _plan(c)
        keys = seen = 0
        for n, L in zip(rows, lens):
            w = c["window"] or L
            keys += min(L, w + n - 1)
            seen += sum(min(w, p + 1) for p in range(L - n, L))
        moved = keys * 2 * row * 9 / 16 + 2 * sum(rows) * c["group"] * row * SIZE[c["type"]]
        moved += 4 * sum(rows) * c["heads"] * c["group"] if c["lse"] else 0
        moved += 2 * 4 * sum(lens) * c["heads"] if c["mass"] else 0
        return {"bytes": moved, "flops": 4 * seen * c["group"] * row}
    lens = [max(1, c["length"] - i * c["length"] // (3 * c["B"])) for i in range(c["B"])]
    left = sum(min(n, c["budget"]) for n in lens)
    entry = 2 * row * 9 / 16
    # the weights, the entries that stay (read, written, read again), their new weights and places, their values
    return {"bytes": 4 * sum(lens) * c["heads"] + left * (3 * entry + 8 * c["heads"] + 2 * 2 * row), "flops": 4 * sum(lens) * c["heads"]}
