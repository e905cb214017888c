"""Refusals of rope, cache_write, cache_read, cache_attention and cache_evict, without a GPU: every validation error is
returned by the host before any HIP call (the pointers are never dereferenced), and the binding refuses tensors it cannot
pass on."""
import ctypes

import pytest
import torch

import bit_quantized_mat_quantize_amd as qmm
from bit_quantized_mat_quantize_amd._binding import _Cache
from test_abi import EALIGN, EINVAL, EUNSUP, OK, _last, lib  # noqa: F401
from test_abi_operators import BIG, _far

CACHE = dict(data=_far(0), bytes=BIG, pages=8, page=32, heads=2, dim=128, table=_far(1), seqs=3, width=4, lens=_far(2),
             starts=_far(3), rows=7)


def _cache(**kw):
    return ctypes.byref(_Cache(**{**CACHE, **kw}))


def _split(kw):
    return _cache(**{k: v for k, v in kw.items() if k in CACHE}), {k: v for k, v in kw.items() if k not in CACHE}


def _cache_refusals(call, rows=True):
    for bad in (dict(page=8), dict(page=48), dict(page=2048), dict(dim=80), dict(dim=32), dict(heads=0), dict(heads=1025),
                dict(pages=0), dict(pages=2**31), dict(seqs=65537), dict(width=0), dict(width=2**30 // 32 + 1)):
        assert call(**bad) == EUNSUP, bad
    assert call(seqs=-1) == EINVAL
    for p in ("data", "table", "lens") + (("starts",) if rows else ()):
        if p != "starts":
            assert call(**{p: None}) == EINVAL, p
        assert call(**{p: CACHE[p] + 4}) == EALIGN, p
    need = 8 * 2 * 2 * 32 * 72
    assert call(bytes=need - 1) == EINVAL and "the cache holds" in _last_of(call)
    if rows:
        assert call(rows=-1) == EINVAL and call(rows=2**22 + 1) == EUNSUP
        assert call(starts=None) == EINVAL and "one row" in _last_of(call)
        assert call(rows=0, data=CACHE["data"]) == OK and call(seqs=0, rows=0, data=None, table=None, lens=None) == OK


def _last_of(call):
    return _last(call.lib)


def test_cache_bytes(lib):  # noqa: F811
    assert lib.qmm_cache_bytes(8, 32, 2, 128) == 8 * 2 * 2 * 32 * 72
    for bad in ((0, 32, 2, 128), (8, 8, 2, 128), (8, 33, 2, 128), (8, 32, 0, 128), (8, 32, 2, 100), (2**31, 32, 2, 128)):
        assert lib.qmm_cache_bytes(*bad) == 0, bad
    assert lib.qmm_cache_bytes(2**31 - 1, 1024, 1024, 256) == (2**31 - 1) * 2 * 1024 * 1024 * 144


def test_rope_refusals(lib):  # noqa: F811
    base = dict(t=0, x=_far(0), xb=BIG, ldx=1024, hx=128, pos=_far(1), f=None, o=_far(2), ob=BIG, ldo=1024, ho=128, T=5,
                H=8, D=128, rot=64, inter=0, base=1e4, fs=1.0, lo=0.0, hi=0.0, m=1.0)

    def call(**kw):
        a = {**base, **kw}
        return lib.qmm_rope(a["t"], a["x"], a["xb"], a["ldx"], a["hx"], a["pos"], a["f"], a["o"], a["ob"], a["ldo"],
                            a["ho"], a["T"], a["H"], a["D"], a["rot"], a["inter"], a["base"], a["fs"], a["lo"], a["hi"],
                            a["m"], None)

    nan, inf = float("nan"), float("inf")
    assert call(t=3) == EUNSUP and call(T=-1) == EINVAL and call(T=2**22 + 1) == EUNSUP
    assert call(H=0) == EUNSUP and call(H=65537) == EUNSUP and call(D=1025) == EUNSUP and call(D=1, rot=2) == EUNSUP
    assert call(rot=0) == EUNSUP and call(rot=63) == EUNSUP and call(rot=130) == EUNSUP
    for bad in (dict(base=0.0), dict(base=-1.0), dict(base=nan), dict(base=inf), dict(fs=-1.0), dict(fs=nan), dict(lo=nan),
                dict(hi=inf), dict(m=nan), dict(m=inf), dict(ldx=-1), dict(hx=-1)):
        assert call(**bad) == EINVAL, bad
    for p in ("x", "pos", "o"):
        assert call(**{p: None}) == EINVAL and call(**{p: base[p] + 4}) == EALIGN, p
    assert call(f=_far(3) + 4) == EALIGN
    assert call(xb=5 * 1024 * 4 - 1) == EINVAL and call(ob=5 * 1024 * 4 - 1) == EINVAL
    assert call(t=2, xb=5 * 1024 * 2 - 1) == EINVAL
    # out's own rows: tokens within heads and heads within tokens are both orders, anything between is not
    assert call(ho=64) == EINVAL and "overlap" in _last(lib)
    assert call(ldo=512) == EINVAL and call(ldo=-128) == EINVAL and call(ldo=64, ho=128) == EINVAL
    assert call(ldx=2**32 + 1) == EUNSUP
    # in place only with the same strides; column ranges of one matrix share nothing
    assert call(o=_far(0), ldo=2048) == EINVAL and "without being x" in _last(lib)
    assert call(o=_far(0) + 512) == EINVAL
    assert call(o=_far(1)) == EINVAL and call(f=_far(4), o=_far(4)) == EINVAL and "positions or factors" in _last(lib)
    wide = dict(ldx=2048, ldo=2048)
    assert call(o=_far(0) + 1020 * 4, **wide) == EINVAL
    assert call(T=0, x=None, pos=None, o=None) == OK


def test_cache_write_refusals(lib):  # noqa: F811
    base = dict(t=0, k=_far(4), kb=BIG, ldk=256, v=_far(5), vb=BIG, ldv=256)

    def call(**kw):
        c, kw = _split(kw)
        a = {**base, **kw}
        return lib.qmm_cache_write(c, a["t"], a["k"], a["kb"], a["ldk"], a["v"], a["vb"], a["ldv"], None)

    call.lib = lib
    _cache_refusals(call)
    assert lib.qmm_cache_write(None, 0, _far(4), BIG, 256, _far(5), BIG, 256, None) == EINVAL
    assert call(t=3) == EUNSUP and call(ldk=255) == EINVAL and call(ldv=2**32 + 4) == EUNSUP
    assert call(ldk=258) == EALIGN and call(t=1, ldv=260) == EALIGN and "16 bytes" in _last(lib)
    for p in ("k", "v"):
        assert call(**{p: None}) == EINVAL and call(**{p: base[p] + 8}) == EALIGN, p
        assert call(**{p + "b": 7 * 256 * 4 - 1}) == EINVAL
        assert call(**{p: _far(0) + 1024}) == EINVAL and "overlaps" in _last(lib)
    for p in ("table", "lens", "starts"):
        assert call(**{p: _far(0) + 64}) == EINVAL and "overlaps" in _last(lib), p


def test_cache_read_refusals(lib):  # noqa: F811
    need = 7 * 256 * 2
    base = dict(t=1, k=_far(4), kb=need, v=_far(5), vb=need)

    def call(**kw):
        c, kw = _split(kw)
        a = {**base, **kw}
        return lib.qmm_cache_read(c, a["t"], a["k"], a["kb"], a["v"], a["vb"], None)

    call.lib = lib
    _cache_refusals(call)
    assert call(t=4) == EUNSUP and call(kb=need - 1) == EINVAL and call(t=0) == EINVAL
    for p in ("k", "v"):
        assert call(**{p: None}) == EINVAL and call(**{p: base[p] + 8}) == EALIGN, p
        for other in ("data", "table", "lens", "starts"):
            assert call(**{p: CACHE[other]}) == EINVAL and "overlaps" in _last(lib), (p, other)
    assert call(v=_far(4) + need - 16) == EINVAL


def test_cache_attention_refusals(lib):  # noqa: F811
    base = dict(t=0, q=_far(4), qb=BIG, ldq=768, hq=6, o=_far(5), ob=BIG, ldo=768, scale=0.1, causal=1, window=0,
                lse=_far(6), mass=_far(7), ldm=128, ws=_far(8), wsb=BIG)

    def call(**kw):
        c, kw = _split(kw)
        a = {**base, **kw}
        return lib.qmm_cache_attention(c, a["t"], a["q"], a["qb"], a["ldq"], a["hq"], a["o"], a["ob"], a["ldo"], a["scale"],
                                       a["causal"], a["window"], a["lse"], a["mass"], a["ldm"], a["ws"], a["wsb"], None)

    call.lib = lib
    _cache_refusals(lambda_with(call, width=4))
    assert call(t=3) == EUNSUP and call(hq=5) == EUNSUP and call(hq=0) == EUNSUP and call(hq=1026) == EUNSUP
    assert call(scale=float("nan")) == EINVAL and call(scale=float("inf")) == EINVAL
    assert call(window=-1) == EINVAL and call(window=5, causal=0) == EUNSUP
    for p in ("q", "o", "ws"):
        assert call(**{p: None}) == EINVAL, p
    for p in ("q", "o", "lse", "mass", "ws"):
        assert call(**{p: base[p] + 8}) == EALIGN, p
    assert call(ldq=767) == EINVAL and call(ldo=767) == EINVAL and call(ldq=770) == EALIGN and call(t=1, ldo=772) == EALIGN
    assert call(qb=7 * 768 * 4 - 1) == EINVAL and call(ob=7 * 768 * 4 - 1) == EINVAL
    assert call(ldm=127) == EINVAL and "ld_mass" in _last(lib)
    size = lib.qmm_cache_attention_workspace_bytes
    need = size(0, 7, 6, 2, 128, 3, 4, 32, 1, 1)
    assert need > 0 and call(wsb=need - 1) == EINVAL and "workspace" in _last(lib)
    for o in ("o", "lse", "mass", "ws"):
        for i in ("data", "table", "lens", "starts"):
            assert call(**{o: CACHE[i]}) == EINVAL and "overlaps" in _last(lib), (o, i)
        assert call(**{o: _far(4)}) == EINVAL and "overlaps q" in _last(lib), o
        for other in ("o", "lse", "mass", "ws"):
            if other != o:
                assert call(**{o: base[other]}) == EINVAL and "overlaps another" in _last(lib), (o, other)
    # out beside q in one matrix, but not on it
    assert call(ldq=2048, ldo=2048, o=_far(4) + 760 * 4) == EINVAL
    # too many workgroups: 2^24 - 1 of 256 threads are one launch
    many = dict(heads=1024, hq=1024, dim=64, seqs=65536, width=2**26, page=16, rows=65536, starts=None, mass=None,
                bytes=BIG, ldq=65536, ldo=65536, qb=1 << 62, ob=1 << 62, wsb=1 << 62, lse=None)
    assert call(**many) == EUNSUP and "workgroups" in _last(lib)
    for bad in ((0, 6, 2, 128, 3, 4, 32), (7, 5, 2, 128, 3, 4, 32), (7, 6, 2, 100, 3, 4, 32), (7, 6, 2, 128, 0, 4, 32),
                (7, 6, 2, 128, 3, 0, 32), (7, 6, 2, 128, 3, 4, 40), (2**22 + 1, 6, 2, 128, 3, 4, 32)):
        assert size(0, *bad, 1, 1) == 0, bad
    assert size(3, 7, 6, 2, 128, 3, 4, 32, 1, 1) == 0


def lambda_with(call, **more):
    def f(**kw):
        return call(**{**more, **kw})
    f.lib = call.lib
    return f


def test_cache_evict_refusals(lib):  # noqa: F811
    base = dict(mass=_far(4), ldm=128, budget=50, recent=10, to=_far(5), tw=2, lo=_far(6), mo=_far(7), ldo=64, ids=_far(8))

    def call(**kw):
        c, kw = _split(kw)
        a = {**base, **kw}
        return lib.qmm_cache_evict(c, a["mass"], a["ldm"], a["budget"], a["recent"], a["to"], a["tw"], a["lo"], a["mo"],
                                   a["ldo"], a["ids"], None)

    call.lib = lib
    _cache_refusals(call, rows=False)
    assert call(budget=0) == EUNSUP and call(budget=2**30 + 1, tw=2**25) == EUNSUP
    assert call(recent=-1) == EINVAL and call(recent=51) == EINVAL
    assert call(tw=0) == EINVAL and call(budget=65) == EINVAL and call(tw=2**26) == EINVAL
    assert call(ldm=127) == EINVAL and call(ldo=49) == EINVAL
    for p in ("mass", "to", "lo", "mo", "ids"):
        assert call(**{p: None}) == EINVAL and call(**{p: base[p] + 4}) == EALIGN, p
    for o in ("lo", "mo", "ids", "data"):
        mine = CACHE["data"] if o == "data" else base[o]
        for i in ("table", "lens", "mass", "to"):
            assert call(**{i: mine}) == EINVAL and "overlaps" in _last(lib), (o, i)
        for other in ("lo", "mo", "ids"):
            if other != o:
                assert call(**{other: mine}) == EINVAL and "overlaps another" in _last(lib), (o, other)
    assert call(seqs=65536, heads=1024) == EUNSUP
    assert call(seqs=0, data=None, mass=None) == OK


def test_rows_times_heads_and_tables_of_another_width(lib):  # noqa: F811
    """More query rows than 32-bit row numbers count are refused; so is the table itself read with another width."""
    size = lib.qmm_cache_attention_workspace_bytes
    assert size(1, 2**20, 1024, 1024, 64, 9, 4, 32, 1, 1) > 0
    assert size(1, 2**20 + 1, 1024, 1024, 64, 9, 4, 32, 1, 1) == 0
    c = _cache(heads=1024, rows=2**20 + 1, dim=64)
    assert lib.qmm_cache_attention(c, 1, _far(4), 1 << 62, 65536, 1024, _far(5), 1 << 62, 65536, 0.1, 1, 0, None, None, 0,
                                   _far(8), 1 << 62, None) == EUNSUP and "2^30" in _last(lib)
    for width in (2, 5):
        assert lib.qmm_cache_evict(_cache(), _far(4), 128, 50, 10, CACHE["table"], width, _far(6), _far(7), 64, _far(8),
                                   None) == EINVAL and "to is the table" in _last(lib)


def test_binding_refusals():
    """Shapes and types are checked before the library is called; CPU tensors are refused."""
    i32 = torch.int32
    x, pos = torch.zeros(3, 4, 64), torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError, match="GPU tensor"):
        qmm.rope(x, pos)
    for kw in (dict(layout="pairs"), dict(ramp=(3.0, 2.0)), dict(factors=torch.zeros(31)), dict(factors=torch.zeros(32).half())):
        with pytest.raises(ValueError):
            qmm.rope(x, pos, **kw)
    for bad in (pos.long(), pos[:2]):
        with pytest.raises(ValueError):
            qmm.rope(x, bad)
    with pytest.raises(ValueError, match="unit stride"):
        qmm.rope(x.transpose(1, 2), pos)
    with pytest.raises(ValueError, match="no cache"):
        qmm.cache_new(4, 2, 80, device="cpu")
    cache = qmm.cache_new(4, 2, 64, page=16, device="cpu")
    assert cache.numel() == qmm.cache_bytes(4, 2, 64, page=16)
    table, lens, starts = torch.zeros(3, 2, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(4, dtype=i32)
    k = torch.zeros(5, 2, 64)
    q = torch.zeros(5, 6, 64)
    mass = torch.zeros(3, 2, 32)
    with pytest.raises(ValueError, match="GPU tensor"):
        qmm.cache_write(cache, k, k, table, lens, starts)
    with pytest.raises(ValueError, match="GPU tensor"):
        qmm.cache_read(cache, 5, table, lens, starts)
    with pytest.raises(ValueError, match="GPU tensor"):
        qmm.cache_attention(q, cache, table, lens, starts)
    with pytest.raises(ValueError, match="GPU tensor"):
        qmm.cache_evict(cache, table, lens, mass, 20)
    for bad in (dict(cache=cache.float()), dict(cache=cache[:, :1]), dict(cache=cache[..., :35]), dict(table=table.long()),
                dict(table=table[:, :1]), dict(table=table[0]), dict(lens=lens[:2]), dict(lens=lens.long()),
                dict(starts=starts[:3]), dict(k=k[:, :1]), dict(k=k[..., :32]), dict(v=k.half()),
                dict(k=k.transpose(1, 2).contiguous().transpose(1, 2))):
        a = dict(cache=cache, k=k, v=k, table=table, lens=lens, starts=starts)
        a.update(bad)
        with pytest.raises(ValueError):
            qmm.cache_write(**a)
    for kw in (dict(budget=33), dict(budget=0), dict(budget=20, recent=21), dict(budget=20, mass=mass[:, :, :31]),
               dict(budget=20, mass=mass.half()), dict(budget=20, to=table[:2]), dict(budget=20, to=table.long())):
        with pytest.raises(ValueError):
            qmm.cache_evict(**{**dict(cache=cache, table=table, lens=lens, mass=mass), **kw})
    for t in (x, k, q, mass):
        t.requires_grad_()
    for call in (lambda: qmm.rope(x, pos), lambda: qmm.cache_write(cache, k, k, table, lens, starts),
                 lambda: qmm.cache_attention(q, cache, table, lens, starts),
                 lambda: qmm.cache_evict(cache, table, lens, mass, 20)):
        with pytest.raises(ValueError, match="no backward"):
            call()


def test_ramp_of_a_stretched_context():
    """Pairs that turn often keep their angles, slow ones are scaled; the formulas by hand for 64 of base 10000."""
    r = qmm.rope_ramp(64, 10000.0, 4096, 16.0)
    # turns of pair i within 4096 positions: 4096 * 10000^(-i/32) / 2 pi; 32 turns at i = 10.47, 1 turn at i = 22.51
    assert r["ramp"] == (10.0, 23.0) and r["freq_scale"] == 1 / 16 and abs(r["magnitude"] - 1.2772588722239782) < 1e-15
    assert qmm.rope_ramp(64, 10000.0, 4096, 1.0)["magnitude"] == 1.0
