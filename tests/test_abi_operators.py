"""Refusals of embed_rows, lora_add and logprobs, without a GPU: every validation
error is returned by the host before any HIP call (the pointers are never
dereferenced), and the binding refuses tensors it cannot pass on."""
import pytest
import torch

import bit_quantized_mat_quantize_amd as qmm
from test_abi import A, EALIGN, EINVAL, EUNSUP, OK, _last, lib  # noqa: F401

BIG = 1 << 50


def _far(i):
    """Aligned fake addresses 2^52 bytes apart: buffers of any accepted size do not overlap."""
    return A + (i << 52)


def test_embed_rows_refusals(lib):  # noqa: F811
    base = dict(t=1, w=_far(0), wb=BIG, l=1, ids=_far(1), T=3, scale=1.0, o=_far(2), ob=BIG, N=8, K=512)

    def call(**kw):
        a = {**base, **kw}
        return lib.qmm_embed_rows(a["t"], a["w"], a["wb"], a["l"], a["ids"], a["T"], a["scale"], a["o"], a["ob"],
                                  a["N"], a["K"], None)

    assert call(t=4) == EUNSUP and "weight type" in _last(lib)
    assert call(l=2) == EUNSUP
    assert call(K=384) == EUNSUP and call(K=0) == EUNSUP and call(t=0, K=48) == EUNSUP
    assert call(T=-1) == EINVAL and call(N=-1) == EINVAL and call(N=0) == EINVAL
    assert call(T=2**24 + 1) == EUNSUP and call(N=2**24 + 1) == EUNSUP
    assert call(w=None) == EINVAL and call(ids=None) == EINVAL and call(o=None) == EINVAL
    assert call(ids=_far(1) + 4) == EALIGN and call(o=_far(2) + 8) == EALIGN
    assert call(wb=8 * 2 * 144 - 1) == EINVAL and call(ob=3 * 512 * 4 - 1) == EINVAL
    assert call(t=2, wb=256 + 8 * 2 * 208 - 1) == EINVAL      # repacked Q6_K needs its padding
    assert call(o=_far(0) + 8 * 2 * 144 - 16) == EINVAL and "overlaps" in _last(lib)
    assert call(o=_far(1) - 3 * 512 * 4 + 16) == EINVAL
    assert call(T=0, w=None, ids=None, o=None) == OK


def test_lora_add_refusals(lib):  # noqa: F811
    base = dict(t=1, A=_far(0), ab=BIG, B=_far(1), bb=BIG, E=4, R=8, sc=None, rk=None, x=_far(2), xb=BIG,
                ids=_far(3), b=_far(4), bbytes=BIG, ldb=96, o=_far(5), ob=BIG, ldo=96, M=3, N=96, K=64,
                ws=_far(6), wsb=BIG)

    def call(**kw):
        a = {**base, **kw}
        return lib.qmm_lora_add(a["t"], a["A"], a["ab"], a["B"], a["bb"], a["E"], a["R"], a["sc"], a["rk"], a["x"],
                                a["xb"], a["ids"], a["b"], a["bbytes"], a["ldb"], a["o"], a["ob"], a["ldo"], a["M"],
                                a["N"], a["K"], a["ws"], a["wsb"], None)

    assert call(t=3) == EUNSUP and "adapter type" in _last(lib)
    assert call(E=0) == EUNSUP and call(E=4097) == EUNSUP and call(R=0) == EUNSUP and call(R=257) == EUNSUP
    assert call(K=0) == EUNSUP and call(K=48) == EUNSUP and call(K=2**20 + 32) == EUNSUP
    assert call(M=-1) == EINVAL and call(N=-1) == EINVAL and call(M=2**24 + 1) == EUNSUP
    assert call(ldb=95) == EINVAL and "ld_base" in _last(lib)
    assert call(ldo=95) == EINVAL and call(ldo=2**32 + 1) == EUNSUP
    for p in ("A", "B", "x", "ids", "b", "o", "ws"):
        assert call(**{p: None}) == EINVAL, p
        assert call(**{p: base[p] + 4}) == EALIGN, p
    assert call(sc=A + 4) == EALIGN and call(rk=A + 8) == EALIGN
    assert call(ab=4 * 8 * 64 * 2 - 1) == EINVAL and call(bb=4 * 8 * 96 * 2 - 1) == EINVAL
    assert call(t=0, ab=4 * 8 * 64 * 4 - 1) == EINVAL
    assert call(xb=3 * 64 * 4 - 1) == EINVAL
    assert call(ldb=100, bbytes=(2 * 100 + 96) * 4 - 1) == EINVAL and "base holds" in _last(lib)
    assert call(ob=3 * 96 * 4 - 1) == EINVAL
    need = lib.qmm_lora_workspace_bytes(3, 8, 64, 4)
    assert need > 0 and call(wsb=need - 1) == EINVAL and "workspace" in _last(lib)
    # out may be base, not a shifted or differently strided part of it
    assert call(o=_far(4) + 16) == EINVAL and "overlaps base" in _last(lib)
    assert call(o=_far(4), ldo=100) == EINVAL
    assert call(o=_far(2)) == EINVAL and call(o=_far(0)) == EINVAL and call(o=_far(6)) == EINVAL
    for p in ("ids", "sc", "rk", "A", "B", "x", "b"):  # the workspace and out against each input
        other = {"sc": _far(7), "rk": _far(8)}.get(p, base[p])
        assert call(**{p: other, "ws": other}) == EINVAL and "overlaps" in _last(lib), p
        if p != "b":
            assert call(**{p: other, "o": other}) == EINVAL and "overlaps" in _last(lib), p
    assert call(M=0, A=None, x=None, ws=None) == OK and call(N=0, A=None, x=None, ws=None) == OK
    for bad in ((0, 8, 64, 4), (3, 0, 64, 4), (3, 8, 60, 4), (3, 8, 64, 0), (3, 257, 64, 4), (3, 8, 64, 4097)):
        assert lib.qmm_lora_workspace_bytes(*bad) == 0


def test_logprobs_refusals(lib):  # noqa: F811
    base = dict(t=0, x=_far(0), xb=BIG, ld=1000, M=3, V=1000, scale=1.0, mask=None, mb=0, mld=0, tok=_far(1), G=1,
                lp=_far(2), ent=_far(3), k=4, ti=_far(4), tl=_far(5), ws=_far(6), wsb=BIG)

    def call(**kw):
        a = {**base, **kw}
        return lib.qmm_logprobs(a["t"], a["x"], a["xb"], a["ld"], a["M"], a["V"], a["scale"], a["mask"], a["mb"],
                                a["mld"], a["tok"], a["G"], a["lp"], a["ent"], a["k"], a["ti"], a["tl"], a["ws"],
                                a["wsb"], None)

    assert call(t=3) == EUNSUP and "logit type" in _last(lib)
    assert call(M=-1) == EINVAL and call(V=-1) == EINVAL and call(V=0) == EINVAL
    assert call(M=2**23, xb=2**60) == EUNSUP and call(V=2**24 + 1) == EUNSUP
    for s in (0.0, -1.0, float("inf"), float("nan"), 2e30):
        assert call(scale=s) == EINVAL, s
    assert call(k=-1) == EUNSUP and call(k=65) == EUNSUP and call(G=-1) == EINVAL and call(G=2**31 // 3 + 1) == EUNSUP
    assert call(ld=999) == EINVAL and call(xb=3 * 1000 * 4 - 1) == EINVAL
    assert call(t=1, ld=1003, xb=(2 * 1003 + 1000) * 2 - 1) == EINVAL
    for p in ("x", "tok", "lp", "ti", "tl"):
        assert call(**{p: None}) == EINVAL, p
    for p in ("x", "tok", "lp", "ent", "ti", "tl"):
        assert call(**{p: base[p] + 4}) == EALIGN, p
    assert call(mask=A + 4, mb=BIG) == EALIGN
    assert call(mask=_far(7), mb=32 * 4 - 1) == EINVAL and call(mask=_far(7), mb=BIG, mld=31) == EINVAL
    assert call(mask=_far(7), mb=(2 * 40 + 32) * 4 - 1, mld=40) == EINVAL
    assert call(ent=_far(0) + 3 * 4000 - 16) == EINVAL and "overlaps" in _last(lib)
    need = lib.qmm_logprobs_workspace_bytes(3, 100000, 4)
    big = dict(V=100000, ld=100000)
    for o in ("lp", "ent", "ti", "tl"):  # against each input and the next output
        for i in ("x", "tok", "mask"):
            assert call(**{"mask": _far(7), "mb": BIG, o: _far(7) if i == "mask" else base[i]}) == EINVAL, (o, i)
            assert "overlaps an input" in _last(lib)
        nxt = {"lp": "ent", "ent": "ti", "ti": "tl", "tl": "lp"}[o]
        assert call(**{o: base[nxt]}) == EINVAL and "overlaps another" in _last(lib)
        assert call(ws=base[o], **big) == EINVAL and "overlaps" in _last(lib)
    for i in ("x", "tok"):
        assert call(ws=base[i], **big) == EINVAL and "overlaps an input" in _last(lib)
    assert need > 0 and call(wsb=need - 1, **big) == EINVAL and call(ws=None, **big) == EINVAL
    assert call(M=0, x=None, tok=None, lp=None, ti=None, tl=None, ws=None) == OK
    # many rows or a short vocabulary are not split: no workspace
    assert lib.qmm_logprobs_workspace_bytes(2000, 100000, 4) == 0 and lib.qmm_logprobs_workspace_bytes(1, 2048, 4) == 0
    assert lib.qmm_logprobs_workspace_bytes(3, 100000, 65) == 0 and lib.qmm_logprobs_workspace_bytes(0, 100000, 1) == 0


def test_mul_mat_logprobs_refusals(lib):  # noqa: F811
    base = dict(t=1, w=_far(0), wb=BIG, l=1, y=_far(1), yb=BIG, M=20, N=1001, K=512, scale=1.0, mask=None, mb=0, mld=0,
                tok=_far(2), G=1, lp=_far(3), ent=_far(4), k=4, ti=_far(5), tl=_far(6), ws=_far(7), wsb=BIG)

    def call(**kw):
        a = {**base, **kw}
        return lib.qmm_mul_mat_logprobs(a["t"], a["w"], a["wb"], a["l"], a["y"], a["yb"], a["M"], a["N"], a["K"],
                                        a["scale"], a["mask"], a["mb"], a["mld"], a["tok"], a["G"], a["lp"], a["ent"],
                                        a["k"], a["ti"], a["tl"], a["ws"], a["wsb"], None)

    bytes_ = lib.qmm_mul_mat_logprobs_workspace_bytes
    assert call(t=4) == EUNSUP and call(l=2) == EUNSUP and call(K=384) == EUNSUP
    assert call(M=-1) == EINVAL and call(N=0) == EINVAL and call(N=2**24 + 1) == EUNSUP
    assert call(scale=0.0) == EINVAL and call(k=65) == EUNSUP and call(G=-1) == EINVAL
    for p in ("w", "y", "tok", "lp", "ti", "tl", "ws"):
        assert call(**{p: None}) == EINVAL, p
        assert call(**{p: base[p] + 4}) == EALIGN, p
    assert call(wb=1001 * 2 * 144 - 1) == EINVAL and call(yb=20 * 2 * 292 - 1) == EINVAL
    assert call(mask=_far(8), mb=20 * 32 * 4 - 1, mld=32) == EINVAL
    # room for eight rows at least, or for all of fewer
    assert call(wsb=bytes_(8, 1001, 4) - 1) == EINVAL and "workspace" in _last(lib)
    assert call(M=3, wsb=bytes_(3, 1001, 4) - 1) == EINVAL
    assert call(lp=_far(7) + bytes_(20, 1001, 4) - 16) == EINVAL and "overlaps" in _last(lib)
    for p in ("w", "y", "tok"):
        assert call(ws=base[p]) == EINVAL and call(ent=base[p]) == EINVAL, p
    assert call(M=0, w=None, y=None, ws=None) == OK
    assert bytes_(8, 1001, 4) == 8 * bytes_(1, 1001, 4) >= 8 * 1001 * 4
    assert bytes_(0, 1001, 4) == 0 and bytes_(1, 0, 4) == 0 and bytes_(1, 1001, 65) == 0


def test_binding_refusals():
    """Shapes and types are checked before the library is called; CPU tensors are refused."""
    ids = torch.zeros(3, dtype=torch.int32)
    w = torch.zeros(8 * 144, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU tensor"):
        qmm.embed_rows("q4_K", w, ids, 8, 256)
    with pytest.raises(ValueError, match="int32"):
        qmm.embed_rows("q4_K", w, ids.long(), 8, 256)
    x, base = torch.zeros(3, 64), torch.zeros(3, 96)
    Aw, Bw = torch.zeros(4, 8, 64), torch.zeros(4, 96, 8)
    with pytest.raises(ValueError, match="GPU tensor"):
        qmm.lora_add(base, x, Aw, Bw, ids)
    for bad in (dict(x=x.half()), dict(x=torch.zeros(3, 65)), dict(Bw=Bw.half()), dict(Bw=torch.zeros(4, 95, 8)),
                dict(ids=ids.long()), dict(ids=ids[:2]), dict(base=base.half()), dict(scales=torch.zeros(3)),
                dict(ranks=torch.zeros(4))):
        a = dict(base=base, x=x, Aw=Aw, Bw=Bw, ids=ids, scales=None, ranks=None)
        a.update(bad)
        with pytest.raises(ValueError):
            qmm.lora_add(a["base"], a["x"], a["Aw"], a["Bw"], a["ids"], scales=a["scales"], ranks=a["ranks"])
    logits = torch.zeros(3, 1000)
    with pytest.raises(ValueError, match="GPU tensor"):
        qmm.logprobs(logits)
    for kw in (dict(tokens=ids[:2]), dict(tokens=ids.long()), dict(mask=torch.zeros(3, 31, dtype=torch.int32)),
               dict(mask=torch.zeros(2, 32, dtype=torch.int32)), dict(mask=torch.zeros(3, 32))):
        with pytest.raises(ValueError):
            qmm.logprobs(logits, **kw)
