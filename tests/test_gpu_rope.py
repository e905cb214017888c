"""rope against the rotation in 64 bits.

Tolerance: sine and cosine are rounded to fp32 once (their angles are formed in 64 bits: at most 2^21 turns of 2^-53
each), one product is rounded, then the sum: 3 half steps of 2^-24 on |a c| + |b s| at most, plus 1e-9 of |a| + |b|
for the angle, plus half a step of the result's type."""
import numpy as np
import pytest
import torch

from kv_reference import TYPES, qmm, to_host

pytestmark = pytest.mark.gpu

STEP = {"f32": 0.0, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def reference(x, pos, rot, layout, base, freq_scale=1.0, ramp=None, magnitude=1.0, factors=None):
    x = np.asarray(x, np.float64)
    out, slack = x.copy(), np.zeros_like(x)
    for i in range(rot // 2):
        f = float(base) ** (-2.0 * i / rot)
        if factors is not None:
            f /= float(factors[i])
        r = 1.0 if ramp is None else min(1.0, max(0.0, (i - ramp[0]) / (ramp[1] - ramp[0])))
        th = (pos.astype(np.float64) * (f * (1 - r * (1 - freq_scale))))[:, None]
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = np.cos(th) * magnitude, np.sin(th) * magnitude
        out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        for e, u, v in ((a, c, s), (b, s, c)):
            slack[..., e] = 3 * 2.0 ** -24 * (np.abs(x[..., a] * u) + np.abs(x[..., b] * v)) + \
                1e-9 * abs(magnitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, slack


def check(kind, got, want, slack):
    got = to_host(got).astype(np.float64)
    tol = slack * (1 + STEP[kind]) + STEP[kind] * np.abs(want) + (2.0 ** -25 if kind == "f16" else 0.0)
    err = np.abs(got - want)
    assert (err <= tol).all(), (kind, err.max(), (err - tol).max())


def inputs(seed, T, H, D, kind, far):
    g = np.random.default_rng(seed)
    x = torch.from_numpy(g.standard_normal((T, H, D)).astype(np.float32) * 3).to(TYPES[kind])
    return x, g.integers(-far, far, T).astype(np.int32)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 2, 2), (1, 40, 128, 128), (3, 5, 80, 80), (7, 3, 96, 64), (2, 2, 64, 6),
                                       (5, 1, 33, 32), (300, 9, 128, 32), (2, 70, 1024, 1024), (1, 3, 250, 248)])
def test_sizes(T, H, D, rot, kind, layout):
    print(T, H, D, rot, kind, layout, flush=True)
    x, pos = inputs([1, T, D], T, H, D, kind, 10000)
    got = qmm.rope(x.cuda(), torch.from_numpy(pos).cuda(), rot=rot, layout=layout, base=500000.0)
    want, slack = reference(x.double().numpy(), pos, rot, layout, 500000.0)
    check(kind, got, want, slack)
    assert torch.equal(got.cpu()[..., rot:], x[..., rot:])


@pytest.mark.parametrize("kw", [dict(freq_scale=0.125), dict(freq_scale=1 / 16, ramp=(9.0, 20.0), magnitude=1.277),
                                dict(factors=True, magnitude=1.19), dict(freq_scale=0.0, ramp=(-3.0, 2.5)),
                                dict(factors=True, freq_scale=0.5, ramp=(0.0, 100.0), magnitude=-2.0)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_scaling_far_positions(kw, layout):
    print(kw, layout, flush=True)
    T, H, D, rot = 64, 3, 64, 48
    x, _ = inputs([2, T], T, H, D, "f32", 2)
    pos = np.random.default_rng(3).integers(-2**21, 2**21, T).astype(np.int32)
    pos[:4] = 2**21, -2**21, 0, 1000003
    kw = dict(kw)
    if kw.get("factors"):
        kw["factors"] = np.random.default_rng(4).uniform(1, 8, rot // 2).astype(np.float32)
    dev = {k: torch.from_numpy(v).cuda() if k == "factors" else v for k, v in kw.items()}
    got = qmm.rope(x.cuda(), torch.from_numpy(pos).cuda(), rot=rot, layout=layout, **dev)
    check("f32", got, *reference(x.double().numpy(), pos, rot, layout, 10000.0, **kw))


def test_stretched_context():
    x, pos = inputs(5, 40, 2, 64, "f32", 65536)
    kw = qmm.rope_ramp(64, 10000.0, 4096, 16.0)
    got = qmm.rope(x.cuda(), torch.from_numpy(pos).cuda(), **kw)
    check("f32", got, *reference(x.double().numpy(), pos, 64, "half", 10000.0, **kw))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_strides_and_places(kind, layout):
    """Column ranges of a projection's output, heads before tokens, odd strides; in place, beside itself, into a new one:
    all the same bits."""
    T, H, D, rot = 21, 4, 64, 32
    x, pos = inputs(6, T, H, D, kind, 5000)
    p = torch.from_numpy(pos).cuda()
    plain = qmm.rope(x.cuda(), p, rot=rot, layout=layout)
    for make in ("columns", "odd", "heads first"):
        print(kind, layout, make, flush=True)
        if make == "columns":
            wide = torch.full((T, 3 * H * D), 7.0, dtype=x.dtype, device="cuda")
            view = wide[:, H * D:2 * H * D].unflatten(1, (H, D))
        elif make == "odd":
            wide = torch.full((T, H * (D + 3) + 1), 7.0, dtype=x.dtype, device="cuda")
            view = wide.as_strided((T, H, D), (H * (D + 3) + 1, D + 3, 1))
        else:
            wide = torch.full((H, T, D), 7.0, dtype=x.dtype, device="cuda")
            view = wide.transpose(0, 1)
        view.copy_(x)
        assert torch.equal(qmm.rope(view, p, rot=rot, layout=layout), plain)
        if make == "columns":
            beside = wide[:, :H * D].unflatten(1, (H, D))
            qmm.rope(view, p, rot=rot, layout=layout, out=beside)
            assert torch.equal(beside, plain) and torch.equal(view.cpu(), x) and (wide[:, 2 * H * D:] == 7).all()
            with pytest.raises(qmm.QmmError, match="overlaps"):
                qmm.rope(view, p, out=wide[:, 64:64 + H * D].unflatten(1, (H, D)))
        before = wide.clone()
        assert qmm.rope(view, p, rot=rot, layout=layout, out=view) is view
        assert torch.equal(view, plain)
        view.copy_(x)
        assert torch.equal(wide, before)  # nothing beside the heads was touched


def test_back_and_forth():
    """Positions -p undo p: to the two rounded sums' steps (4 half steps of |a| + |b| each)."""
    x, pos = inputs(7, 50, 3, 128, "f32", 100000)
    p = torch.from_numpy(pos).cuda()
    back = to_host(qmm.rope(qmm.rope(x.cuda(), p), -p))
    pair = np.abs(x.numpy())
    pair = pair + np.roll(pair, 64, -1)
    assert (np.abs(back - x.numpy()) <= 8 * 2.0 ** -24 * 1.5 * pair).all()


def test_infinities_stay_in_their_pair():
    x, pos = inputs(8, 2, 2, 64, "f32", 100)
    clean = qmm.rope(x.cuda(), torch.from_numpy(pos).cuda())
    y = x.clone()
    y[0, 1, 5] = float("inf")
    y[1, 0, 40] = float("nan")
    got = qmm.rope(y.cuda(), torch.from_numpy(pos).cuda())
    for t, h, i in ((0, 1, 5), (1, 0, 8)):
        assert not torch.isfinite(got[t, h, [i, i + 32]]).any()
        got[t, h, [i, i + 32]] = clean[t, h, [i, i + 32]]
    assert torch.equal(got, clean)


def test_many_tokens_empty_stream_and_graph():
    for T, H in ((0, 4), (4, 0)):
        if H:
            assert qmm.rope(torch.zeros(T, H, 64, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")).shape == (T, H, 64)
    T, H, D = 5000, 2, 64
    x, pos = inputs(9, T, H, D, "f16", 4096)
    xd, p = x.cuda(), torch.from_numpy(pos).cuda()
    want = qmm.rope(xd, p)
    check("f16", want, *reference(x.double().numpy(), pos, D, "half", 10000.0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = qmm.rope(xd, p, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, want)
    out = torch.empty_like(xd)
    held = p.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        qmm.rope(xd, held, out=out)
    for rep in range(4):
        held.copy_(p if rep % 2 == 0 else p.flip(0))
        expect = qmm.rope(xd, held)
        out.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, expect), rep
