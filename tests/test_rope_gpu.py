"""fa_rope_axes against the reference rotation.

Tolerance per element: half a bf16 step of the result, 2^-8 |y|, plus what the
fp32 arithmetic may add before that rounding.  The angle is off by at most
2^-32 of a turn (its fixed point) and half an fp32 step of itself (2^-24 pi),
and the fast sine and cosine by 2^-21 on [-pi, pi]: together below 2^-20 of
each factor, so 2^-20 (|x1| + |x2|), doubled for the two products' own
roundings.
"""
import numpy as np
import pytest
import torch

import synth
from exact_attention_94_gb300 import ops
from oracle import serving

pytestmark = pytest.mark.gpu


def partner(x, neighbours):
    return x.reshape(*x.shape[:-1], -1, 2)[..., ::-1].reshape(x.shape) if neighbours else np.roll(x, x.shape[-1] // 2, -1)


def check(y, x, pos, axis, freq, neighbours, inverse=False):
    x64 = synth.to_f64(x)
    want = serving.rope_axes(x64, pos, axis, freq, neighbours, inverse)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * (np.abs(x64) + np.abs(partner(x64, neighbours)))
    err = np.abs(synth.to_f64(y) - want)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-30)).max())


def bf(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def plan_lists(d, kind):
    half = d // 2
    if kind == "one":
        return [0] * half, [10000.0 ** (-p / half) for p in range(half)]
    if kind == "three":
        n = [half // 4, half // 4, half // 4]  # a quarter is copied
        return [a for a in range(3) for _ in range(n[a])] + [-1] * (half - sum(n)), \
               [10000.0 ** (-j / n[a]) for a in range(3) for j in range(n[a])] + [0.0] * (half - sum(n))
    rng = np.random.default_rng(d)
    return rng.integers(-1, 4, half).tolist(), (rng.standard_normal(half) * 40).tolist()  # axes in any order, any sign


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("kind", ["one", "three", "any"])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (3, 8, 2), (129, 5, 0), (67, 0, 3), (2000, 32, 8)])
def test_forward_and_gradient(d, neighbours, kind, T, Hq, Hkv):
    axis, freq = plan_lists(d, kind)
    plan = ops.RopePlan(d, axis, freq, neighbours)
    rng = np.random.default_rng(T)
    pos = rng.integers(-5000, 2 ** 20, (plan.n_axes, T))
    p = torch.tensor(pos, dtype=torch.int32).cuda()
    q, k = (bf((T, H, d), s) if H else None for s, H in ((1, Hq), (2, Hkv)))
    for inverse, f in ((False, ops.rope_axes), (True, ops.rope_axes_bwd)):
        for x, y in zip((q, k), f(q, k, p, plan)):
            if x is None:
                assert y is None
            else:
                check(y, x, pos, axis, freq, neighbours, inverse)


def test_far_positions_lose_nothing():
    d, T = 128, 7
    axis, freq = plan_lists(d, "one")
    pos = np.array([[0, 1, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31, -1]])
    plan = ops.RopePlan(d, axis, freq)
    q = bf((T, 2, d), 3)
    y, _ = ops.rope_axes(q, None, torch.tensor(pos, dtype=torch.int32).cuda(), plan)
    # position times frequency in float64 is itself off by half a step: 2^31 * 2^-53
    # radians, far below the tolerance
    check(y, q, pos, axis, freq, False)


def test_slices_of_a_projection_in_place_and_four_dimensions():
    d, B, N, Hq, Hkv = 128, 2, 33, 4, 2
    plan = ops.rope_plan(d, [64])
    axis, freq = plan_lists(d, "one")
    pos = np.tile(np.arange(N), B)[None]
    p = torch.tensor(pos, dtype=torch.int32).cuda()
    qkv = bf((B, N, (Hq + 2 * Hkv) * d), 4)
    was = qkv.clone()
    q, k = qkv[..., :Hq * d].unflatten(-1, (Hq, d)), qkv[..., Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d))
    q0, k0 = q.clone().reshape(-1, Hq, d), k.clone().reshape(-1, Hkv, d)
    oq, ok = ops.rope_axes(q, k, p, plan)
    assert torch.equal(qkv, was) and oq.shape == q.shape and oq.is_contiguous()
    check(oq.reshape(-1, Hq, d), q0, pos, axis, freq, False)
    check(ok.reshape(-1, Hkv, d), k0, pos, axis, freq, False)
    ops.rope_axes(q, k, p, plan, out=(q, k))
    assert torch.equal(q, oq) and torch.equal(k, ok)
    assert torch.equal(qkv[..., (Hq + Hkv) * d:], was[..., (Hq + Hkv) * d:])  # the values stay


def test_copied_pairs_keep_infinities_and_nan():
    d = 64
    plan = ops.rope_plan(d, [8])
    x = bf((4, 2, d), 5)
    x[:, :, 20] = float("inf")
    x[:, :, 25] = float("nan")
    y, _ = ops.rope_axes(x, None, torch.arange(4, dtype=torch.int32, device="cuda")[None], plan)
    same = list(range(8, 32)) + list(range(40, 64))
    assert torch.equal(y[..., same].view(torch.int16), x[..., same].view(torch.int16))
    assert torch.isfinite(y[..., :8]).all()


def test_empty_and_refusals():
    plan = ops.rope_plan(64, [32])
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    y, _ = ops.rope_axes(e, None, torch.empty((1, 0), dtype=torch.int32, device="cuda"), plan)
    assert y.shape == e.shape
    x, p = bf((4, 2, 64), 6), torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    for bad in (lambda: ops.rope_axes(x.transpose(0, 1), None, p, plan),            # heads not side by side
                lambda: ops.rope_axes(x[:1].expand(4, 2, 64), None, p, plan),       # rows on top of each other
                lambda: ops.rope_axes(x, None, p[:, :3], plan),
                lambda: ops.rope_axes(x, None, p.long(), plan),
                lambda: ops.rope_axes(x, bf((5, 2, 64), 7), p, plan),
                lambda: ops.rope_axes(x, None, p, ops.rope_plan(128, [64])),
                lambda: ops.rope_axes(x, None, p, plan, out=(x[:, :1], None)),
                lambda: ops.rope_axes(None, None, p, plan)):
        with pytest.raises(ValueError):
            bad()


def test_a_gradient_by_differences():
    """<rope(x), g> moves by <rope_bwd(g), e> when x moves by e: exact up to roundings, the map being linear."""
    d, T, H = 64, 9, 3
    axis, freq = plan_lists(d, "three")
    plan = ops.RopePlan(d, axis, freq, True)
    pos = torch.randint(0, 100000, (3, T), generator=torch.Generator().manual_seed(8)).to(torch.int32).cuda()
    x, g = bf((T, H, d), 9), bf((T, H, d), 10)
    y, _ = ops.rope_axes(x, None, pos, plan)
    dx, _ = ops.rope_axes_bwd(g, None, pos, plan)
    a, b = (synth.to_f64(y) * synth.to_f64(g)).sum((1, 2)), (synth.to_f64(x) * synth.to_f64(dx)).sum((1, 2))
    size = (np.abs(synth.to_f64(y) * synth.to_f64(g))).sum((1, 2)) + (np.abs(synth.to_f64(x) * synth.to_f64(dx))).sum((1, 2))
    assert np.all(np.abs(a - b) <= 2.0 ** -8 * 1.01 * size)


@pytest.mark.parametrize("sections", [[32, 0, 0], [16, 16, 0], [0, 20, 0], [0, 0, 0]])
def test_axes_without_pairs(sections):
    """Positions have a row for each section, empty or not; the last empty ones' may be left out."""
    d, T = 64, 50
    plan = ops.rope_plan(d, sections)
    axis, freq = list(plan.struct.axis[:d // 2]), list(plan.struct.inv_freq[:d // 2])
    x = bf((T, 3, d), 11)
    pos = np.random.default_rng(1).integers(0, 5000, (3, T))
    p = torch.tensor(pos, dtype=torch.int32).cuda()
    for n in range(plan.used_axes, 4):
        for f, inverse in ((ops.rope_axes, False), (ops.rope_axes_bwd, True)):
            y, _ = f(x, None, p[:n].contiguous(), plan)
            check(y, x, pos, axis, freq, False, inverse)
    for bad in (p[:plan.used_axes - 1].contiguous(), torch.cat([p, p[:1]]), p[0].contiguous()):
        with pytest.raises(ValueError):
            ops.rope_axes(x, None, bad, plan)
