"""fa_qk_norm_rope and its gradient against the reference in 64 bits.

Tolerances.  Forward: half a bf16 step of the result, 2^-8 |y|, and what the
fp32 arithmetic adds before: the squares' sum has 19 roundings of 2^-24, rsqrt
2 ulp, the factors three more roundings, sine and cosine 2 ulp and an angle
rounded to fp32, together below 2^-20 of each product; two products, so 2^-19
(|w n| + |partner's|).
Gradient: with S = |dy| + |partner's| and u = w g, errors of u are below 2^-20
w S, those of mean(u n) below 2^-19 mean(w S |n|), so 2^-18 r (w S + |n| mean(w S
|n|)) and 2^-8 |dx|.  dw: 2^-19 of sum |S n| for the terms, and 2^-24 for each
addition that a term passes through: the rows of a thread and 45 more (16 heads
a block at a time, then lanes, warps and blocks in threads of 32, all counted
at their most).
"""
import numpy as np
import pytest
import torch

import synth
from exact_attention_94_gb300 import _lib, ops
from oracle import sampling
from tests.test_rope_gpu import bf, partner, plan_lists

pytestmark = pytest.mark.gpu
EPS = 1e-6


def weights(d, seed, wide):
    w = 1 + 0.3 * torch.randn(d, generator=torch.Generator().manual_seed(seed))
    return (w if wide else w.to(torch.bfloat16)).cuda()


def f64(w):
    return w.double().cpu().numpy()


def check_fwd(y, x, w, pos, axis, freq, nb, eps=EPS):
    x64, w64 = synth.to_f64(x), f64(w)
    want = sampling.qk_norm_rope(x64, w64, pos, axis, freq, nb, eps)
    wn = np.abs(sampling.norm(x64, eps)[0] * w64)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * (wn + partner(wn, nb)) + 1e-38
    err = np.abs(synth.to_f64(y) - want)
    assert np.all(err <= tol), float((err / tol).max())


def rows_per_thread(T, H, others, d):
    """Heads that a thread of the gradient adds up, at most."""
    blocks = _lib.load().fa_qk_norm_rope_bwd_workspace_bytes(T, H, others, d) // (4 * d) - 64 // d - 1
    return T * H / (128 // (d // 16) * max(1.0, blocks * H / (H + others) - 2)) + 8


def check_bwd(dx, dw, dy, x, w, pos, axis, freq, nb, others, eps=EPS):
    x64, g64, w64 = synth.to_f64(x), synth.to_f64(dy), f64(w)
    want, want_w = sampling.qk_norm_rope_bwd(g64, x64, w64, pos, axis, freq, nb, eps)
    n, r = sampling.norm(x64, eps)
    S = np.abs(g64) + np.abs(partner(g64, nb))
    wS = np.abs(w64) * S
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * r * (wS + np.abs(n) * (wS * np.abs(n)).mean(-1, keepdims=True)) + 1e-38
    err = np.abs(synth.to_f64(dx) - want)
    assert np.all(err <= tol), float((err / tol).max())
    T, H, d = x64.shape
    tol = (2.0 ** -19 + 2.0 ** -24 * (rows_per_thread(T, H, others, d) + 45)) * (S * np.abs(n)).sum((0, 1)) + 1e-38
    err = np.abs(f64(dw) - want_w)
    assert dw.dtype == torch.float32 and np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nb", [False, True])
@pytest.mark.parametrize("kind", ["one", "three", "any"])
@pytest.mark.parametrize("T,Hq,Hkv,wide", [(1, 1, 1, 0), (3, 8, 2, 1), (129, 5, 0, 0), (67, 0, 3, 1), (700, 14, 2, 0)])
def test_forward_and_gradient(d, nb, kind, T, Hq, Hkv, wide):
    axis, freq = plan_lists(d, kind)
    plan = ops.RopePlan(d, axis, freq, nb)
    pos = np.random.default_rng(T).integers(-5000, 2 ** 20, (plan.n_axes, T))
    p = torch.tensor(pos, dtype=torch.int32).cuda()
    q, k, dyq, dyk = (bf((T, H, d), s) if H else None for s, H in enumerate((Hq, Hkv, Hq, Hkv)))
    wq, wk = (weights(d, s, wide) if H else None for s, H in ((5, Hq), (6, Hkv)))
    y = ops.qk_norm_rope(q, k, wq, wk, p, plan, EPS)
    g = ops.qk_norm_rope_bwd(dyq, dyk, q, k, wq, wk, p, plan, EPS)
    for i, (x, dy, w, others) in enumerate(((q, dyq, wq, Hkv), (k, dyk, wk, Hq))):
        if x is None:
            assert y[i] is None and g[i] is None and g[2 + i] is None
        else:
            check_fwd(y[i], x, w, pos, axis, freq, nb)
            check_bwd(g[i], g[2 + i], dy, x, w, pos, axis, freq, nb, others)


@pytest.mark.parametrize("T,H", [(20000, 1), (3001, 40)])
def test_many_rows(T, H):
    """Threads with eight heads, and blocks with many rounds."""
    d = 64
    axis, freq = plan_lists(d, "one")
    plan = ops.RopePlan(d, axis, freq)
    pos = np.arange(T)[None]
    p = torch.tensor(pos, dtype=torch.int32).cuda()
    x, dy, w = bf((T, H, d), 1), bf((T, H, d), 2), weights(d, 3, False)
    check_fwd(ops.qk_norm_rope(x, None, w, None, p, plan, EPS)[0], x, w, pos, axis, freq, False)
    dx, _, dw, _ = ops.qk_norm_rope_bwd(dy, None, x, None, w, None, p, plan, EPS)
    check_bwd(dx, dw, dy, x, w, pos, axis, freq, False, 0)
    again = ops.qk_norm_rope_bwd(dy, None, x, None, w, None, p, plan, EPS)
    assert torch.equal(again[0], dx) and torch.equal(again[2], dw)  # the same bits


@pytest.mark.parametrize("size,eps", [(2.0 ** 100, 1e-6), (2.0 ** -60, 0.0), (2.0 ** -60, 1e-30), (2.0 ** -60, 1e-6), (1e-3, 1e-6)])
def test_sizes_whose_squares_leave_fp32(size, eps):
    d, T, H = 128, 5, 3
    axis, freq = plan_lists(d, "one")
    plan = ops.RopePlan(d, axis, freq)
    pos = np.arange(T)[None]
    p = torch.tensor(pos, dtype=torch.int32).cuda()
    x, w = (bf((T, H, d), 1).float() * size).to(torch.bfloat16), weights(d, 3, True)
    dy = (bf((T, H, d), 2).float() * min(size, 1.0)).to(torch.bfloat16)
    check_fwd(ops.qk_norm_rope(x, None, w, None, p, plan, eps)[0], x, w, pos, axis, freq, False, eps)
    dx, _, dw, _ = ops.qk_norm_rope_bwd(dy, None, x, None, w, None, p, plan, eps)
    check_bwd(dx, dw, dy, x, w, pos, axis, freq, False, 0, eps)


def test_rows_with_an_infinity_leave_the_others():
    d = 64
    plan = ops.rope_plan(d, [8])
    x, w, p = bf((4, 2, d), 5), weights(d, 3, False), torch.arange(4, dtype=torch.int32, device="cuda")[None]
    plain = ops.qk_norm_rope(x, None, w, None, p, plan)[0]
    x[1, 1, 20] = float("inf")
    x[2, 0, 3] = float("nan")
    y = ops.qk_norm_rope(x, None, w, None, p, plan)[0]
    fine = torch.ones((4, 2), dtype=torch.bool)
    fine[1, 1] = fine[2, 0] = False
    assert torch.equal(y[fine], plain[fine])
    assert torch.isnan(y[1, 1, 20]) and y[1, 1].float().nan_to_num().abs().sum() == 0  # r = 0
    assert torch.isnan(y[2, 0]).all()


def test_slices_of_a_projection_in_place():
    d, B, N, Hq, Hkv = 128, 2, 33, 4, 2
    axis, freq = plan_lists(d, "one")
    plan = ops.RopePlan(d, axis, freq)
    pos = np.tile(np.arange(N), B)[None]
    p = torch.tensor(pos, dtype=torch.int32).cuda()
    qkv, wq, wk = bf((B, N, (Hq + 2 * Hkv) * d), 4), weights(d, 5, False), weights(d, 6, False)
    was = qkv.clone()
    q, k = qkv[..., :Hq * d].unflatten(-1, (Hq, d)), qkv[..., Hq * d:(Hq + Hkv) * d].unflatten(-1, (Hkv, d))
    q0, k0 = q.clone().reshape(-1, Hq, d), k.clone().reshape(-1, Hkv, d)
    yq, yk = ops.qk_norm_rope(q, k, wq, wk, p, plan)
    assert torch.equal(qkv, was) and yq.shape == q.shape and yq.is_contiguous()
    check_fwd(yq.reshape(-1, Hq, d), q0, wq, pos, axis, freq, False)
    check_fwd(yk.reshape(-1, Hkv, d), k0, wk, pos, axis, freq, False)
    dyq, dyk = bf(q.shape, 7), bf(k.shape, 8)
    g = ops.qk_norm_rope_bwd(dyq, dyk, q, k, wq, wk, p, plan)
    for outs in ((dyq.clone(), dyk.clone()), (q, k)):  # over the gradients, and over the inputs
        qkv.copy_(was)
        dy = outs if outs[0] is not q else (dyq, dyk)
        h = ops.qk_norm_rope_bwd(*dy, q, k, wq, wk, p, plan, out=outs)
        assert h[0] is outs[0] and all(torch.equal(a, b) for a, b in zip(g, h))
    qkv.copy_(was)
    ops.qk_norm_rope(q, k, wq, wk, p, plan, out=(q, k))
    assert torch.equal(q, yq) and torch.equal(k, yk)
    assert torch.equal(qkv[..., (Hq + Hkv) * d:], was[..., (Hq + Hkv) * d:])  # the values stay


def test_norm_alone_is_the_norm():
    d = 64
    plan = ops.RopePlan(d, [-1] * 32, [0.0] * 32)
    x, w = bf((9, 3, d), 1), weights(d, 2, True)
    p = torch.zeros((1, 9), dtype=torch.int32, device="cuda")
    check_fwd(ops.qk_norm_rope(x, None, w, None, p, plan)[0], x, w, np.zeros((1, 9)), [-1] * 32, [0.0] * 32, False)


def test_gradients_by_differences():
    """The loss <y, c> in 64 bits moves by <dx, e> and <dw, e>: central differences with h = 2^-12,
    whose own error is h^2 of a third derivative, below 2^-20 here."""
    d, T, H = 64, 5, 3
    axis, freq = plan_lists(d, "three")
    plan = ops.RopePlan(d, axis, freq, True)
    pos = np.random.default_rng(8).integers(0, 100000, (3, T))
    x, c, w = bf((T, H, d), 9), bf((T, H, d), 10), weights(d, 11, True)
    dx, _, dw, _ = ops.qk_norm_rope_bwd(c, None, x, None, w, None, torch.tensor(pos, dtype=torch.int32).cuda(), plan, EPS)
    x64, c64, w64 = synth.to_f64(x), synth.to_f64(c), f64(w)
    rng, h = np.random.default_rng(1), 2.0 ** -12
    loss = lambda x, w: (sampling.qk_norm_rope(x, w, pos, axis, freq, True, EPS) * c64).sum()
    for _ in range(8):
        e, ew = rng.standard_normal(x64.shape), rng.standard_normal(d)
        a = (loss(x64 + h * e, w64) - loss(x64 - h * e, w64)) / (2 * h)
        b = (synth.to_f64(dx) * e).sum()
        assert abs(a - b) <= 2.0 ** -8 * 1.1 * np.abs(synth.to_f64(dx) * e).sum() + 2.0 ** -10
        a = (loss(x64, w64 + h * ew) - loss(x64, w64 - h * ew)) / (2 * h)
        assert abs(a - (f64(dw) * ew).sum()) <= 2.0 ** -16 * np.abs(c64).sum()


def test_empty_streams_and_graphs():
    d, T = 128, 300
    plan = ops.rope_plan(d, [64])
    w = weights(d, 1, False)
    e = torch.empty((0, 2, d), dtype=torch.bfloat16, device="cuda")
    p0 = torch.empty((1, 0), dtype=torch.int32, device="cuda")
    assert ops.qk_norm_rope(e, None, w, None, p0, plan)[0].shape == e.shape
    dx, _, dw, _ = ops.qk_norm_rope_bwd(e, None, e, None, w, None, p0, plan)
    assert dx.shape == e.shape and not dw.any()
    x, dy, p = bf((T, 6, d), 2), bf((T, 6, d), 3), torch.arange(T, dtype=torch.int32, device="cuda")[None]
    y, g = ops.qk_norm_rope(x, None, w, None, p, plan)[0], ops.qk_norm_rope_bwd(dy, None, x, None, w, None, p, plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    h = ops.qk_norm_rope_bwd(dy, None, x, None, w, None, p, plan, stream=s)
    s.synchronize()
    assert torch.equal(h[0], g[0]) and torch.equal(h[2], g[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yy, gg = ops.qk_norm_rope(x, None, w, None, p, plan)[0], ops.qk_norm_rope_bwd(dy, None, x, None, w, None, p, plan)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(yy, y) and torch.equal(gg[0], g[0]) and torch.equal(gg[2], g[2])


def test_refusals():
    plan = ops.rope_plan(64, [32])
    x, w, p = bf((4, 2, 64), 6), weights(64, 1, False), torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    for bad in (lambda: ops.qk_norm_rope(x.transpose(0, 1), None, w, None, p, plan),
                lambda: ops.qk_norm_rope(x, None, w[:32], None, p, plan),
                lambda: ops.qk_norm_rope(x, None, w.cpu(), None, p, plan),
                lambda: ops.qk_norm_rope(x, x, w, w.float(), p, plan),
                lambda: ops.qk_norm_rope(x, None, w, None, p[:, :3], plan),
                lambda: ops.qk_norm_rope(x, None, w, None, p.long(), plan),
                lambda: ops.qk_norm_rope(x, bf((5, 2, 64), 7), w, w, p, plan),
                lambda: ops.qk_norm_rope(None, None, None, None, p, plan),
                lambda: ops.qk_norm_rope(x, None, w, None, p, ops.rope_plan(128, [64])),
                lambda: ops.qk_norm_rope_bwd(None, None, x, None, w, None, p, plan),
                lambda: ops.qk_norm_rope_bwd(x[:3], None, x, None, w, None, p, plan),
                lambda: ops.qk_norm_rope_bwd(x, None, x, None, w, None, p, plan, workspace=torch.empty(8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ops.qk_norm_rope(x.float(), None, w, None, p, plan), lambda: ops.qk_norm_rope(x, None, w.half(), None, p, plan),
                lambda: ops.qk_norm_rope(x, None, w, None, p, None), lambda: ops.qk_norm_rope(x, None, None, None, p, plan)):
        with pytest.raises(TypeError):
            bad()
    for eps in (-1e-6, float("nan"), float("inf")):
        with pytest.raises(_lib.FaError):
            ops.qk_norm_rope(x, None, w, None, p, plan, eps)
