"""The serving-step operators together, as a server uses them: prompts, then
steps of one token, then drafts, each step planned on the GPU, rotated, written
to the 8-bit cache and attended, against the same steps in the reference."""
import math

import numpy as np
import pytest
import torch

import synth
from exact_attention_94_gb300 import ops
from oracle import paged as PG
from oracle import serving
from tests.test_decode_kv8_gpu import assert_close
from tests.test_kv8_append_gpu import same_codes

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


@pytest.mark.parametrize("d,P", [(64, 16), (128, 32)])
def test_prompts_steps_and_drafts(d, P):
    B, Hq, Hkv, blocks, pages, cap = 3, 4, 2, 12, 30, 160
    half = d // 2
    plan = ops.rope_plan(d, [half // 4, half // 4, half // 2])
    axis, freq = list(plan.struct.axis[:half]), list(plan.struct.inv_freq[:half])
    g = torch.Generator().manual_seed(d)
    free, count = i32(np.random.default_rng(1).permutation(pages)), i32([pages])
    lens, table = i32([0] * B), i32(np.zeros((B, blocks)))
    kc, vc = (torch.full((pages, Hkv, P, d), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.full((pages, Hkv), math.nan, device="cuda") for _ in range(2))
    r = [(x.cpu().numpy().copy(), s.cpu().numpy().copy()) for x, s in ((kc, ks), (vc, vs))]
    r_lens, r_count, r_table = [0] * B, pages, np.zeros((B, blocks), np.int64)
    steps = [[70, 1, 33]] + [[1] * B] * 3 + [[4] * B] + [[0, 9, 1]] + [[1] * B] * 2
    for n in steps:
        p = ops.page_plan(lens, i32(n), free, count, table, P, cap)
        lens, count = p.seq_lens, p.free_count
        total = sum(n)
        qkv = torch.randn((cap, (Hq + 2 * Hkv) * d), generator=g).to(torch.bfloat16).cuda()
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
        pos = torch.stack([p.position, p.position // 3, p.position % 7])
        qr, kr = ops.rope_axes(q, k, pos, plan)
        ops.kv8_append(kr, v, kc, vc, ks, vs, p.page, p.slot)

        r_lens, cu, page, slot, position, r_count, r_table = serving.page_plan(r_lens, n, free.tolist(), r_count, r_table, P, cap)
        assert p.page.tolist() == page and p.slot.tolist() == slot and lens.tolist() == r_lens
        rp = np.array([position, [x // 3 for x in position], [x % 7 for x in position]])
        for got, x in ((qr, q), (kr, k)):
            want = serving.rope_axes(synth.to_f64(x), rp, axis, freq, False)
            assert np.all(np.abs(synth.to_f64(got) - want)[:total] <= 2.0 ** -8 * np.abs(want)[:total] + 2.0 ** -15)
        for x, (c, s) in ((kr, r[0]), (v, r[1])):   # the rotated keys as the GPU rounded them
            serving.kv8_append(synth.to_f64(x), c, s, page, slot)
        for x, s, (c, t) in ((kc, ks, r[0]), (vc, vs, r[1])):
            same_codes(x, c)
            assert np.array_equal(s.cpu().numpy(), t, equal_nan=True)

        if min(n) == max(n):                        # a step: every request's tokens attend
            o, lse = ops.decode_kv8(qr[:total].reshape(B, n[0], Hq, d), kc, vc, ks, vs, table, lens, blocks * P)
            qn = synth.to_f64(qr[:total]).reshape(B, n[0], Hq, d)
            assert_close(o, lse, serving.decode_kv8(qn, r[0][0], r[1][0], r[0][1], r[1][1], r_table, r_lens, -1, d ** -0.5))
    assert ops.device_error() == 0


def test_the_plan_feeds_the_bf16_cache_too():
    """page and slot of a plan without padding are what fa_paged_append takes."""
    P, pages, Hkv, d, B = 16, 12, 2, 64, 3
    free, count, lens, table = i32(range(pages)), i32([pages]), i32([0] * B), i32(np.zeros((B, 4)))
    kp = torch.zeros((pages, P, Hkv, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    rk, rv = np.zeros(kp.shape), np.zeros(kp.shape)
    g = torch.Generator().manual_seed(2)
    for n in ([17, 3, 16], [1, 1, 1], [1, 14, 1]):
        p = ops.page_plan(lens, i32(n), free, count, table, P, sum(n))
        lens, count = p.seq_lens, p.free_count
        kn, vn = (torch.randn((sum(n), Hkv, d), generator=g).to(torch.bfloat16) for _ in range(2))
        ops.paged_append(kn.cuda(), vn.cuda(), kp, vp, p.page, p.slot, torch.full_like(p.page, -1))
        for i, (pg, sl) in enumerate(zip(p.page.tolist(), p.slot.tolist())):
            PG.apply_append(rk, rv, pg, sl, -1, synth.to_f64(kn[i]), synth.to_f64(vn[i]))
    assert np.array_equal(synth.to_f64(kp), rk) and np.array_equal(synth.to_f64(vp), rv)
    q = torch.randn((B, 1, Hkv, d), generator=g).to(torch.bfloat16).cuda()
    o, lse = ops.decode_paged(q, kp, vp, table, lens, 64)
    assert torch.isfinite(o.float()).all() and ops.device_error() == 0


def test_the_host_pool_feeds_the_8_bit_cache():
    """Slots and copies from PagePool.reserve_append, forks among them."""
    P, pages, Hkv, d = 16, 16, 2, 64
    rng = np.random.default_rng(3)
    pool = ops.PagePool(pages, P, 4, 6)
    kc = torch.zeros((pages, Hkv, P, d), dtype=torch.uint8, device="cuda")
    vc, ks = kc.clone(), torch.zeros((pages, Hkv), device="cuda")
    vs = ks.clone()
    r = [(x.cpu().numpy().copy(), s.cpu().numpy().copy()) for x, s in ((kc, ks), (vc, vs))]

    def step(seqs):
        page, slot, src = pool.reserve_append(seqs)
        x = torch.tensor(rng.standard_normal((2, len(seqs), Hkv, d)) * 2.0 ** rng.integers(-3, 4)).to(torch.bfloat16)
        ops.kv8_append(x[0].cuda(), x[1].cuda(), kc, vc, ks, vs, page.cuda(), slot.cuda(), src.cuda())
        for y, (c, s) in zip(x, r):
            serving.kv8_append(synth.to_f64(y), c, s, page.tolist(), slot.tolist(), src.tolist())

    a = pool.add_seq()
    for _ in range(21):
        step([a])
    b = pool.fork(a)
    c = pool.fork(a)
    for t in range(20):
        step([[a, b, c], [c, a, b]][t % 2])
    for (x, s), (y, t) in zip(((kc, ks), (vc, vs)), r):
        same_codes(x, y)
        assert np.array_equal(s.cpu().numpy(), t)
    assert ops.device_error() == 0
