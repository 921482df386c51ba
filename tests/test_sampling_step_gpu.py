"""Steps of sampling several answers to one prompt, end to end: head norms with
the rotation, the append to the cache, forks of the prompt's pages, and the
attention that reads them once; against the 64-bit references.  And the same in
training: the norms' gradients within a small attention."""
import numpy as np
import pytest
import torch

import synth
from exact_attention_94_gb300 import ops
from oracle import sampling
from oracle.fp8 import e4m3_decode
from tests.test_decode_shared_gpu import check, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("d,Hq,Hkv", [(64, 4, 2), (128, 8, 1)])
def test_answers_to_a_prompt(kv8, d, Hq, Hkv):
    P, pages, answers, prompt, eps = 16, 24, 3, 37, 1e-6
    plan = ops.rope_plan(d, [d // 2])
    axis, freq = list(plan.struct.axis[:d // 2]), list(plan.struct.inv_freq[:d // 2])
    g = torch.Generator().manual_seed(d)
    wq, wk = ((1 + 0.2 * torch.randn(d, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    if kv8:
        k, v = (torch.zeros((pages, Hkv, P, d), dtype=torch.uint8, device="cuda") for _ in range(2))
        ks, vs = (torch.zeros((pages, Hkv), device="cuda") for _ in range(2))
    else:
        k, v = (torch.zeros((pages, P, Hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pool = ops.PagePool(pages, P, answers + 1, 6)

    def step(seqs, position):
        """Appends a token of each; returns its queries."""
        n = len(seqs)
        qkv = torch.randn((n, (Hq + 2 * Hkv) * d), generator=g).to(torch.bfloat16).cuda()
        q, kn, vn = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], 1))
        qr, kr = ops.qk_norm_rope(q, kn, wq, wk, i32([[position] * n]), plan, eps=eps)
        for got, x, w in ((qr, q, wq), (kr, kn, wk)):
            want = sampling.qk_norm_rope(synth.to_f64(x), synth.to_f64(w), np.array([[position] * n]), axis, freq, False, eps)
            assert np.all(np.abs(synth.to_f64(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -15)
        page, slot, src = (x.cuda() for x in pool.reserve_append(seqs))
        if kv8:
            ops.kv8_append(kr, vn, k, v, ks, vs, page, slot, src)
        else:
            ops.paged_append(kr, vn.contiguous(), k, v, page, slot, src)
        return qr

    first = pool.add_seq()
    for t in range(prompt):
        step([first], t)
    seqs = [first] + [pool.fork(first) for _ in range(answers - 1)]
    shared = prompt // P * P if kv8 else prompt  # (a partly filled page's copies each have a scale of their own)
    for t in range(prompt, prompt + 20):
        q = step(seqs, t).unsqueeze(1)
        table, lens = pool.export()
        table, lens = table[seqs].contiguous(), lens[seqs].contiguous()
        assert lens.tolist() == [t + 1] * answers
        tail = (i32(table), i32(lens), i32([0, answers]), i32([shared]), 6 * P)
        if kv8:
            got = ops.decode_kv8_shared(q, k, v, ks, vs, *tail)
            kf, vf = (e4m3_decode(x.cpu().numpy()) * s.double().cpu().numpy()[:, :, None, None] for x, s in ((k, ks), (v, vs)))
            ref = sampling.decode_shared(synth.to_f64(q), lambda p, s: kf[p, :, s], lambda p, s: vf[p, :, s], table.numpy(),
                                         lens.tolist(), [0, answers], [shared], P, -1, d ** -0.5)
        else:
            got = ops.decode_paged_shared(q, k, v, *tail)
            kf, vf = synth.to_f64(k), synth.to_f64(v)
            ref = sampling.decode_shared(synth.to_f64(q), lambda p, s: kf[p, s], lambda p, s: vf[p, s], table.numpy(),
                                         lens.tolist(), [0, answers], [shared], P, -1, d ** -0.5)
        check(got, ref)
    assert ops.device_error() == 0


def test_a_captured_step():
    """Norms and attention of a step in one graph, replayed with other inputs."""
    B, Hq, Hkv, d, P = 4, 8, 2, 64, 16
    plan = ops.rope_plan(d, [d // 2])
    g = torch.Generator().manual_seed(1)
    new = lambda *size: torch.randn(size, generator=g).to(torch.bfloat16).cuda()
    k, v, wq, wk = new(20, P, Hkv, d), new(20, P, Hkv, d), new(d), new(d)
    table = i32([[0, 1, 2, 3 + 2 * b, 4 + 2 * b] for b in range(B)])
    tail = (i32([0, B]), i32([48]), 80)
    q, kn, pos, lens = new(B, Hq, d), new(B, Hkv, d), i32([[60] * B]), i32([61, 62, 70, 80])

    def step():
        qr, _ = ops.qk_norm_rope(q, kn, wq, wk, pos, plan)
        return ops.decode_paged_shared(qr.unsqueeze(1), k, v, table, lens, *tail)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for n in ([61, 62, 70, 80], [49, 48, 79, 0]):
        q.copy_(new(B, Hq, d)), lens.copy_(i32(n)), pos.fill_(n[0])
        graph.replay()
        want = step()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert ops.device_error() == 0


def test_gradients_through_an_attention():
    """Norms, rotation and the dense attention, forward and backward, against torch's derivatives in 64 bits."""
    B, N, H, d, eps = 1, 64, 2, 64, 1e-5
    plan = ops.rope_plan(d, [d // 2])
    axis, freq = list(plan.struct.axis[:d // 2]), list(plan.struct.inv_freq[:d // 2])
    g = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn((B, N, H, d), generator=g).to(torch.bfloat16).cuda() for _ in range(4))
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g)).cuda(), (1 + 0.2 * torch.randn(d, generator=g)).cuda()
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[None]
    qr, kr = ops.qk_norm_rope(q, k, wq, wk, pos, plan, eps=eps)
    o, lse = ops.fwd(qr, kr, v, causal=True)
    dqr, dkr, _ = ops.bwd(qr, kr, v, o, lse, do, causal=True)
    dq, dk, dwq, dwk = ops.qk_norm_rope_bwd(dqr, dkr, q, k, wq, wk, pos, plan, eps=eps)

    x = [t.double().requires_grad_() for t in (q, k, wq, wk)]
    angle = pos[0].double()[:, None] * torch.tensor(freq, dtype=torch.float64, device="cuda")
    co, si = angle.cos()[:, None], angle.sin()[:, None]

    def side(t, w):
        n = t * (t.square().mean(-1, keepdim=True) + eps).rsqrt() * w
        a, b = n.chunk(2, -1)
        return torch.cat([a * co - b * si, a * si + b * co], -1)

    s = torch.einsum("bihd,bjhd->bhij", side(x[0], x[2]), side(x[1], x[3])) * d ** -0.5
    s = s.masked_fill(torch.ones(N, N, device="cuda").triu(1).bool(), -torch.inf)
    torch.einsum("bhij,bjhd->bihd", s.softmax(-1), v.double()).backward(do.double())
    for got, leaf in ((dq, x[0]), (dk, x[1]), (dwq, x[2]), (dwk, x[3])):
        want = leaf.grad
        # every value on the way (q, k after the norms, O, dq, dk before them) is rounded to bf16, 2^-8 of itself, and
        # a score's derivative is a difference of such: 8 roundings of the gradient's norm at the very most
        assert (got.double() - want).norm() <= 8 * 2.0 ** -8 * want.norm()
