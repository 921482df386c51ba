"""Guard bands around what the serving-step operators write, as in
test_canary_gpu.py: outputs, caches and workspaces lie inside sentinel-filled
buffers; every byte outside them stays, and they hold what the plain call gives.
Sizes are ragged, batches padded, pages partly filled, shares cut everywhere."""
import math

import numpy as np
import pytest
import torch

from exact_attention_94_gb300 import _lib, ops
from tests.test_canary_gpu import Guarded, _p, _s, _same
from tests.test_decode_kv8_gpu import dev, make

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


@pytest.mark.parametrize("cap", [37, 5003])
def test_page_plan(cap):
    B, P, pages, blocks = 7, 16, 800, 330
    rng = np.random.default_rng(cap)
    new = i32(rng.multinomial(cap - 5, np.ones(B) / B))
    free, count, ctx = i32(rng.permutation(pages)), i32([pages]), i32([0] * B)
    plain_table = i32(np.full((B, blocks), -7))
    plain = ops.page_plan(ctx, new, free, count, plain_table, P, cap)
    g = [Guarded((n,), torch.int32, 16 * i) for i, n in enumerate((B, B + 1, cap, cap, cap, 1))]
    table = Guarded((B, blocks), torch.int32)
    table.t.fill_(-7)
    ops.page_plan(ctx, new, free, count, table.t, P, cap, out=ops.PagePlan(*(x.t for x in g)))
    for x, y, name in zip(g, plain, ops.PagePlan._fields):
        x.check(name)
        _same(x.t, y, name)
    table.check("block_table")
    _same(table.t, plain_table, "block_table")
    assert ops.device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (67, 5, 1), (1000, 17, 3)])
def test_rope(d, T, Hq, Hkv):
    plan = ops.rope_plan(d, [d // 8, d // 8, d // 4])
    q, k = (torch.randn((T, H, d), device="cuda").to(torch.bfloat16) for H in (Hq, Hkv))
    pos = torch.randint(0, 9999, (3, T), device="cuda", dtype=torch.int32)
    plain = ops.rope_axes(q, k, pos, plan)
    gq, gk = Guarded(q.shape, torch.bfloat16), Guarded(k.shape, torch.bfloat16, 16)
    ops.rope_axes(q, k, pos, plan, out=(gq.t, gk.t))
    gq.check("q"), gk.check("k")
    _same(gq.t, plain[0], "q"), _same(gk.t, plain[1], "k")


@pytest.mark.parametrize("d,Hkv,P", [(64, 3, 16), (128, 2, 48)])
def test_append(d, Hkv, P):
    pages = 6
    page = [0] * P + [5] * 3 + [-1] * 2 + [2] * (P - 1)
    slot = list(range(P)) + [P - 3, P - 2, P - 1] + [-1] * 2 + list(range(1, P))
    n = len(page)
    x = torch.randn((2, n, Hkv, d), device="cuda").to(torch.bfloat16)
    side = []
    for shift in (0, 16):
        c = Guarded((pages, Hkv, P, d), torch.uint8, shift)
        s = Guarded((pages, Hkv), torch.float32, shift)
        c.t.copy_(torch.randint(0, 127, c.t.shape, device="cuda").to(torch.uint8))
        s.t.fill_(0.25)
        side.append((c, s, c.t.clone(), s.t.clone()))
    (kc, ks, kc2, ks2), (vc, vs, vc2, vs2) = side
    ops.kv8_append(x[0], x[1], kc.t, vc.t, ks.t, vs.t, i32(page), i32(slot))
    ops.kv8_append(x[0], x[1], kc2, vc2, ks2, vs2, i32(page), i32(slot))
    for a, b, name in ((kc, kc2, "k codes"), (vc, vc2, "v codes"), (ks, ks2, "k scales"), (vs, vs2, "v scales")):
        a.check(name)
        _same(a.t, b, name)
    assert ops.device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Hq,Hkv", [(1, 3, 3), (1, 8, 1), (3, 10, 2), (2, 40, 1)])
@pytest.mark.parametrize("shares", [1, 5, 40])
def test_decode(d, Nq, Hq, Hkv, shares):
    a = dev(make([1, 300, 0, 129], Nq, Hq, Hkv, d, 16, seed=Nq))
    o_plain, l_plain = ops.decode_kv8(*a, 300, num_shares=shares)
    lib = _lib.load()
    B, pages, blocks = 4, a[1].shape[0], a[5].shape[1]
    o, l = Guarded(a[0].shape, torch.bfloat16), Guarded((B, Hq, Nq), torch.float32, 16)
    ws = Guarded((lib.fa_decode_kv8_workspace_bytes(B, Nq, Hq, Hkv, d, shares),), torch.uint8)
    assert lib.fa_decode_kv8(*(_p(t) for t in a), _p(o.t), _p(l.t), B, Nq, Hq, Hkv, d, 16, pages, blocks, 300, -1, shares,
                             _p(ws.t), 1 / math.sqrt(d), _s()) == _lib.FA_OK
    for x, name in ((o, "o"), (l, "lse"), (ws, "workspace")):
        x.check(name)
    _same(o.t, o_plain, "o"), _same(l.t, l_plain, "lse")
    assert ops.device_error() == 0


def test_two_graphs_share_a_workspace_one_after_the_other():
    one, two = dev(make([700, 30], 1, 8, 2, 128, 16, seed=1)), dev(make([90, 300], 4, 8, 2, 64, 16, seed=2))
    plain = [ops.decode_kv8(*one, 700), ops.decode_kv8(*two, 300)]
    lib = _lib.load()
    ws = torch.empty(max(lib.fa_decode_kv8_workspace_bytes(2, 1, 8, 2, 128, 456),
                         lib.fa_decode_kv8_workspace_bytes(2, 4, 8, 2, 64, 456)), dtype=torch.uint8, device="cuda")
    graphs, got = [], []
    for a, n in ((one, 700), (two, 300)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(ops.decode_kv8(*a, n, workspace=ws))
        graphs.append(g)
    for _ in range(10):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    for x, y in zip(got, plain):
        _same(x[0], y[0], "o"), _same(x[1], y[1], "lse")
