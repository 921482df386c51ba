"""Guard bands around what the sampling-step operators write: outputs and
workspaces lie inside sentinel-filled buffers; every byte outside them stays, and
they hold what the plain call gives.  Sizes are ragged, shares cut everywhere."""
import ctypes
import math

import pytest
import torch

from exact_attention_94_gb300 import _lib, ops
from tests.test_canary_gpu import Guarded, _p, _s, _same
from tests.test_decode_kv8_shared_gpu import make8
from tests.test_decode_shared_gpu import i32, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Hq,Hkv", [(1, 3, 3), (1, 16, 1), (3, 10, 2), (2, 40, 1)])
@pytest.mark.parametrize("shares", [1, 5, 200])
def test_shared(kv8, d, Nq, Hq, Hkv, shares):
    groups = [(300, [301, 420, 300, 0, 17]), (0, [5]), (150, [700, 151]), (40, [60] * 70)]
    m = (make8 if kv8 else make)(groups, Nq, Hq, Hkv, d, 16, seed=Nq)
    sides = ("q", "k", "v") + (("k_scale", "v_scale") if kv8 else ())
    a = [m[x].cuda() for x in sides] + [i32(m[x]) for x in ("table", "lens", "starts", "shared")]
    plain = (ops.decode_kv8_shared if kv8 else ops.decode_paged_shared)(*a, 700, num_shares=shares)
    lib = _lib.load()
    B, blocks, G = len(m["lens"]), a[-4].shape[1], len(groups)
    o, l = Guarded(a[0].shape, torch.bfloat16), Guarded((B, Hq, Nq), torch.float32, 16)
    ws = Guarded((lib.fa_decode_shared_workspace_bytes(B, Nq, Hq, Hkv, d, G, shares),), torch.uint8)
    call = lib.fa_decode_kv8_shared if kv8 else lib.fa_decode_paged_shared
    assert call(*(_p(t) for t in a), _p(o.t), _p(l.t), B, Nq, Hq, Hkv, d, 16, a[1].shape[0], blocks, 700, G, -1, shares,
                _p(ws.t), 1 / math.sqrt(d), _s()) == _lib.FA_OK
    for x, name in ((o, "o"), (l, "lse"), (ws, "workspace")):
        x.check(name)
    _same(o.t, plain[0], "o"), _same(l.t, plain[1], "lse")
    assert ops.device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (67, 5, 1), (1000, 17, 3), (333, 0, 2)])
def test_norms(d, T, Hq, Hkv):
    plan = ops.rope_plan(d, [d // 8, d // 8, d // 4])
    q, k, dyq, dyk = (torch.randn((T, H, d), device="cuda").to(torch.bfloat16) if H else None for H in (Hq, Hkv) * 2)
    w = torch.randn((2, d), device="cuda")
    wq = w[0] if Hq else None
    pos = torch.randint(0, 9999, (3, T), device="cuda", dtype=torch.int32)
    plain, grads = ops.qk_norm_rope(q, k, wq, w[1], pos, plan), ops.qk_norm_rope_bwd(dyq, dyk, q, k, wq, w[1], pos, plan)
    for back, want in ((False, plain), (True, grads[:2])):
        g = [Guarded(x.shape, torch.bfloat16, 16 * i) if x is not None else None for i, x in enumerate((q, k))]
        out = tuple(x.t if x else None for x in g)
        if back:
            size = _lib.load().fa_qk_norm_rope_bwd_workspace_bytes(T, Hq, Hkv, d)
            ws = Guarded((size,), torch.uint8)
            got = ops.qk_norm_rope_bwd(dyq, dyk, q, k, wq, w[1], pos, plan, out=out, workspace=ws.t)
            ws.check("workspace")
            for x, y in zip(got[2:], grads[2:]):
                assert (x is None and y is None) or torch.equal(x, y)
        else:
            ops.qk_norm_rope(q, k, wq, w[1], pos, plan, out=out)
        for x, y, name in zip(g, want, ("q", "k")):
            if x:
                x.check(name)
                _same(x.t, y, name)


def test_many_requests_in_many_groups():
    """More groups and entries than the plan keeps in shared memory."""
    groups = [(16 + g % 3, [17 + g % 5 + 3 * i for i in range(2)]) for g in range(1100)]
    m = make(groups, 1, 4, 1, 64, 16, seed=9)
    a = [m[x].cuda() for x in ("q", "k", "v")] + [i32(m[x]) for x in ("table", "lens", "starts", "shared")]
    o, lse = ops.decode_paged_shared(*a, max(m["lens"]))
    po, pl = ops.decode_paged_window(a[0], a[1], a[2], a[3], a[4], max(m["lens"]))
    assert ops.device_error() == 0
    assert torch.allclose(lse[..., 0], pl, atol=2.0 ** -11, rtol=0)
    # both round O and the probabilities to bf16: 2^-8 of the largest |v| (below 8) four times
    assert (o.float() - po.float()).abs().max() <= 4 * 2.0 ** -8 * 8


@pytest.mark.parametrize("kv8", [False, True])
def test_two_calls_at_once(kv8):
    """On two streams, each with workspace and outputs of its own."""
    many = [(300, [301 + i for i in range(40)])]
    one, two = ((make8 if kv8 else make)(g, 1, 16, 2, d, 16, seed=3) for g, d in ((many, 64), ([(0, [4000, 17, 900])] * 9, 128)))
    call = ops.decode_kv8_shared if kv8 else ops.decode_paged_shared
    sides = ("q", "k", "v") + (("k_scale", "v_scale") if kv8 else ())
    args = [[m[x].cuda() for x in sides] + [i32(m[x]) for x in ("table", "lens", "starts", "shared")] + [max(m["lens"])] for m in (one, two)]
    plain = [call(*a) for a in args]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append(call(*args[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, plain[i][0]) and torch.equal(lse, plain[i][1])


@pytest.mark.parametrize("kv8", [False, True])
def test_pages_beyond_32_bits(kv8):
    """The same pages at the far end of a pool of more than 4 GB a side give the same bits."""
    m = (make8 if kv8 else make)([(150, [200, 151, 700]), (40, [60] * 20)], 1, 8, 1, 128, 64, seed=4, **({} if kv8 else dict(fill=0.0)))
    call = ops.decode_kv8_shared if kv8 else ops.decode_paged_shared
    sides = ("k", "v") + (("k_scale", "v_scale") if kv8 else ())
    tail = [i32(m[x]) for x in ("lens", "starts", "shared")] + [700]
    near = [m[x].cuda() for x in sides]
    plain = call(m["q"].cuda(), *near, i32(m["table"]), *tail)
    n = near[0].shape[0]
    pool = (1 << 32) // (64 * 128) // near[0].element_size() * 2 + n
    far = []
    for x in near:
        y = torch.empty((pool, *x.shape[1:]), dtype=x.dtype, device="cuda")
        y[-n:] = x
        far.append(y)
    got = call(m["q"].cuda(), *far, i32(m["table"] + pool - n), *tail)
    assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
    assert ops.device_error() == 0
