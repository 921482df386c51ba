"""Attention of requests that share prefixes, over pages of 8-bit codes, against
the reference in 64 bits on the values that the codes stand for.

Tolerances as for bf16 pages: half a bf16 step of O, 2^-8 |o|; scores are fp32
sums of exact products, times a scale: 2^-11 a, a = sum_j P_j |v_j|; and 2^-8 a,
what probabilities rounded to bf16 would take, where these are f16: 2^-8 |o| +
(2^-8 + 2^-11) a; lse 2^-12.  test_decode_kv8_shared_rounding.py has the tolerance
that f16 leaves.
"""
import numpy as np
import pytest
import torch

import synth
from exact_attention_94_gb300 import _lib, ops
from oracle import sampling
from oracle.fp8 import e4m3_decode
from tests.test_decode_shared_gpu import SHAPES, check, i32, make

pytestmark = pytest.mark.gpu


def make8(groups, Nq, Hq, Hkv, d, P, seed=0, garbage=True):
    """As `make`, with codes and a power of two per page and head; what no request uses is NaN."""
    m = make(groups, Nq, Hq, Hkv, d, P, seed, fill=float("nan") if garbage else None)
    rng = np.random.default_rng(seed + 1)
    for name, low in (("k", -2), ("v", -4)):
        x = m[name].transpose(1, 2).float()  # [pages, Hkv, P, d]
        m[name] = (x * 2.0 ** (-low)).to(torch.float8_e4m3fn).view(torch.uint8).contiguous()
        scale = 2.0 ** (low + rng.integers(-2, 3, x.shape[:2]))
        m[name + "_scale"] = torch.tensor(scale, dtype=torch.float32)
    unused = torch.ones(m["k"].shape[0], dtype=torch.bool)
    for b, n in enumerate(m["lens"]):
        unused[torch.tensor(m["table"][b, :-(-n // P)]).long()] = False
    for name in ("k_scale", "v_scale"):
        m[name][unused] = float("nan")
    return m


def call(m, window=-1, max_len=None, **kw):
    return ops.decode_kv8_shared(m["q"].cuda(), m["k"].cuda(), m["v"].cuda(), m["k_scale"].cuda(), m["v_scale"].cuda(),
                                 i32(m["table"]), i32(m["lens"]), i32(m["starts"]), i32(m["shared"]),
                                 max(m["lens"]) if max_len is None else max_len, window_left=window, **kw)


def want(m, window=-1):
    k, v = (e4m3_decode(m[x].numpy()) * m[x + "_scale"].double().numpy()[:, :, None, None] for x in ("k", "v"))
    return sampling.decode_shared(synth.to_f64(m["q"]), lambda p, t: k[p, :, t], lambda p, t: v[p, :, t], m["table"], m["lens"],
                                  m["starts"], m["shared"], m["P"], window, m["q"].shape[-1] ** -0.5)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Hq,Hkv", [(1, 4, 4), (1, 8, 1), (1, 10, 2), (3, 7, 1)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("shares", [0, 1, 5])
def test_groups(d, Nq, Hq, Hkv, shape, shares):
    m = make8(SHAPES[shape], Nq, Hq, Hkv, d, (16, 48, 128)[(shape + Nq) % 3], seed=shape)
    check(call(m, num_shares=shares), want(m))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,n", [(1, 300), (8, 40), (5, 60), (128, 3), (7, 37), (33, 13), (16, 11)])
def test_many_rows(heads, n, d):
    m = make8([(150, [151 + i % 20 for i in range(n)]), (40, [60] * 4), (700, [700 + i for i in range(n)])], 1, heads, 1, d, 16, seed=n)
    ref = want(m)
    for shares in (0, 1, 7):
        check(call(m, num_shares=shares), ref)


@pytest.mark.parametrize("window", [0, 1, 40, 127, 300])
@pytest.mark.parametrize("Nq", [1, 4])
def test_windows(window, Nq):
    m = make8([(300, [301, 330, 420, 310, 300, 7, 0]), (100, [500, 103])], Nq, 4, 2, 64, 16, seed=window)
    ref = want(m, window)
    for g, (s, e) in enumerate(zip(m["starts"], m["starts"][1:])):
        least = min(n for n in m["lens"][s:e] if n > 0)
        for b in range(s, e):
            gone = max(0, min(least, m["lens"][b]) - Nq - window) // 16
            m["table"][b, :gone] = 10 ** 6
    for shares in (0, 3):
        check(call(m, window, num_shares=shares), ref)


@pytest.mark.parametrize("heads", [1, 8, 40])
def test_requests_without_keys_share_nothing(heads):
    m = make8([(520, [530, 0, 700, 0]), (300, [0, 300])], 1, heads, 1, 64, 16, seed=heads)
    for shares in (0, 1):
        check(call(m, num_shares=shares), want(m))


@pytest.mark.parametrize("heads", [4, 12])  # the shared keys by a warp, and by tiles
@pytest.mark.parametrize("Nq,window,key", [(1, -1, 30), (4, -1, 128), (4, -1, 127), (1, 20, 100), (3, 50, 60), (1, -1, 310)])
def test_odd_values_stay_with_the_queries_that_see_them(Nq, window, key, heads):
    """A NaN code; a value scale that is no number."""
    m = make8([(90, [130, 131, 129, 320])], Nq, heads, 1, 128, 16, seed=5)
    plain = call(m, window)
    for name, bad in (("v", 0x7F), ("v", 0xFF), ("v_scale", float("inf")), ("v_scale", float("nan"))):
        odd = dict(m, **{name: m[name].clone()})
        first, last = (key, key) if name == "v" else (key // 16 * 16, key // 16 * 16 + 15)
        for b in range(4):
            if key < m["lens"][b]:
                if name == "v":
                    odd[name][m["table"][b, key // 16], 0, key % 16, 3] = bad
                else:
                    odd[name][m["table"][b, key // 16], 0] = bad
        o, lse = call(odd, window)
        # (a scale takes part in the choice of the sums' reference: both are within 2^-12 of the sum)
        assert torch.equal(lse, plain[1]) if name == "v" else torch.allclose(lse, plain[1], atol=2.0 ** -11, rtol=0)
        for b in range(4):
            for i in range(Nq):
                pos = m["lens"][b] - Nq + i
                keys = [j for j in range(first, last + 1) if j <= pos and (window < 0 or j >= pos - window)]
                if keys and key < m["lens"][b]:
                    assert not torch.isfinite(o[b, i, :, 3]).any()
                elif not keys:
                    assert torch.equal(o[b, i], plain[0][b, i]), (b, i)


@pytest.mark.parametrize("shared", [90, 0])
def test_odd_keys(shared):
    m = make8([(shared, [130, 131])], 2, 4, 1, 64, 16, seed=5)
    plain = call(m)
    m["k"][m["table"][0, 129 // 16], 0, 129 % 16, 3] = 0x7F  # the last key of the first request
    o, lse = call(m)
    assert torch.isnan(o[0, 1]).all() and torch.isnan(lse[0, :, 1]).all()
    assert torch.equal(o[0, 0], plain[0][0, 0]) and torch.equal(o[1], plain[0][1])


@pytest.mark.parametrize("heads", [2, 20])
def test_scales(heads):
    """Pages of zeros, loud and faint pages."""
    m = make8([(300, [310, 500, 301])], 1, heads, 1, 64, 16, seed=heads)
    used = sorted({int(p) for b, n in enumerate(m["lens"]) for p in m["table"][b, :-(-n // 16)]})
    for i, p in enumerate(used):
        if i % 5 == 0:
            m["v_scale"][p] = 0.0
            m["k_scale"][p] = 0.0
        elif i % 5 == 1:
            m["v_scale"][p] = 2.0 ** 70
        elif i % 5 == 2:
            m["v_scale"][p] = 2.0 ** -70
    check(call(m), want(m))


def test_the_largest_and_smallest_codes():
    """Every finite code as a key and as a value."""
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 0x7F) != 0x7F]  # 254
    for heads in (4, 16):
        m = make8([(254, [254 + i for i in range(3)])], 1, heads, 1, 64, 16, seed=heads)
        for j in range(254):
            for b in range(3):
                m["v"][m["table"][b, j // 16], 0, j % 16] = codes[j]
                m["k"][m["table"][b, j // 16], 0, j % 16, :] = torch.roll(m["k"][m["table"][b, j // 16], 0, j % 16], 1)
                m["k"][m["table"][b, j // 16], 0, j % 16, j % 64] = codes[j]
        m["k_scale"][~m["k_scale"].isnan()] = 2.0 ** -6
        check(call(m), want(m))


def test_bad_pages_and_lengths_are_reported():
    m = make8([(100, [120, 130]), (50, [60, 200])], 1, 4, 2, 64, 16, seed=2)
    plain = call(m)
    bad = dict(m, table=m["table"].copy())
    bad["table"][3, 11] = 10 ** 8
    o, _ = call(bad)
    assert ops.device_error() == 0x2000 and torch.equal(o[:3], plain[0][:3])
    o, _ = call(dict(m, lens=[120, 130, 60, 201]), max_len=200)
    assert ops.device_error() == 0x2001 and torch.equal(o, plain[0])
    o, lse = call(dict(m, lens=[120, 130, 60, -5]), max_len=200)
    assert ops.device_error() == 0x2001 and not o[3].any() and torch.isneginf(lse[3]).all()


def test_graphs_that_share_a_workspace():
    one, two = make8([(100, [120, 130, 300])], 1, 8, 2, 128, 16, seed=1), make8([(40, [90, 50])] * 3, 4, 8, 2, 64, 16, seed=2)
    plain = [call(one), call(two)]
    size = _lib.load().fa_decode_shared_workspace_bytes
    ws = torch.empty(max(size(3, 1, 8, 2, 128, 1, 0), size(6, 4, 8, 2, 64, 3, 0)), dtype=torch.uint8, device="cuda")
    graphs, got = [], []
    for m in (one, two):
        args = [m[x].cuda() for x in ("q", "k", "v", "k_scale", "v_scale")] + [i32(m[x]) for x in ("table", "lens", "starts", "shared")]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(ops.decode_kv8_shared(*args, max(m["lens"]), workspace=ws))
        graphs.append((g, args))
    for _ in range(10):
        graphs[0][0].replay()
        graphs[1][0].replay()
    torch.cuda.synchronize()
    for x, y in zip(got, plain):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_it_agrees_with_the_decode_that_shares_nothing():
    m = make8([(992, [1001 + 37 * i for i in range(20)])], 4, 16, 4, 128, 16, seed=3)
    got = call(m)
    o, lse = ops.decode_kv8(m["q"].cuda(), m["k"].cuda(), m["v"].cuda(), m["k_scale"].cuda(), m["v_scale"].cuda(), i32(m["table"]),
                            i32(m["lens"]), max(m["lens"]))
    assert torch.allclose(got[1], lse, atol=2.0 ** -11, rtol=0)
    # a = sum P |v| and |o| are at most the largest |v|: the roundings of both O to bf16, 2^-8 of it each, of the
    # probabilities, 2^-8 here and 2^-11 there, and the scores' errors, 2^-11 of it each
    used = ~m["v_scale"].isnan()
    largest = float((m["v"].view(torch.float8_e4m3fn).float().nan_to_num(0).abs().amax((2, 3)) * m["v_scale"])[used].max())
    assert (got[0].float() - o.float()).abs().max() <= (3 * 2.0 ** -8 + 3 * 2.0 ** -11) * largest
