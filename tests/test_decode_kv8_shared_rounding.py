"""What fa_decode_kv8_shared promises of its roundings: a probability times its
value scale is off by 2^-11 of itself, or by 2^-32 of the row's largest, and
queries within 2^28 of their row's largest are exact.

Tolerance of O: half a bf16 step of the result, 2^-8 |o|; 2^-11 a for the
rounding of the products P_j scale_j (a = sum_j P_j |v_j|); 2^-11 a for the scores
and the exponential, in numerator and sum, as over bf16 pages; and 2^-32 of the
row's largest product for each key, times its code: with n keys 2^-32 n 448
times the largest value scale.  Values come in pairs of opposite sign whose keys
differ little, so o is far below a and its own rounding hides nothing: what a
probability rounded to bf16 would do is outside, and is tested to be.
lse: 2^-12.
"""
import numpy as np
import pytest
import torch

import synth
from exact_attention_94_gb300 import ops
from oracle.fp8 import e4m3_decode
from tests.test_decode_kv8_shared_gpu import call, make8, want


def pairs(groups, Nq, Hq, Hkv, d, seed):
    """Keys 2j and 2j + 1 differ in the last bit of four codes, and their values in the sign."""
    m = make8(groups, Nq, Hq, Hkv, d, 16, seed)
    m["k"][:, :, 1::2] = m["k"][:, :, 0::2]
    m["k"][:, :, 1::2, :4] ^= 1
    m["v"][:, :, 1::2] = m["v"][:, :, 0::2] ^ 0x80
    return m


def tolerance(m, o, a):
    largest = float(m["v_scale"][~m["v_scale"].isnan()].max())
    return 2.0 ** -8 * np.abs(o) + 2.0 ** -10 * a + 2.0 ** -32 * 448 * max(m["lens"]) * largest


def check(m, got, ref):
    o, lse, a = ref
    err, tol = np.abs(synth.to_f64(got[0]) - o), tolerance(m, o, a)
    assert np.all(err <= tol), float((err / tol).max())
    assert np.all(np.abs(got[1].double().cpu().numpy() - lse) <= 2.0 ** -12)
    assert ops.device_error() == 0


OWN, SHARED = [(0, [32] * 20)], [(32, [34] * 20)]


@pytest.mark.parametrize("dtype,inside", [(torch.bfloat16, False), (torch.float16, True)])
def test_the_bound_tells_roundings_apart(dtype, inside):
    m = pairs(OWN, 1, 8, 1, 64, 1)
    o, _, a = want(m)
    k, v = (e4m3_decode(m[x].numpy()) for x in ("k", "v"))
    rounded = np.zeros_like(o)
    for b in range(20):
        t = m["table"][b, :2]
        ks, vs = (np.repeat(m[x][t, 0].double().numpy(), 16) for x in ("k_scale", "v_scale"))
        s = 64 ** -0.5 * synth.to_f64(m["q"][b, 0]) @ (k[t, 0].reshape(32, 64) * ks[:, None]).T
        p = np.exp(s - s.max(1, keepdims=True))
        pv = torch.tensor(p * vs * 128).to(dtype).double().numpy() / 128
        rounded[b, 0] = pv @ v[t, 0].reshape(32, 64) / p.sum(1, keepdims=True)
    assert np.all(np.abs(rounded - o) <= tolerance(m, o, a)) == inside


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,heads", [(1, 8), (2, 8), (1, 20), (4, 40)])  # by warps (of d = 64 the second too); by tiles
@pytest.mark.parametrize("groups", [OWN, SHARED, [(96, [98, 100, 96, 128])]])
def test_products_are_rounded_as_promised(groups, Nq, heads, d):
    for seed in (1, 2):
        m = pairs(groups, Nq, heads, 1, d, seed)
        ref = want(m)
        for shares in (0, 1):
            check(m, call(m, num_shares=shares), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [4, 20])
@pytest.mark.parametrize("largest", [-60, 14, 90])
def test_queries_far_below_their_rows_largest(largest, heads, d):
    """The largest meets codes of 0; the scores are made of elements 2^25 to 2^28 below it."""
    m = make8([(64, [70, 64, 129])], 1, heads, 1, d, 16, seed=heads)
    gen = torch.Generator().manual_seed(7)
    at = torch.rand(m["q"].shape, generator=gen) * 3 + largest - 28
    q = torch.ldexp(1 + torch.randint(0, 128, at.shape, generator=gen) / 128, at.floor().int())
    m["q"] = torch.where(torch.rand(at.shape, generator=gen) < 0.5, q, -q).to(torch.bfloat16)
    m["q"][..., 5] = 2.0 ** largest
    m["k"][..., 5] = 0
    m["k_scale"] = m["k_scale"] * 2.0 ** (26 - largest)
    check(m, call(m), want(m))
