"""Attention of requests that share prefixes over 8-bit pages whose value scales
lie far apart, up to the 2^-80 .. 2^80 (or 0) that are allowed: what a key's
value weighs takes no part in its weight in the sum of the softmax, whatever
comes before or behind it.

Tolerances as in test_decode_kv8_shared_gpu.py: the scales are powers of two and
round nothing; a reference of a row's sum that a scale has moved by up to 2^80
keeps the sum's exponents below 127, and costs the lse 2^-17 of its 2^-12.
"""
import pytest

from tests.test_decode_kv8_shared_gpu import call, make8, want
from tests.test_decode_shared_gpu import check

pytestmark = pytest.mark.gpu

ORDERS = {
    "faint, loud": lambda j, n: -70 if j < n // 2 else 70,
    "none, loud": lambda j, n: None if j < n // 2 else 70,
    "faintest, loudest": lambda j, n: -80 if j < n // 2 else 80,
    "loudest, faintest": lambda j, n: 80 if j < n // 2 else -80,
    "loud, none": lambda j, n: 70 if j < n // 2 else None,
    "a loud page at the end": lambda j, n: 75 if j == n - 1 else -60,
    "rising": lambda j, n: -80 + 160 * j // max(1, n - 1),
    "none, faint, loud, in turn": lambda j, n: (None, -80, 80)[j % 3],
    "eight pages each in turn": lambda j, n: (-75, 75)[j // 8 % 2],
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,n", [(2, 3), (8, 2), (20, 3), (40, 7)])  # by warps; one tile of rows; two
@pytest.mark.parametrize("order", ORDERS)
@pytest.mark.parametrize("shares", [0, 1])
def test_scales_far_apart(order, heads, n, d, shares):
    m = make8([(600, [650 + i for i in range(n)]), (0, [500])], 1, heads, 1, d, 16, seed=heads)
    for b, length in enumerate(m["lens"]):
        pages = -(-length // 16) if b == n else 41  # (requests that share pages agree on their scales)
        for j in range(-(-length // 16)):
            e = ORDERS[order](j, pages)
            m["v_scale"][m["table"][b, j]] = 0.0 if e is None else 2.0 ** e
    check(call(m, num_shares=shares), want(m))


@pytest.mark.parametrize("heads", [2, 20])
@pytest.mark.parametrize("Nq,window", [(4, 200), (3, -1)])
def test_scales_far_apart_with_drafts(heads, Nq, window):
    m = make8([(400, [430, 470, 401])], Nq, heads, 1, 64, 16, seed=heads)
    for b, length in enumerate(m["lens"]):
        for j in range(-(-length // 16)):
            m["v_scale"][m["table"][b, j]] = 2.0 ** (-80 if j < 20 else 80)
    check(call(m, window, num_shares=1), want(m, window))
