"""The serving-step reference against what defines it: the host page pool, a
rotation's invariants and differences, the e4m3 rounding bound, plain attention."""
import numpy as np
import pytest

import oracle
from oracle import fp8, paged, serving


def test_plan_takes_the_pages_that_the_pool_takes():
    rng = np.random.default_rng(1)
    P, n_pages, S, blocks = 4, 64, 5, 20
    pool = paged.PagePool(n_pages, P, S, blocks)
    for _ in range(S):
        pool.add_seq()
    for _ in range(6):
        table, lens = pool.block_table()
        free, count = list(pool.free), len(pool.free)
        new = rng.integers(0, 4, S).tolist()
        seq, cu, page, slot, pos, left, table2 = serving.page_plan(lens.tolist(), new, free + [0] * (n_pages - count),
                                                                  count, table, P, sum(new) + 3)
        want = [pool.reserve_append(s) for s in range(S) for _ in range(new[s])]
        assert [(p, t, -1) for p, t in zip(page, slot)][: sum(new)] == want
        assert page[sum(new):] == [-1] * 3 and pos[sum(new):] == [0] * 3
        table3, lens3 = pool.block_table()
        assert np.array_equal(table2, table3) and seq == lens3.tolist() and left == len(pool.free)
        assert cu[-1] == sum(new)


def test_plan_refuses():
    t = np.zeros((1, 2), np.int32)
    for ctx, new, count, cap, code in (([0], [-1], 3, 9, 0x2001), ([-1], [1], 3, 9, 0x2001), ([0], [9], 3, 99, 0x2001),
                                       ([0], [8], 3, 7, 0x2001), ([0], [5], 1, 9, 0x2002), ([0], [1], 5, 9, 0x2001)):
        with pytest.raises(serving.PlanError) as e:
            serving.page_plan(ctx, new, [0, 1, 2], count, t, 4, cap)
        assert e.value.code == code


@pytest.mark.parametrize("neighbours", [False, True])
def test_rope_is_a_rotation_and_its_inverse_the_gradient(neighbours):
    rng = np.random.default_rng(2)
    T, H, d = 5, 2, 16
    x, g = rng.standard_normal((T, H, d)), rng.standard_normal((T, H, d))
    pos = rng.integers(-1000, 100000, (3, T))
    axis, freq = [0, 0, 1, 2, 1, -1, 2, 0], [1.0, 0.5, 0.25, 0.7, 0.01, 3.0, 1e-4, 0.1]
    y = serving.rope_axes(x, pos, axis, freq, neighbours)
    assert np.allclose((y * y).sum(-1), (x * x).sum(-1))
    assert np.allclose(serving.rope_axes(y, pos, axis, freq, neighbours, True), x)
    # the gradient of <rope(x), g>, by central differences
    dx = serving.rope_axes(g, pos, axis, freq, neighbours, True)
    for idx in [(0, 0, 0), (3, 1, 7), (4, 0, 15), (2, 1, 5)]:
        e = np.zeros_like(x)
        e[idx] = 1e-4
        diff = (serving.rope_axes(x + e, pos, axis, freq, neighbours) - serving.rope_axes(x - e, pos, axis, freq, neighbours))
        assert abs((diff * g).sum() / 2e-4 - dx[idx]) < 1e-7
    # only differences of positions matter to a score
    k = rng.standard_normal((T, H, d))
    s0 = (serving.rope_axes(x, pos, axis, freq, neighbours) * serving.rope_axes(k, pos - 7, axis, freq, neighbours)).sum(-1)
    s1 = (serving.rope_axes(x, pos + 50, axis, freq, neighbours) * serving.rope_axes(k, pos + 43, axis, freq, neighbours)).sum(-1)
    assert np.allclose(s0, s1)


def test_scale_is_the_smallest_power_of_two():
    for amax in (1e-45, 2.0 ** -120, 0.1, 1.0, 447.0, 448.0, 449.0, 3e38):
        s = serving.pow2_scale(amax)
        assert np.log2(s) == round(np.log2(s)) and amax <= 448 * s
        assert s == 2.0 ** -126 or amax > 224 * s
    assert serving.pow2_scale(0.0) == 0.0


def test_append_token_by_token_stays_within_the_rounding():
    """Each code is off by half a step of e4m3 at most, and one more half step
    below its normal range for every time the scale has grown since."""
    rng = np.random.default_rng(3)
    P, H, d, pages = 16, 2, 8, 3
    codes, scales = np.full((pages, H, P, d), 0x7F, np.uint8), np.full((pages, H), 7.0, np.float32)
    rows = []
    for t in range(P + 5):
        x = rng.standard_normal((1, H, d)) * (1.0 + 10.0 * (t % 7 == 6))
        rows.append(x[0])
        serving.kv8_append(x, codes, scales, [2 if t < P else 0], [t % P])
    want = np.stack(rows)                                        # [tokens, H, d]
    got = serving.kv8_values(codes, scales)
    for page, lo, n in ((2, 0, P), (0, P, 5)):
        w, s = want[lo:lo + n].transpose(1, 0, 2), scales[page][:, None, None].astype(np.float64)
        assert np.all(np.abs(got[page, :, :n] - w) <= 2.0 ** -4 * np.abs(w) + 2 * 2.0 ** -10 * s)
        assert np.array_equal(scales[page], [serving.pow2_scale(np.abs(w[h]).max()) for h in range(H)])
    assert np.all(codes[0, :, 5:] == 0x7F) and np.all(codes[1] == 0x7F)


def test_append_of_a_whole_page_is_plain_quantisation_and_nan_is_kept():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((16, 1, 8))
    x[3, 0, 2], x[5, 0, 1] = np.nan, np.inf
    codes, scales = np.zeros((1, 1, 16, 8), np.uint8), np.zeros((1, 1), np.float32)
    serving.kv8_append(x, codes, scales, [0] * 16, list(range(16)))
    fine = np.isfinite(x[:, 0])
    s = serving.pow2_scale(np.abs(x[np.isfinite(x)]).max())
    assert scales[0, 0] == s
    assert np.array_equal(codes[0, 0][fine], fp8.e4m3_encode(x[:, 0][fine] / s))
    assert np.all(codes[0, 0][~fine] == 0x7F)


def test_attention_equals_the_plain_one():
    rng = np.random.default_rng(5)
    P, Hkv, g, d, n = 16, 2, 3, 8, 37
    codes = rng.integers(0, 0x7F, (2, 4, Hkv, P, d)).astype(np.uint8)
    scales = (2.0 ** rng.integers(-12, -6, (2, 4, Hkv))).astype(np.float32)
    table = np.array([[3, 1, 0]])
    q = rng.standard_normal((1, 1, Hkv * g, d))
    o, lse, a, f = serving.decode_kv8(q, codes[0], codes[1], scales[0], scales[1], table, [n], -1, 0.3)
    k, v = (serving.kv8_values(codes[i], scales[i])[table[0]].transpose(0, 2, 1, 3).reshape(1, -1, Hkv, d)[:, :n]
            for i in (0, 1))
    o2, lse2 = oracle.gqa_decode_forward(q, k, v, 0.3)
    assert np.allclose(o, o2) and np.allclose(lse[:, :, 0], lse2) and np.all(a >= np.abs(o) - 1e-12) and np.all(f >= a / n)
    # four queries, a window: the masked oracle's bottom-right alignment
    q = rng.standard_normal((1, 4, Hkv * g, d))
    o, lse, _, _ = serving.decode_kv8(q, codes[0], codes[1], scales[0], scales[1], table, [n], 5, 0.3)
    o2, lse2 = oracle.masked_forward(q, k, v, 0.3, 5, 0)
    assert np.allclose(o, o2) and np.allclose(lse, lse2)
    # more queries than keys: the first see nothing
    o, lse, _, _ = serving.decode_kv8(q, codes[0], codes[1], scales[0], scales[1], table, [2], -1, 0.3)
    assert np.all(o[0, :2] == 0) and np.all(lse[0, :, :2] == -np.inf) and np.all(np.isfinite(lse[0, :, 2:]))
