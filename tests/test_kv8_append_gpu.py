"""fa_kv8_append against the reference: codes and scales bit for bit (a NaN code
of either sign counts as one)."""
import numpy as np
import pytest
import torch

import synth
from exact_attention_94_gb300 import ops
from oracle import serving

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def cache(rng, pages, Hkv, P, d):
    """Both sides of a cache with arbitrary codes (NaN among them) and powers of two."""
    out = []
    for _ in range(2):
        out.append((rng.integers(0, 256, (pages, Hkv, P, d)).astype(np.uint8),
                    (2.0 ** rng.integers(-10, -4, (pages, Hkv))).astype(np.float32)))
    return out


def same_codes(got, want):
    got = got.cpu().numpy()
    nan = lambda c: (c & 0x7F) == 0x7F  # noqa: E731
    assert np.array_equal(nan(got), nan(want))
    assert np.array_equal(np.where(nan(got), 0, got), np.where(nan(want), 0, want))


def run(rng, pages, Hkv, P, d, page, slot, src=None, amp=None, stride=0, state=None, x=None):
    n = len(page)
    state = state if state is not None else cache(rng, pages, Hkv, P, d)
    if x is None:
        x = torch.tensor(rng.standard_normal((n, 2 * Hkv * d + stride)), dtype=torch.float32)
        if amp is not None:
            x = x * torch.tensor(amp, dtype=torch.float32)[:, None]
    x = x.to(torch.bfloat16).cuda()
    kn, vn = x[:, :Hkv * d].unflatten(1, (Hkv, d)), x[:, Hkv * d:2 * Hkv * d].unflatten(1, (Hkv, d))
    dev = [(torch.tensor(c).cuda(), torch.tensor(s).cuda()) for c, s in state]
    ops.kv8_append(kn, vn, dev[0][0], dev[1][0], dev[0][1], dev[1][1], i32(page), i32(slot),
                   None if src is None else i32(src))
    for new, (c, s) in zip((kn, vn), state):
        serving.kv8_append(synth.to_f64(new), c, s, page, slot, src)
    for (gc, gs), (c, s) in zip(dev, state):
        assert np.array_equal(gs.cpu().numpy(), s)
        same_codes(gc, c)
    return state


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("P", [16, 48, 128])
def test_runs_of_every_kind(d, Hkv, P):
    rng = np.random.default_rng(d + Hkv + P)
    page, slot = [], []
    for pg, first, n in ((4, 0, 1), (2, P - 1, 1), (7, 0, P), (0, 5, P - 5), (3, 0, 7), (6, 11, 2), (1, 15, 1)):
        page += [pg] * n
        slot += list(range(first, first + n))
    page[2:2] = [-1, -1]      # padding between runs
    slot[2:2] = [-1, -1]
    amp = np.where(rng.random(len(page)) < 0.3, 30.0, 0.01)
    run(rng, 9, Hkv, P, d, page, slot, amp=amp, stride=8)
    assert ops.device_error() == 0


def test_a_page_filled_token_by_token_and_then_once_more():
    rng = np.random.default_rng(7)
    state = cache(rng, 2, 2, 16, 64)
    for t in range(35):
        run(rng, 2, 2, 16, 64, [t // 16 % 2], [t % 16], amp=[2.0 ** (t % 9 - 4)], state=state)
    assert ops.device_error() == 0


def test_long_prompts_of_many_requests():
    rng = np.random.default_rng(8)
    P, page, slot, pages = 32, [], [], 400
    order = rng.permutation(pages)
    at = 0
    for n, ctx in ((700, 3), (1, 31), (33, 0), (2047, 17), (64, 0), (5, 30)):
        for t in range(ctx, ctx + n):
            page.append(order[at + t // P])
            slot.append(t % P)
        at += (ctx + n) // P + 1
    run(rng, pages, 2, P, 128, page + [-1] * 77, slot + [-1] * 77)
    assert ops.device_error() == 0


@pytest.mark.parametrize("amp", [0.01, 1.0, 100.0])
def test_copy_on_write(amp):
    """Two children and the parent go on in one call: the children copy, the parent
    writes (and rescales) the very page that they copy from."""
    rng = np.random.default_rng(9)
    run(rng, 12, 4, 16, 128, [5, 3, 8, 1], [9, 9, 9, 2], src=[3, -1, 3, -1], amp=[amp, 100.0, amp, amp])
    run(rng, 12, 4, 16, 128, [5, 5, 3, 3, 3], [9, 10, 9, 10, 11], src=[3, -1, -1, -1, -1], amp=[amp] * 5)
    run(rng, 12, 4, 16, 128, [5], [0], src=[3])
    assert ops.device_error() == 0


def test_zeros_extremes_and_numbers_that_are_none():
    rng = np.random.default_rng(10)
    Hkv, d = 2, 64
    x = torch.randn((6, 2 * Hkv * d), generator=torch.Generator().manual_seed(1))
    x[0] = 0.0
    x[1] *= 1e-38                 # below bf16's normal range in places
    x[2] *= 3e37
    x[3, ::5] = float("nan")
    x[4, ::7] = float("inf")
    x[4, 1::7] = -float("inf")
    x[5] = float("inf")           # nothing finite at all
    run(rng, 8, Hkv, 16, d, [0, 1, 2, 3, 4, 5], [0] * 6, x=x)
    run(rng, 8, Hkv, 16, d, [0, 1, 2, 3, 4, 5], [3] * 6, x=x)
    state = [(np.zeros((2, Hkv, 16, d), np.uint8), np.zeros((2, Hkv), np.float32)) for _ in range(2)]
    for t in range(3):            # a page of zeros that a number joins
        run(rng, 2, Hkv, 16, d, [1], [t], x=torch.zeros((1, 2 * Hkv * d)) + (t == 2), state=state)
    assert ops.device_error() == 0


@pytest.mark.parametrize("page,slot,src", [(9, 0, -1), (-2, 0, -1), (2, 16, -1), (2, -1, -1), (2, 3, 9), (2, 3, -2)])
def test_bad_rows_are_skipped_and_reported(page, slot, src):
    rng = np.random.default_rng(11)
    state = cache(rng, 9, 2, 16, 64)
    dev = [(torch.tensor(c).cuda(), torch.tensor(s).cuda()) for c, s in state]
    x = torch.randn((3, 2, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    ops.kv8_append(x, x, dev[0][0], dev[1][0], dev[0][1], dev[1][1], i32([5, page, 6]), i32([0, slot, 1]),
                   i32([-1, src, -1]))
    assert ops.device_error() == 0x2000
    for c, s in state:
        serving.kv8_append(synth.to_f64(x), c, s, [5, -1, 6], [0, -1, 1])
    for (gc, gs), (c, s) in zip(dev, state):
        assert np.array_equal(gs.cpu().numpy(), s)
        same_codes(gc, c)


def test_a_run_does_not_leave_its_page():
    rng = np.random.default_rng(12)
    state = cache(rng, 3, 1, 16, 64)
    dev = [(torch.tensor(c).cuda(), torch.tensor(s).cuda()) for c, s in state]
    x = torch.randn((4, 1, 64), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    ops.kv8_append(x, x, dev[0][0], dev[1][0], dev[0][1], dev[1][1], i32([1] * 4), i32([14, 15, 16, 17]))
    assert ops.device_error() == 0x2000
    for c, s in state:
        serving.kv8_append(synth.to_f64(x), c, s, [1, 1, -1, -1], [14, 15, -1, -1])
    for (gc, gs), (c, s) in zip(dev, state):
        assert np.array_equal(gs.cpu().numpy(), s)
        same_codes(gc, c)


def test_refusals():
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    c, s, i = torch.zeros((3, 1, 16, 64), dtype=torch.uint8, device="cuda"), torch.zeros((3, 1), device="cuda"), i32([0, 1])
    ops.kv8_append(x[:0], x[:0], c, c.clone(), s, s.clone(), i[:0], i[:0])
    for bad in (lambda: ops.kv8_append(x, x, c, c, s, s, i[:1], i), lambda: ops.kv8_append(x, x[:1], c, c, s, s, i, i),
                lambda: ops.kv8_append(x, x, c.view(3, 16, 1, 64), c, s, s, i, i),
                lambda: ops.kv8_append(x, x, c, c, s.half(), s, i, i), lambda: ops.kv8_append(x, x, c, c, s, s, i.long(), i)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("n,Hkv,d,P", [(1500, 8, 64, 16), (3001, 8, 64, 32), (9011, 8, 64, 32), (2300, 32, 128, 16),
                                       (700, 32, 64, 48)])
def test_from_few_rows_to_many(n, Hkv, d, P):
    """How many warps share 32 rows goes by rows times heads: 5, 2, 1, 1 and 3 in these
    cases.  Prompts and single tokens in one call, that begin anywhere in their pages,
    padding between them."""
    rng = np.random.default_rng(n)
    page, slot, used = [], [], 0
    order = rng.permutation(n)          # (more pages than are used)
    while len(page) < n:
        new, first = (1 if rng.random() < 0.4 else int(rng.integers(2, 150))), int(rng.integers(0, P))
        for t in range(first, first + min(new, n - len(page))):
            page.append(int(order[used + t // P]))
            slot.append(t % P)
        used += (first + new - 1) // P + 1
        if rng.random() < 0.1:
            page, slot = page + [-1] * 3, slot + [-1] * 3
    pages = int(max(page)) + 1
    amp = 2.0 ** rng.integers(-6, 6, len(page))
    run(rng, pages, Hkv, P, d, page, slot, amp=amp, stride=8)
    assert ops.device_error() == 0
