"""fa_decode_kv8 against the reference attention over the dequantised cache.

Tolerances, with A = sum_j P_j |v_j| and F = max_j (P_j vs_j) sum_j |v8_j|
(element by element; v8 the codes' values, vs their scales):
  O   : half a bf16 step of the result, 2^-8 |O|, plus 2^-11 A + 2^-24 F for
        what comes before it.  The products are exact in the tensor cores'
        inputs but for P vs, which is rounded to f16, by 2^-11 of itself, at a
        scale where a row's largest is 4096 or more (and held as the sum of three
        e5m2 numbers, exactly).  Below f16's normal range it is off by 2^-23 at
        most, against the largest's 4096 2^-35 of max_j (P_j vs_j), for each key's
        |v8|: that is 2^-35 F; the 2^-24 F here are from a form of e4m3 parts.
        Scores and sums are fp32: with |s| <= 2^6 a score is off by a few 2^-24 *
        2^6 = 2^-18, its exponential by as much of itself.
  lse : 2^-13 absolute: the score error above, the fp32 logarithm and sum.
"""
import math

import numpy as np
import pytest
import torch

import synth
from exact_attention_94_gb300 import _lib, ops
from oracle import serving

pytestmark = pytest.mark.gpu


def make(lens, Nq, Hq, Hkv, d, P, seed=0, amp=1.0, garbage=True):
    """A cache of quantised normal values; slots that no request holds, and whole
    spare pages, are NaN codes with NaN scales; tables are padded with nonsense."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    blocks = [-(-n // P) for n in lens]
    pages, mb = sum(blocks) + 2, max(1, max(blocks)) + 1
    order = rng.permutation(pages)
    table = rng.integers(-10, 10 ** 6, (len(lens), mb))
    out, at = {}, 0
    held = np.zeros((pages, P), bool)
    for b, n in enumerate(lens):
        table[b, :blocks[b]] = order[at:at + blocks[b]]
        at += blocks[b]
        for j in range(n):
            held[table[b, j // P], j % P] = True
    for name in ("k", "v"):
        x = torch.randn((pages, Hkv, P, d), generator=g).numpy() * (amp * 2.0 ** rng.integers(-3, 3, (pages, Hkv, 1, 1)))
        codes, scales = np.empty(x.shape, np.uint8), np.empty((pages, Hkv), np.float32)
        for p in range(pages):
            for h in range(Hkv):
                scales[p, h] = serving.pow2_scale(np.abs(x[p, h]).max()) if held[p].any() or not garbage else np.nan
                codes[p, h] = serving._encode(x[p, h] / scales[p, h])
        if garbage:
            codes[~np.broadcast_to(held[:, None, :], codes.shape[:3])] = 0x7F
        out[name] = (codes, scales)
    q = (torch.randn((len(lens), Nq, Hq, d), generator=g)).to(torch.bfloat16)
    return q, out["k"], out["v"], table, np.array(lens)


def cu(a, dt):
    return torch.tensor(np.ascontiguousarray(a), dtype=dt).cuda()


def dev(case):
    q, (kc, ks), (vc, vs), table, lens = case
    return (q.cuda(), cu(kc, torch.uint8), cu(vc, torch.uint8), cu(ks, torch.float32), cu(vs, torch.float32),
            cu(table, torch.int32), cu(lens, torch.int32))


def assert_close(o, lse, ref):
    o_ref, l_ref, a, f = ref
    o, lse = synth.to_f64(o), lse.cpu().numpy()
    assert np.all(np.isfinite(o))
    err = np.abs(o - o_ref)
    tol = 2.0 ** -8 * np.abs(o_ref) + 2.0 ** -11 * a + 2.0 ** -24 * f
    assert np.all(err <= tol), float((err - tol).max())
    none = np.isneginf(l_ref)
    assert np.array_equal(none, np.isneginf(lse))
    assert np.all(np.abs(lse[~none] - l_ref[~none]) <= 2.0 ** -13)
    assert np.all(o[np.moveaxis(none, 1, 2)] == 0)


def check(case, window=-1, shares=0, L=None, scale=None):
    q, (kc, ks), (vc, vs), table, lens = case
    sc = 1 / math.sqrt(q.shape[3]) if scale is None else scale
    L = int(lens.max()) if L is None else L
    o, lse = ops.decode_kv8(*dev(case), L, window_left=window, num_shares=shares, scale=scale)
    assert ops.device_error() == 0
    assert_close(o, lse, serving.decode_kv8(synth.to_f64(q), kc, vc, ks, vs, table, lens, window, sc))
    return o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("P", [16, 48, 64, 128, 256])
def test_lengths_around_every_border(d, P):
    lens = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]
    check(make(lens, 1, 4, 2, d, P, seed=P + d))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (8, 1), (7, 1), (12, 4), (16, 1), (40, 2), (33, 1), (64, 1)])
def test_head_groups(d, Hq, Hkv):
    check(make([200, 1, 130], 1, Hq, Hkv, d, 16, seed=Hq))


@pytest.mark.parametrize("Nq", [2, 3, 4, 8, 17])
@pytest.mark.parametrize("Hq,Hkv,d", [(2, 2, 64), (8, 2, 128), (10, 2, 128), (8, 1, 64)])
def test_drafts(Nq, Hq, Hkv, d):
    """Rows of one request end at different keys; the first rows of short requests see none."""
    check(make([1, 3, 130, 257, 0], Nq, Hq, Hkv, d, 32, seed=Nq))


@pytest.mark.parametrize("window", [0, 1, 15, 100, 127, 128, 129, 1000])
@pytest.mark.parametrize("Nq", [1, 4])
@pytest.mark.parametrize("d", [64, 128])
def test_windows(window, Nq, d):
    check(make([1, 2, 128, 129, 300, 511, 0], Nq, 4, 2, d, 16, seed=window), window=window)
    check(make([300, 700], Nq, 4, 1, d, 64, seed=window), window=window, shares=3)


@pytest.mark.parametrize("shares", [1, 2, 3, 5, 7, 16, 64])
@pytest.mark.parametrize("Nq", [1, 9])
def test_any_number_of_shares(shares, Nq):
    """Shares of several requests, requests of several shares, more shares than tiles; a capacity above the lengths.
    (Nq = 9: the 36 query rows of a K/V head take two tiles.)"""
    case = make([1, 640, 0, 129, 0], Nq, 8, 2, 128, 16, seed=3)
    check(case, shares=shares)
    check(case, shares=shares, L=656)


def test_rising_scores():
    """Keys whose scores grow tile by tile: the reference moves again and again, in every way that it can."""
    for up in (0.5, 2.0, 40.0):
        q, (kc, ks), (vc, vs), table, lens = make([1000], 1, 8, 2, 128, 16, seed=4)
        q = torch.ones_like(q)
        for j in range(63):
            kc[table[0, j]] = serving._encode(np.full((2, 16, 128), 1.0))
            ks[table[0, j]] = 2.0 ** -6 * (j // 8 * up + (j % 3) * 0.25)
        check((q, (kc, ks), (vc, vs), table, lens), shares=1)
        vs[table[0, :63]] = 2.0 ** np.arange(-31, 32)[:, None]          # and the value scales with them
        check((q, (kc, ks), (vc, vs), table, lens), shares=1)
        vs[table[0, :63]] = 2.0 ** np.arange(31, -32, -1)[:, None]
        check((q, (kc, ks), (vc, vs), table, lens), shares=2)


def test_large_and_small_values():
    check(make([300, 40], 1, 4, 2, 128, 16, seed=1, amp=2.0 ** 40), scale=2.0 ** -45)
    check(make([300, 40], 1, 4, 2, 128, 16, seed=1, amp=2.0 ** -40), scale=2.0 ** 35)
    q, k, v, table, lens = make([300, 40], 1, 4, 2, 64, 16, seed=2)
    q = q * torch.logspace(-25, 20, 64, base=2.0).to(torch.bfloat16)      # queries of a wide range
    check((q, k, v, table, lens), scale=2.0 ** -22)
    check(make([300, 40], 1, 4, 2, 64, 16, seed=2), scale=30.0 / 8)       # peaked: scores of a hundred and more


def test_pages_of_zeros_and_one_loud_page():
    q, (kc, ks), (vc, vs), table, lens = make([200], 1, 4, 2, 128, 16, seed=5)
    kc[table[0, 3]], ks[table[0, 3]] = 0, 0.0      # a page whose keys and values were all zero: scale 0
    vc[table[0, 3]], vs[table[0, 3]] = 0, 0.0
    vs[table[0, 7]] *= 2.0 ** 30
    check((q, (kc, ks), (vc, vs), table, lens))
    vc[table[0, :13]], vs[table[0, :13]] = 0, 0.0  # no values at all
    o, lse = check((q, (kc, ks), (vc, vs), table, lens))
    assert torch.all(o == 0) and torch.isfinite(lse).all()


def test_a_loud_page_that_hardly_counts():
    """Values 2^40 times the others' in pages whose keys weigh 2^-98 of theirs: the quiet pages' average, to the
    same precision."""
    q, (kc, ks), (vc, vs), table, lens = make([400], 1, 4, 2, 128, 16, seed=6)
    q = torch.ones_like(q)
    for j in (0, 9, 24):
        kc[table[0, j]] = serving._encode(np.full((2, 16, 128), -1.0))
        ks[table[0, j]] = 68 * 128 ** -0.5            # scores of -68: e^-68 = 2^-98
        vs[table[0, j]] *= 2.0 ** 40
    check((q, (kc, ks), (vc, vs), table, lens), shares=2)
    o, _ = check((q, (kc, ks), (vc, vs), table, lens), shares=5)
    assert float(o.float().abs().max()) < 100


def test_equal_keys_average_the_values():
    """With q = 0 every weight is 1 / n and lse = log n, whatever the keys."""
    for n in (1, 100, 1000):
        q, k, v, table, lens = make([n], 1, 2, 1, 64, 16, seed=n)
        o, lse = check((q * 0, k, v, table, lens))
        assert np.all(np.abs(lse.cpu().numpy() - math.log(n)) <= 2.0 ** -13)


def test_bad_tables_and_lengths_are_reported():
    q, k, v, table, lens = make([100, 50], 1, 4, 2, 64, 16, seed=6, garbage=False)
    a = dev((q, k, v, table, lens))
    for bad in (-1, k[0].shape[0], 2 ** 31 - 1):
        t = a[5].clone()
        t[0, 2] = bad
        ops.decode_kv8(*a[:5], t, a[6], 100)
        assert ops.device_error() == 0x2000
    for n in (-5, 101, 2 ** 31 - 1):
        s = a[6].clone()
        s[1] = n
        o, lse = ops.decode_kv8(*a[:5], a[5].clamp(0, k[0].shape[0] - 1), s, 100)
        assert ops.device_error() == 0x2001
        if n < 0:
            assert torch.all(o[1] == 0) and torch.all(lse[1] == -math.inf)


def test_a_captured_call_follows_the_lengths():
    case = make([700, 300], 1, 8, 2, 128, 16, seed=7)
    a = dev(case)
    ws = torch.empty(_lib.load().fa_decode_kv8_workspace_bytes(2, 1, 8, 2, 128, 456), dtype=torch.uint8, device="cuda")
    ops.decode_kv8(*a, 700, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = ops.decode_kv8(*a, 700, workspace=ws)
    ws.fill_(0xFF)
    for lens in ([700, 300], [1, 0], [512, 129]):
        a[6].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        q, (kc, ks), (vc, vs), table, _ = case
        assert_close(o, lse, serving.decode_kv8(synth.to_f64(q), kc, vc, ks, vs, table, lens, -1, 128 ** -0.5))
    assert ops.device_error() == 0


def test_two_calls_at_once_and_another_stream():
    one, two = make([700], 1, 8, 2, 128, 16, seed=8), make([650, 3], 1, 4, 2, 64, 32, seed=9)
    a, b = dev(one), dev(two)
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(20):
        got.append((ops.decode_kv8(*a, 700, stream=s), ops.decode_kv8(*b, 650, stream=t)))
    s.synchronize(), t.synchronize()
    for x, case in ((0, one), (1, two)):
        q, (kc, ks), (vc, vs), table, lens = case
        ref = serving.decode_kv8(synth.to_f64(q), kc, vc, ks, vs, table, lens, -1, q.shape[3] ** -0.5)
        for pair in got:
            assert_close(*pair[x], ref)


def test_refusals():
    a = list(dev(make([20], 1, 4, 2, 64, 16)))
    with pytest.raises(ValueError):
        ops.decode_kv8(a[0][..., :32], *a[1:], 20)
    with pytest.raises(ValueError):
        ops.decode_kv8(*a, 20, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(_lib.FaError):
        ops.decode_kv8(*a, 10 ** 6)                       # more keys than the table has blocks for
    with pytest.raises(_lib.FaError):
        ops.decode_kv8(a[0][:, :, :3].contiguous(), *a[1:], 20)
    with pytest.raises(ValueError):
        ops.decode_kv8(a[0].repeat(1, 1, 1, 2)[..., ::2], *a[1:], 20)


@pytest.mark.parametrize("Hq,d", [(2, 64), (8, 128), (16, 128)])
def test_nan_in_a_draft_stays_with_the_rows_that_see_it(Hq, d):
    """A NaN among the values (or keys) of a draft token: rows before that token are
    what they are without it; rows that see it are NaN, their lse only if the key is."""
    Nq, Hkv, n = 4, 2, [130, 257]
    case = make(n, Nq, Hq, Hkv, d, 16, seed=Hq + d)
    q, (kc, ks), (vc, vs), table, lens = case
    j = n[0] - 2                                   # seen by the last two rows of request 0
    vc[table[0, j // 16], 0, j % 16, 5] = 0xFF
    j = n[1] - 1                                   # seen by the last row of request 1
    kc[table[1, j // 16], 1, j % 16, 3] = 0x7F
    o, lse = ops.decode_kv8(*dev(case), 257)
    assert ops.device_error() == 0
    with np.errstate(invalid="ignore"):
        o_ref, l_ref, a, f = serving.decode_kv8(synth.to_f64(q), kc, vc, ks, vs, table, lens, -1, d ** -0.5)
    bad = np.zeros((2, Nq, Hq), bool)
    bad[0, 2:, :Hq // 2] = True
    bad[1, 3:, Hq // 2:] = True
    o, lse = synth.to_f64(o), lse.cpu().numpy()
    assert np.all(np.isnan(o[bad])) and np.all(np.isnan(o_ref[bad]).any(-1))
    good = ~bad
    assert np.all(np.abs(o - o_ref)[good] <= (2.0 ** -8 * np.abs(o_ref) + 2.0 ** -11 * a + 2.0 ** -24 * f)[good])
    none = np.isnan(l_ref)
    assert np.array_equal(np.isnan(lse), none) and none.sum() == Hq // 2
    assert np.all(np.abs(lse - l_ref)[~none] <= 2.0 ** -13)


def test_queries_that_are_no_numbers():
    """An infinity or a NaN in a query row makes that row NaN, and no other."""
    q, k, v, table, lens = make([200, 3], 2, 8, 2, 128, 16, seed=12)
    q[0, 0, 1, 7], q[1, 1, 6, 0] = float("inf"), float("nan")
    o, lse = ops.decode_kv8(*dev((q, k, v, table, lens)), 200)
    bad = torch.zeros((2, 2, 8), dtype=torch.bool, device="cuda")
    bad[0, 0, 1] = bad[1, 1, 6] = True
    assert torch.equal(torch.isnan(o).all(-1), bad) and torch.equal(torch.isnan(o).any(-1), bad)
    assert torch.equal(torch.isnan(lse).transpose(1, 2), bad)


def test_pages_beyond_4_gib():
    """Offsets that pass 32 bits: a few pages at the end of a cache of 5 GiB a side."""
    Hkv, P, d, pages = 8, 64, 128, 5 * 2 ** 30 // (8 * 64 * 128)
    kc, vc = (torch.zeros((pages, Hkv, P, d), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, Hkv), device="cuda") for _ in range(2))
    n = 150
    table = np.array([[pages - 1, 3, pages - 2]])
    rows = np.arange(n)
    x = torch.randn((2, n, Hkv, d), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    ops.kv8_append(x[0].cuda(), x[1].cuda(), kc, vc, ks, vs, cu(table[0, rows // P], torch.int32),
                   cu(rows % P, torch.int32))
    q = torch.randn((1, 1, 16, d), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    o, lse = ops.decode_kv8(q.cuda(), kc, vc, ks, vs, cu(table, torch.int32), cu([n], torch.int32), n)
    assert ops.device_error() == 0
    at = torch.tensor(table[0], device="cuda")
    small = [t[at].cpu().numpy() for t in (kc, vc, ks, vs)]
    ref = [(np.zeros((3, Hkv, P, d), np.uint8), np.zeros((3, Hkv), np.float32)) for _ in range(2)]
    for y, (c, s) in zip(x, ref):
        serving.kv8_append(synth.to_f64(y), c, s, (rows // P).tolist(), (rows % P).tolist())
    for side in (0, 1):
        assert np.array_equal(small[side], ref[side][0]) and np.array_equal(small[2 + side], ref[side][1])
    assert_close(o, lse, serving.decode_kv8(synth.to_f64(q), ref[0][0], ref[1][0], ref[0][1], ref[1][1], np.array([[0, 1, 2]]),
                                            [n], -1, d ** -0.5))
    assert int((kc[4:-2] != 0).sum()) == 0 and int((vc[:3] != 0).sum()) == 0


@pytest.mark.parametrize("P,d", [(16, 64), (16, 128), (32, 128), (64, 64), (128, 128), (256, 64), (48, 128)])
@pytest.mark.parametrize("window,Nq", [(0, 1), (60, 1), (127, 3), (200, 4)])
def test_pages_before_the_window_may_be_gone(P, d, window, Nq):
    """A server frees them: their entries are nonsense, and the pages, if they still
    are any, hold NaN codes and NaN scales."""
    lens = [700, 333, 1, 129 + Nq, 512]
    q, (kc, ks), (vc, vs), table, lens = make(lens, Nq, 4, 2, d, P, seed=P + window)
    ref = serving.decode_kv8(synth.to_f64(q), kc, vc, ks, vs, table, lens, window, d ** -0.5)
    for b, n in enumerate(lens):
        for blk in range(max(0, n - Nq - window) // P):
            for codes, scales in ((kc, ks), (vc, vs)):
                codes[table[b, blk]], scales[table[b, blk]] = 0x7F, np.nan
            table[b, blk] = (-1, 10 ** 6, table[b, blk])[blk % 3]
    for shares in (0, 1, 7):
        o, lse = ops.decode_kv8(*dev((q, (kc, ks), (vc, vs), table, lens)), 700, window_left=window, num_shares=shares)
        assert ops.device_error() == 0
        assert_close(o, lse, ref)


@pytest.mark.parametrize("B,Nq,Hq,Hkv,shares", [(240, 1, 4, 2, 0), (90, 1, 4, 2, 37), (200, 3, 12, 1, 0), (600, 1, 1, 1, 11),
                                                (1, 1, 8, 2, 0), (1, 4, 16, 1, 0), (3, 1, 1, 1, 900)])
def test_units_fewer_and_more_than_shares(B, Nq, Hq, Hkv, shares):
    """Many short requests, some without keys, whose units the borders of few shares
    cut; and few long ones, each in many shares."""
    rng = np.random.default_rng(B + Nq)
    lens = rng.integers(0, 260, B) * (rng.random(B) < 0.9) if B > 3 else [5000, 0, 1700][:B]
    check(make([int(n) for n in lens], Nq, Hq, Hkv, 64, 16, seed=B), shares=shares)
    check(make([int(n) for n in lens], Nq, Hq, Hkv, 64, 16, seed=B), shares=shares, window=130)


def test_what_the_workspace_held_does_not_matter():
    """A captured call replayed over a workspace of every sort of content, and with many pieces a unit."""
    a = dev(make([3000, 17], 1, 4, 2, 64, 16, seed=13))
    ws = torch.empty(_lib.load().fa_decode_kv8_workspace_bytes(2, 1, 4, 2, 64, 90), dtype=torch.uint8, device="cuda")
    want = ops.decode_kv8(*a, 3000, num_shares=90)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, lse = ops.decode_kv8(*a, 3000, num_shares=90, workspace=ws)
    for fill in (0, 0xFF, 0x01, None, None, 0x80):
        if fill is not None:
            ws.fill_(fill)
        o.zero_(), lse.zero_()
        g.replay()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    q, k, v, table, lens = make([3000, 17], 1, 4, 2, 64, 16, seed=13)
    assert_close(o, lse, serving.decode_kv8(synth.to_f64(q), k[0], v[0], k[1], v[1], table, lens, -1, 64 ** -0.5))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("Hq,d", [(2, 64), (4, 128), (8, 128), (16, 64), (16, 128)])
def test_a_value_scale_that_is_no_number_stays_with_the_rows_that_see_its_page(Hq, d, value):
    """A page that opens between two drafts, and one that ends between two drafts' windows."""
    Nq, Hkv, n, window = 4, 2, [130, 257], 15
    case = make(n, Nq, Hq, Hkv, d, 16, seed=Hq + d)
    q, (kc, ks), (vc, vs), table, lens = case
    ref = serving.decode_kv8(synth.to_f64(q), kc, vc, ks, vs, table, lens, window, d ** -0.5)
    vs[table[0, 8], 0] = value        # keys 128, 129: the last two rows of request 0
    vs[table[1, 14], 1] = value       # keys up to 239, windows from 238, 239, 240, 241: the first two of request 1
    bad = np.zeros((2, Nq, Hq), bool)
    bad[0, 2:, :Hq // 2] = True
    bad[1, :2, Hq // 2:] = True
    for shares in (0, 1):
        o, lse = ops.decode_kv8(*dev(case), 257, window_left=window, num_shares=shares)
        assert ops.device_error() == 0
        o, lse = synth.to_f64(o), lse.cpu().numpy()
        o_ref, l_ref, a, f = ref
        assert np.all(np.isnan(o[bad]))
        assert np.all(np.abs(o - o_ref)[~bad] <= (2.0 ** -8 * np.abs(o_ref) + 2.0 ** -11 * a + 2.0 ** -24 * f)[~bad])
        assert np.all(np.abs(lse - l_ref) <= 2.0 ** -13)


@pytest.mark.parametrize("n", [1000, 32768, 300000])
@pytest.mark.parametrize("Hq,d", [(1, 64), (8, 128), (16, 64), (32, 128)])
@pytest.mark.parametrize("gap", [10.0, 17.0, 24.0])
def test_many_quiet_keys_beside_a_loud_one(gap, Hq, d, n):
    """A first key `gap` above all others, whose value is 0 where theirs is 1: O = m / (1 + m)
    with m = (n - 1) e^-gap, in one piece.  Each probability is rounded to f16, by 2^-11
    of itself, or, below 2^-25 of the largest, by 2^-35 of that."""
    P, blocks = 128, -(-n // 128)
    kc = torch.zeros((2, 1, P, d), dtype=torch.uint8, device="cuda")
    vc = torch.full_like(kc, 0x38)                   # 1
    kc[1, 0, 0, 0], vc[1, 0, 0] = 0x38, 0
    ones = torch.ones((2, 1), device="cuda")
    table = torch.zeros((1, blocks), dtype=torch.int32, device="cuda")
    table[0, 0] = 1
    q = torch.zeros((1, 1, Hq, d), dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    o, lse = ops.decode_kv8(q, kc, vc, ones, ones, table, cu([n], torch.int32), n, num_shares=1, scale=gap)
    assert ops.device_error() == 0
    m = (n - 1) * math.exp(-gap)
    want = m / (1 + m)
    tol = (2.0 ** -8 + 2.0 ** -11) * want + n * 2.0 ** -35
    assert np.all(np.abs(synth.to_f64(o) - want) <= tol), (float(o.float().max()), want)
    assert np.all(np.abs(lse.cpu().numpy() - gap - math.log1p(m)) <= 2.0 ** -13)


@pytest.mark.parametrize("Hq,d", [(2, 64), (8, 128), (16, 128), (32, 64)])
def test_scores_that_fall_and_rise(Hq, d):
    """Keys whose scores fall tile by tile, jump, and fall again; the loudest tiles' values are zero in the
    first half of the channels, so that the quiet tiles' weigh alone there."""
    P, tiles, Hkv = 128, 20, 1
    rng = np.random.default_rng(Hq)
    for step in (2.0, 7.0, 18.0):                    # log2 units a tile
        level = -step * (np.arange(tiles) % 7) + 3.0 * (np.arange(tiles) // 7)
        q, (kc, ks), (vc, vs), table, lens = make([tiles * P - 5], 1, Hq, Hkv, d, P, seed=Hq, garbage=False)
        q = torch.zeros_like(q)
        q[..., 0] = 1
        q[0, 0, :, 1] = torch.linspace(0.25, 1.0, Hq)    # rows differ by how far their keys spread
        for t in range(tiles):
            pg = table[0, t]
            kc[pg], ks[pg] = 0, 1.0
            x = np.zeros((P, d))
            x[:, 0] = abs(level[t]) if level[t] else 0
            x[:, 1] = rng.uniform(-2, 2, P)
            kc[pg, 0] = serving._encode(x * (np.arange(d) < 2) * np.where(np.arange(d) == 0, np.sign(level[t]), 1))
            if t % 7 == 0:
                vc[pg, 0, :, :d // 2] = 0
            vs[pg] = 2.0 ** rng.integers(-4, 4)
        case = (q, (kc, ks), (vc, vs), table, lens)
        for shares in (1, 2):
            check(case, shares=shares, scale=math.log(2))


@pytest.mark.parametrize("up", [84, 40, -40, -70])
@pytest.mark.parametrize("Hq,d", [(2, 64), (16, 128), (64, 128)])
def test_value_scales_at_both_ends_of_their_range(Hq, d, up):
    """Scales (2^-10 to 2^-4 before) up to 2^80 and down to 2^-80, with scores of a hundred and more."""
    q, k, (vc, vs), table, lens = make([300, 40], 1, Hq, 2, d, 16, seed=abs(up))
    assert 2.0 ** -80 <= np.nanmin(vs) * 2.0 ** up and np.nanmax(vs) * 2.0 ** up <= 2.0 ** 80
    for scale in (30.0 / 8, d ** -0.5, 0.001):
        check((q, k, (vc, (vs * 2.0 ** up).astype(np.float32)), table, lens), scale=scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Hq,Hkv", [(1, 4, 2), (1, 16, 2), (1, 32, 2), (2, 16, 2), (4, 16, 2), (1, 12, 1)])
def test_more_tiles_than_ctas(Nq, Hq, Hkv, d):
    """Where the tiles outnumber the CTAs that run at once, units weigh more than their
    tiles when work is dealt: for every tile of rows, of 4 to 32, with and without a window."""
    B = 240 if Hkv > 1 else 320
    rng = np.random.default_rng(Hq + d)
    lens = [int(n) for n in rng.integers(0, 300, B) * (rng.random(B) < 0.9)]
    tiles = B * Hkv * -(-Nq * Hq // Hkv // 32) * -(-max(lens) // 128)
    assert tiles > 2 * 3 * 152
    case = make(lens, Nq, Hq, Hkv, d, 32, seed=B)
    q, (kc, ks), (vc, vs), table, _ = case
    for window in (-1, 150):
        ref = serving.decode_kv8(synth.to_f64(q), kc, vc, ks, vs, table, np.array(lens), window, d ** -0.5)
        for shares in (0, 101):
            o, lse = ops.decode_kv8(*dev(case), max(lens), window_left=window, num_shares=shares)
            assert_close(o, lse, ref)
    assert ops.device_error() == 0


def test_no_keys_at_all():
    """Room for no key, and lengths of 0: O = 0, lse = -inf, whatever the table and the pages hold."""
    for B, Nq, Hq, Hkv in ((1, 1, 1, 1), (3, 4, 16, 2), (500, 1, 8, 2)):
        q, k, v, table, lens = make([0] * B, Nq, Hq, Hkv, 64, 16)
        for L in (0, 16):
            o, lse = ops.decode_kv8(*dev((q, k, v, table, lens)), L)
            assert ops.device_error() == 0
            assert torch.all(o == 0) and torch.all(lse == -math.inf)
