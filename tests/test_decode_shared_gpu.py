"""Attention of requests that share prefixes, over bf16 pages, against the
reference in 64 bits.

Tolerance of O: half a bf16 step, 2^-8 |o|; each probability is rounded to bf16
(2^-8 of itself at most; the sums use it unrounded), a = sum_j P_j |v_j| being
what it is a part of; the scores' fp32 sums of up to 128 products of bf16 are
off by 2^-17 sum |q_c k_c| at the very most, far less as errors differ in sign,
which with the fast exponential counts as 2^-12 of a here (|s| stays below 32):
2^-8 |o| + (2^-8 + 2^-11) a.  lse: 2^-12 absolutely, from the same.
"""
import numpy as np
import pytest
import torch

import synth
from exact_attention_94_gb300 import _lib, ops
from oracle import sampling

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32).cuda()


def make(groups, Nq, Hq, Hkv, d, P, seed=0, spare=3, fill=None):
    """groups: [(shared, [lengths])].  Tables as a server has them: a group's full pages in common (as far as each
    request reaches), its own pages behind, in any order; the partly filled shared page copied for each.  Unused slots and
    spare pages hold `fill`."""
    rng = np.random.default_rng(seed)
    lens = [n for _, ls in groups for n in ls]
    blocks = max(1, max(-(-n // P) for n in lens))
    starts = np.cumsum([0] + [len(ls) for _, ls in groups])
    need, table = 0, np.full((len(lens), blocks), -9)
    for g, (shared, ls) in enumerate(groups):
        full = min(shared, max(ls)) // P if ls else 0
        for x, n in enumerate(ls):
            for j in range(-(-n // P)):
                table[starts[g] + x, j] = need + j if j < full else -1
        need += full
    for b, j in np.argwhere(table == -1):
        table[b, j] = need
        need += 1
    pages = need + spare
    order = rng.permutation(pages)
    table = np.where(table >= 0, order[table], 0)
    gen = torch.Generator().manual_seed(seed)
    k, v = (torch.randn((pages, P, Hkv, d), generator=gen).to(torch.bfloat16) for _ in range(2))
    used = np.zeros((pages, P), bool)
    for g, (shared, ls) in enumerate(groups):
        first = max(range(len(ls)), key=lambda x: (ls[x], -x)) if ls else 0
        for x, n in enumerate(ls):
            for j in range(-(-n // P)):
                used[table[starts[g] + x, j], :max(0, min(P, n - j * P))] = True
            j = shared // P
            if shared % P and ls[first] > j * P and n > j * P:  # the copy of the partly filled page
                for t in (k, v):
                    t[table[starts[g] + x, j], :shared % P] = t[table[starts[g] + first, j], :shared % P]
    if fill is not None:
        k[~torch.tensor(used)] = fill
        v[~torch.tensor(used)] = fill
    q = (1.5 * torch.randn((len(lens), Nq, Hq, d), generator=gen)).to(torch.bfloat16)
    return dict(q=q, k=k, v=v, table=table, lens=lens, starts=starts, shared=[s for s, _ in groups], P=P)


def call(m, window=-1, max_len=None, **kw):
    return ops.decode_paged_shared(m["q"].cuda(), m["k"].cuda(), m["v"].cuda(), i32(m["table"]), i32(m["lens"]),
                                   i32(m["starts"]), i32(m["shared"]), max(m["lens"]) if max_len is None else max_len,
                                   window_left=window, **kw)


def want(m, window=-1):
    k, v = synth.to_f64(m["k"]), synth.to_f64(m["v"])
    return sampling.decode_shared(synth.to_f64(m["q"]), lambda p, t: k[p, t], lambda p, t: v[p, t], m["table"], m["lens"],
                                  m["starts"], m["shared"], m["P"], window, m["q"].shape[-1] ** -0.5)


def check(got, ref):
    o, lse, a = ref
    err = np.abs(synth.to_f64(got[0]) - o)
    tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -11) * a
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-30)).max())
    l = got[1].double().cpu().numpy()
    assert np.array_equal(np.isneginf(l), np.isneginf(lse))
    seen = ~np.isneginf(lse)
    assert np.all(np.abs(l[seen] - lse[seen]) <= 2.0 ** -12)
    assert ops.device_error() == 0


SHAPES = [
    [(100, [101, 120, 128, 350])],                  # one prompt, a few answers
    [(256, [257] * 9)],                             # whole tiles and one key each
    [(0, [1, 2, 130]), (17, [17, 40, 18]), (0, [5])],
    [(400, [401, 400, 399, 130, 0, 3])],            # requests shorter than what is shared, and empty ones
    [(64, [700]), (33, [34, 33]), (5, [])],         # a group of one, an empty group
]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Hq,Hkv", [(1, 4, 4), (1, 8, 1), (1, 10, 2), (3, 7, 1)])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("shares", [0, 1, 5])
def test_groups(d, Nq, Hq, Hkv, shape, shares):
    m = make(SHAPES[shape], Nq, Hq, Hkv, d, (16, 48, 128)[(shape + Nq) % 3], seed=shape, fill=float("nan"))
    check(call(m, num_shares=shares), want(m))


@pytest.mark.parametrize("heads,n", [(1, 300), (8, 40), (5, 60), (128, 3), (7, 37), (33, 13)])
def test_many_rows(heads, n):
    """Two tiles of rows, a third, tiles that heads do not fill."""
    m = make([(150, [151 + i % 20 for i in range(n)]), (40, [60] * 4)], 1, heads, 1, 64, 16, seed=n)
    ref = want(m)
    for shares in (0, 1, 7):
        check(call(m, num_shares=shares), ref)


@pytest.mark.parametrize("heads", [1, 8, 40])
def test_requests_without_keys_share_nothing(heads):
    """Whole tiles that every request with keys sees: one without sees none of them."""
    m = make([(520, [530, 0, 700, 0]), (300, [0, 300])], 1, heads, 1, 64, 16, seed=heads, fill=float("nan"))
    for shares in (0, 1):
        check(call(m, num_shares=shares), want(m))


@pytest.mark.parametrize("window", [0, 1, 40, 127, 300])
@pytest.mark.parametrize("Nq", [1, 4])
def test_windows(window, Nq):
    """Rows of one tile whose windows begin at different keys, pages in front that are gone."""
    m = make([(300, [301, 330, 420, 310, 300, 7, 0]), (100, [500, 103])], Nq, 4, 2, 64, 16, seed=window, fill=float("nan"))
    ref = want(m, window)
    for g, (s, e) in enumerate(zip(m["starts"], m["starts"][1:])):  # pages before every window of a request
        least = min(n for n in m["lens"][s:e] if n > 0)
        for b in range(s, e):
            gone = max(0, min(least, m["lens"][b]) - Nq - window) // 16
            m["table"][b, :gone] = 10 ** 6
    for shares in (0, 3):
        check(call(m, window, num_shares=shares), ref)


@pytest.mark.parametrize("Nq,window,key", [(1, -1, 30), (4, -1, 128), (4, -1, 127), (1, 20, 100), (3, 50, 60), (1, -1, 310)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_odd_values_stay_with_the_queries_that_see_them(Nq, window, key, bad):
    m = make([(90, [130, 131, 129, 320])], Nq, 4, 1, 128, 16, seed=5)
    plain = call(m, window)
    for b in range(4):
        if key < m["lens"][b]:
            m["v"][m["table"][b, key // 16], key % 16, 0, 3] = bad
    o, lse = call(m, window)
    assert torch.equal(lse, plain[1])
    for b in range(4):
        for i in range(Nq):
            pos = m["lens"][b] - Nq + i
            sees = key <= pos and (window < 0 or key >= pos - window)
            if sees:
                assert not torch.isfinite(o[b, i, :, 3]).any()
            else:
                assert torch.equal(o[b, i], plain[0][b, i]), (b, i)


def test_odd_keys():
    m = make([(90, [130, 131])], 2, 4, 1, 64, 16, seed=5)
    plain = call(m)
    m["k"][m["table"][0, 129 // 16], 129 % 16, 0, 3] = float("nan")  # the last key of the first request
    o, lse = call(m)
    assert torch.isnan(o[0, 1]).all() and torch.isnan(lse[0, :, 1]).all()
    assert torch.equal(o[0, 0], plain[0][0, 0]) and torch.equal(o[1], plain[0][1])


def test_long_scores_and_far_references():
    """Scores that rise through the keys move the rows' references again and again."""
    m = make([(600, [700, 640])], 1, 4, 2, 128, 16, seed=8)
    for j in range(700):
        for b in range(2):
            if j < m["lens"][b]:
                m["k"][m["table"][b, j // 16], j % 16] = (m["q"][b, 0, 0].float() * (j / 2000)).to(torch.bfloat16)
    o, lse, a = want(m)
    got = call(m)
    err = np.abs(synth.to_f64(got[0]) - o)
    # scores up to 70: 2^-24 of them in each of their sums' parts, 2^-13 of a probability
    assert np.all(err <= 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2.0 ** -10) * a)
    assert np.all(np.abs(got[1].double().cpu().numpy() - lse) <= 2.0 ** -10)


def test_bad_groups_share_nothing_and_are_reported():
    m = make([(100, [120, 130]), (50, [60, 200])], 1, 4, 2, 64, 16, seed=2)
    ref = want(m)
    for name, value in (("starts", [0, 5, 4]), ("starts", [1, 2, 4]), ("starts", [0, 2, 3]), ("starts", [0, -1, 4]),
                        ("shared", [-1, 50]), ("shared", [100, 10 ** 6])):
        bad = dict(m, **{name: value})
        got = call(bad)
        assert ops.device_error() == 0x2001
        check(got, ref)  # each request's own row names all its pages


def test_bad_pages_and_lengths_are_reported():
    m = make([(100, [120, 130]), (50, [60, 200])], 1, 4, 2, 64, 16, seed=2)
    plain = call(m)
    bad = dict(m, table=m["table"].copy())
    bad["table"][3, 11] = 10 ** 8
    o, _ = call(bad)
    assert ops.device_error() == 0x2000 and torch.equal(o[:3], plain[0][:3])
    o, _ = call(dict(m, lens=[120, 130, 60, 201]), max_len=200)
    assert ops.device_error() == 0x2001 and torch.equal(o, plain[0])
    o, lse = call(dict(m, lens=[120, 130, 60, -5]), max_len=200)
    assert ops.device_error() == 0x2001 and not o[3].any() and torch.isneginf(lse[3]).all()


def test_streams_graphs_and_a_shared_workspace():
    one, two = make([(100, [120, 130, 300])], 1, 8, 2, 128, 16, seed=1), make([(40, [90, 50])] * 3, 4, 8, 2, 64, 16, seed=2)
    plain = [call(one), call(two)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for m, p in zip((one, two), plain):
        o, lse = call(m, stream=s)
        s.synchronize()
        assert torch.equal(o, p[0]) and torch.equal(lse, p[1])
    size = _lib.load().fa_decode_shared_workspace_bytes
    ws = torch.empty(max(size(3, 1, 8, 2, 128, 1, 0), size(6, 4, 8, 2, 64, 3, 0)), dtype=torch.uint8, device="cuda")
    graphs, got = [], []
    for m in (one, two):
        args = (m["q"].cuda(), m["k"].cuda(), m["v"].cuda(), i32(m["table"]), i32(m["lens"]), i32(m["starts"]), i32(m["shared"]))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(ops.decode_paged_shared(*args, max(m["lens"]), workspace=ws))
        graphs.append((g, args))
    for _ in range(10):
        graphs[0][0].replay()
        graphs[1][0].replay()
    torch.cuda.synchronize()
    for x, y in zip(got, plain):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_it_agrees_with_the_decode_that_shares_nothing():
    m = make([(1000, [1001 + 37 * i for i in range(20)])], 1, 16, 4, 128, 16, seed=3)
    got = call(m)
    o, lse = ops.decode_paged_window(m["q"].cuda(), m["k"].cuda(), m["v"].cuda(), i32(m["table"]), i32(m["lens"]), max(m["lens"]))
    assert torch.allclose(got[1][..., 0], lse, atol=2.0 ** -11, rtol=0)
    assert (got[0].float() - o.float()).abs().max() <= 2.0 ** -7
