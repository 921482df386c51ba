"""Refusals of the serving-step entry points: bad arguments are turned away on
the host, before anything touches a GPU."""
import ctypes
import math

import pytest
import torch

from exact_attention_94_gb300 import _lib, build, ops

P = ctypes.c_void_p
A, B16, NUL = P(4096), P(1 << 20), P(0)  # fake pointers, never dereferenced: validation fails first
MIS = P(4096 + 2)
INV, UNS, MISAL = _lib.FA_ERR_INVALID_ARG, _lib.FA_ERR_UNSUPPORTED, _lib.FA_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_page_plan(lib):
    def f(ptrs=(A,) * 11, B=2, cap=8, page=16, pages=4, blocks=2):
        return lib.fa_page_plan(*ptrs, B, cap, page, pages, blocks, NUL)
    for kw in (dict(B=0), dict(B=16385), dict(cap=-1), dict(page=0), dict(pages=0), dict(blocks=0)):
        assert f(**kw) == INV, kw
    for i in range(11):
        assert f(ptrs=tuple(NUL if j == i else A for j in range(11))) == INV, i
        assert f(ptrs=tuple(MIS if j == i else A for j in range(11))) == MISAL, i


def rope_plan(**kw):
    s = _lib.RopePlanStruct(kw.get("n_axes", 1), kw.get("neighbours", 0))
    s.axis[5] = kw.get("axis", 0)
    s.inv_freq[5] = kw.get("freq", 1.0)
    return s


def test_rope(lib):
    def f(plan=None, q=A, k=A, qo=A, ko=A, pos=A, T=4, Hq=2, Hkv=1, d=64, qs=128, ks=64, qos=128, kos=64, inv=0):
        return lib.fa_rope_axes(q, k, qo, ko, pos, ctypes.byref(plan or rope_plan()), T, Hq, Hkv, d, qs, ks, qos, kos,
                                inv, NUL)
    assert lib.fa_rope_axes(A, A, A, A, A, None, 4, 2, 1, 64, 128, 64, 128, 64, 0, NUL) == INV
    for kw in (dict(n_axes=0), dict(n_axes=5), dict(neighbours=2), dict(axis=1), dict(axis=-2), dict(freq=math.inf),
               dict(freq=math.nan)):
        assert f(rope_plan(**kw)) == INV, kw
    for kw in (dict(T=-1), dict(Hq=-1), dict(Hq=0, Hkv=0), dict(Hq=65535), dict(q=NUL), dict(ko=NUL), dict(pos=NUL),
               dict(qs=120), dict(kos=56), dict(inv=2), dict(qs=256)):  # (the last: in place with two strides)
        assert f(**kw) == INV, kw
    for kw in (dict(q=MIS), dict(ko=MIS), dict(pos=MIS), dict(qo=B16, qs=132), dict(k=B16, kos=68)):
        assert f(**kw) == MISAL, kw
    assert f(d=96) == UNS
    assert f(T=0) == _lib.FA_OK


def test_append(lib):
    def f(ptrs=(A,) * 8, src=NUL, n=2, Hkv=2, d=128, page=16, pages=3, ks=256, vs=256):
        return lib.fa_kv8_append(*ptrs, src, n, Hkv, d, page, pages, ks, vs, NUL)
    for kw in (dict(n=-1), dict(Hkv=0), dict(page=8), dict(page=24), dict(pages=0), dict(ks=128), dict(vs=248)):
        assert f(**kw) == INV, kw
    for i in range(8):
        assert f(ptrs=tuple(NUL if j == i else A for j in range(8))) == INV, i
        assert f(ptrs=tuple(MIS if j == i else A for j in range(8))) == MISAL, i
    assert f(src=MIS) == MISAL and f(ks=260) == MISAL
    assert f(d=32) == UNS
    assert f(n=0) == _lib.FA_OK


def test_decode(lib):
    def f(ptrs=(A,) * 9, B=1, Nq=1, Hq=4, Hkv=2, d=128, page=16, pages=8, blocks=4, L=64, wl=-1, shares=1, ws=A, sc=0.1):
        return lib.fa_decode_kv8(*ptrs, B, Nq, Hq, Hkv, d, page, pages, blocks, L, wl, shares, ws, sc, NUL)
    for kw in (dict(B=0), dict(B=16385), dict(Nq=0), dict(Hq=0), dict(Hkv=0), dict(Hkv=3), dict(page=8), dict(page=20),
               dict(pages=0), dict(blocks=0), dict(L=65), dict(L=-1), dict(wl=-2), dict(shares=-1), dict(shares=65536),
               dict(ws=NUL), dict(sc=0.0), dict(sc=math.nan), dict(Nq=20000), dict(pages=1 << 30, Hkv=2),
               dict(blocks=1 << 27, L=(1 << 30) + 1)):
        assert f(**kw) == INV, kw
    for i in range(9):
        assert f(ptrs=tuple(NUL if j == i else A for j in range(9))) == INV, i
        assert f(ptrs=tuple(MIS if j == i else A for j in range(9))) == MISAL, i
    assert f(ws=MIS) == MISAL
    assert f(d=96) == UNS


def test_workspace_and_shares(lib):
    assert lib.fa_decode_kv8_workspace_bytes(3, 2, 8, 2, 128, 5) >= 2 * 5 * 8 * (128 + 1) * 4
    assert lib.fa_decode_kv8_workspace_bytes(0, 2, 8, 2, 128, 5) == 0
    for a in ((1, 1, 8, 8, 0, -1), (1, 1, 8, 8, 1, -1), (64, 1, 64, 8, 32768, -1), (1, 8, 64, 1, 1 << 30, 5)):
        assert 1 <= lib.fa_decode_kv8_num_shares(*a) <= 65535


def test_sizes_that_a_call_refuses_have_no_workspace(lib):
    big = 2 ** 31 - 1
    for a in ((1, big, big, 1, 128, 5), (1, 70000, 1, 1, 128, 5), (1, 1, 70000, 1, 128, 5), (1, 1, 8, 8, 128, big)):
        assert lib.fa_decode_kv8_workspace_bytes(*a) == 0
    assert lib.fa_decode_kv8_num_shares(1, big, big, 1, 777, -1) == 1


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1])
def test_numbers_beyond_32_bits(n):
    """ctypes would pass their lower bits on."""
    for args in ((n, -1, 0), (777, n, 0), (777, -1, n)):
        with pytest.raises(ValueError):
            ops._kv8_shares(0, 1, 1, 8, 8, 128, *args)
    with pytest.raises(ValueError):
        ops._check_int("max_tokens", n)


def test_python_side():
    with pytest.raises(ValueError):
        ops.RopePlan(64, [0] * 31, [1.0] * 31)
    with pytest.raises(ValueError):
        ops.RopePlan(64, [4] * 32, [1.0] * 32)
    with pytest.raises(ValueError):
        ops.RopePlan(64, [0] * 32, [math.nan] * 32)
    with pytest.raises(_lib.FaError):
        ops.RopePlan(96, [0] * 48, [1.0] * 48)
    with pytest.raises(ValueError):
        ops.rope_plan(64, [16, 17])
    p = ops.rope_plan(64, [8, 8, 8])
    assert p.n_axes == 3 and list(p.struct.axis[:32]) == [0] * 8 + [1] * 8 + [2] * 8 + [-1] * 8
    x = torch.zeros((2, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # not on a GPU
        ops.rope_axes(x, x, torch.zeros((3, 2), dtype=torch.int32), p)
    with pytest.raises(TypeError):
        ops.rope_axes(x.float(), None, torch.zeros((3, 2), dtype=torch.int32), p)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.page_plan(i, i, i, i, torch.zeros((1, 1), dtype=torch.int32), 16, 1)
    with pytest.raises(ValueError):
        ops.kv8_append(x, x, x, x, x, x, i, i)


def test_workspace_of_an_automatic_choice(lib):
    """num_shares = 0, which the call takes: the query's bytes cover whatever it chooses."""
    for Nq, Hq, Hkv in ((1, 1, 1), (1, 8, 8), (1, 64, 8), (2, 64, 8), (4, 64, 8), (8, 64, 1), (65535, 1, 1)):
        for d in (64, 128):
            most = lib.fa_decode_kv8_workspace_bytes(16384, Nq, Hq, Hkv, d, 0)
            for B, L, window in ((1, 1, -1), (1, 777, -1), (64, 32768, -1), (16384, 1 << 30, -1), (16384, 1 << 30, 4095)):
                shares = lib.fa_decode_kv8_num_shares(B, Nq, Hq, Hkv, L, window)
                assert most >= lib.fa_decode_kv8_workspace_bytes(B, Nq, Hq, Hkv, d, shares) > 0
                assert lib.fa_decode_kv8_workspace_bytes(B, Nq, Hq, Hkv, d, 0) == most


@pytest.mark.parametrize("bad", [dict(B=0), dict(B=16385), dict(Nq=0), dict(Hq=0), dict(Hkv=0), dict(Hkv=3), dict(Hkv=8),
                                 dict(d=96), dict(d=32), dict(shares=-1), dict(shares=65536), dict(Nq=20000)])
def test_the_workspace_query_refuses_what_the_call_refuses(lib, bad):
    a = dict(B=1, Nq=1, Hq=4, Hkv=2, d=128, shares=1)
    assert lib.fa_decode_kv8_workspace_bytes(*a.values()) > 0
    a.update(bad)
    assert lib.fa_decode_kv8_workspace_bytes(*a.values()) == 0
    sizes = [a[x] for x in ("B", "Nq", "Hq", "Hkv", "d")]
    assert lib.fa_decode_kv8(*(A,) * 9, *sizes, 16, 8, 4, 64, -1, a["shares"], A, 0.1, NUL) in (INV, UNS)


def test_axes_without_pairs():
    """A model with three axes may give a head's pairs to fewer; its positions still have three."""
    for sections, n, used in (([32, 0, 0], 3, 1), ([16, 16, 0], 3, 2), ([0, 0, 8], 3, 3), ([0, 0], 2, 1), ([32], 1, 1),
                              ([8, 0, 8, 0], 4, 3)):
        p = ops.rope_plan(64, sections)
        assert p.n_axes == p.struct.n_axes == n and p.used_axes == used, sections
    assert ops.RopePlan(64, [0] * 32, [1.0] * 32).n_axes == 1
    assert ops.RopePlan(64, [0] * 32, [1.0] * 32, n_axes=4).n_axes == 4
    for axis, n in ((2, 2), (0, 0), (0, 5), (0, -1)):
        with pytest.raises(ValueError):
            ops.RopePlan(64, [axis] * 32, [1.0] * 32, n_axes=n)
