"""Refusals of the sampling-step entry points: bad arguments are turned away on
the host, before anything touches a GPU."""
import ctypes
import math

import pytest
import torch

from exact_attention_94_gb300 import _lib, build, ops
from tests.test_serving_abi import A, B16, INV, MIS, MISAL, NUL, UNS, rope_plan


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_norm(lib):
    def f(plan=None, q=A, k=A, qo=A, ko=A, wq=A, wk=A, pos=A, T=4, Hq=2, Hkv=1, d=64, qs=128, ks=64, qos=128, kos=64, wide=0,
          eps=1e-6):
        return lib.fa_qk_norm_rope(q, k, qo, ko, wq, wk, pos, ctypes.byref(plan or rope_plan()), T, Hq, Hkv, d, qs, ks, qos, kos,
                                   wide, eps, NUL)
    assert lib.fa_qk_norm_rope(A, A, A, A, A, A, A, None, 4, 2, 1, 64, 128, 64, 128, 64, 0, 1e-6, NUL) == INV
    for kw in (dict(n_axes=0), dict(n_axes=5), dict(neighbours=2), dict(axis=1), dict(freq=math.inf)):
        assert f(rope_plan(**kw)) == INV, kw
    for kw in (dict(T=-1), dict(Hq=-1), dict(Hq=0, Hkv=0), dict(Hq=65535), dict(q=NUL), dict(ko=NUL), dict(pos=NUL), dict(wq=NUL),
               dict(wk=NUL), dict(qs=120), dict(kos=56), dict(wide=2), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
               dict(qs=256)):  # (the last: in place with two strides)
        assert f(**kw) == INV, kw
    for kw in (dict(q=MIS), dict(ko=MIS), dict(pos=MIS), dict(qo=B16, qs=132), dict(wq=MIS, wide=1)):
        assert f(**kw) == MISAL, kw
    assert f(d=96) == UNS
    assert f(T=0) == _lib.FA_OK


def test_norm_gradient(lib):
    def f(ptrs=(A,) * 11, T=4, Hq=2, Hkv=1, d=64, strides=(128, 64) * 3, wide=0, eps=1e-6, ws=A, plan=None):
        return lib.fa_qk_norm_rope_bwd(*ptrs, ctypes.byref(plan or rope_plan()), T, Hq, Hkv, d, *strides, wide, eps, ws, NUL)
    for kw in (dict(T=-1), dict(Hq=-1), dict(Hq=0, Hkv=0), dict(Hq=65535), dict(wide=-1), dict(eps=-1.0), dict(ws=NUL),
               dict(strides=(120, 64) * 3), dict(strides=(128, 64, 128, 64, 256, 64))):
        assert f(**kw) == INV, kw
    for i in range(11):
        assert f(ptrs=tuple(NUL if j == i else A for j in range(11))) == INV, i
        if i not in (6, 7):  # weights of bf16 lie at any even address
            assert f(ptrs=tuple(MIS if j == i else A for j in range(11))) == MISAL, i
    assert f(ws=MIS) == MISAL and f(d=32) == UNS
    size = lib.fa_qk_norm_rope_bwd_workspace_bytes
    assert size(16384, 32, 8, 128) > 0 and size(0, 1, 0, 64) > 0
    for a in ((-1, 2, 1, 64), (4, -1, 1, 64), (4, 0, 0, 64), (4, 65535, 1, 64), (4, 2, 1, 96)):
        assert size(*a) == 0, a


@pytest.mark.parametrize("kv8", [False, True])
def test_shared(lib, kv8):
    n = 11 if kv8 else 9

    def f(ptrs=(A,) * n, B=2, Nq=1, Hq=4, Hkv=2, d=128, page=16, pages=8, blocks=4, L=64, G=1, wl=-1, shares=1, ws=A, sc=0.1):
        call = lib.fa_decode_kv8_shared if kv8 else lib.fa_decode_paged_shared
        return call(*ptrs, B, Nq, Hq, Hkv, d, page, pages, blocks, L, G, wl, shares, ws, sc, NUL)
    for kw in (dict(B=0), dict(B=16385), dict(Nq=0), dict(Hq=0), dict(Hkv=0), dict(Hkv=3), dict(page=8), dict(page=20),
               dict(pages=0), dict(blocks=0), dict(L=65), dict(L=-1), dict(wl=-2), dict(shares=-1), dict(shares=65536), dict(G=0),
               dict(G=3), dict(ws=NUL), dict(sc=0.0), dict(sc=math.nan), dict(Nq=20000), dict(pages=1 << 30, Hkv=2),
               dict(blocks=1 << 27, L=(1 << 30) + 1)):
        assert f(**kw) == INV, kw
    for i in range(n):
        assert f(ptrs=tuple(NUL if j == i else A for j in range(n))) == INV, i
        assert f(ptrs=tuple(MIS if j == i else A for j in range(n))) == MISAL, i
    assert f(ws=MIS) == MISAL
    assert f(d=96) == UNS and f(Hq=129, Hkv=1) == UNS


def test_workspace_of_shared(lib):
    size = lib.fa_decode_shared_workspace_bytes
    a = dict(B=8, Nq=1, Hq=8, Hkv=2, d=128, G=2, shares=3)
    assert size(*a.values()) >= 4 * 8 * 8 * (128 + 1) * 4
    for bad in (dict(B=0), dict(B=16385), dict(Nq=0), dict(Hq=0), dict(Hkv=3), dict(d=96), dict(G=0), dict(G=9), dict(shares=-1),
                dict(shares=65536), dict(Nq=20000), dict(Hq=129, Hkv=1), dict(Nq=2 ** 31 - 1, Hq=2 ** 31 - 1, Hkv=1)):
        assert size(*{**a, **bad}.values()) == 0, bad
    # more of anything takes no less, in 64 bits
    assert size(16384, 1, 64, 8, 128, 16384, 65535) > size(16384, 1, 64, 8, 128, 1, 152) > 2 ** 31


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1])
def test_numbers_beyond_32_bits(n):
    for args in ((n, -1, 0), (777, n, 0), (777, -1, n)):
        with pytest.raises(ValueError):
            ops._shared_bytes(0, 1, 1, 8, 8, 128, 1, *args)


def test_python_side():
    p = ops.rope_plan(64, [32])
    x, w, i = torch.zeros((2, 1, 64), dtype=torch.bfloat16), torch.ones(64), torch.zeros((1, 2), dtype=torch.int32)
    with pytest.raises(ValueError):  # not on a GPU
        ops.qk_norm_rope(x, x, w, w, i, p)
    with pytest.raises(TypeError):
        ops.qk_norm_rope(x, None, w, None, i, "plan")
    with pytest.raises(ValueError):
        ops.qk_norm_rope(None, None, w, w, i, p)
    with pytest.raises(ValueError):
        ops.qk_norm_rope_bwd(x, None, None, None, w, w, i, p)
    c, s, t = torch.zeros((2, 1, 16, 64), dtype=torch.uint8), torch.zeros((2, 1)), torch.zeros((1, 1), dtype=torch.int32)
    q, k, n = x[:1, None], torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        ops.decode_paged_shared(q, k, k, t, n, torch.zeros(2, dtype=torch.int32), n, 16)
    with pytest.raises(ValueError):
        ops.decode_kv8_shared(q, c, c, s, s, t, n, torch.zeros(2, dtype=torch.int32), n, 16)
