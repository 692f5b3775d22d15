"""CPU checks of the mixture-of-experts entry points: the argument checks run before
any CUDA call (status codes: 1 null, 2 shape, 3 alignment)."""
from __future__ import annotations

import ctypes

import pytest
import torch

import w8a8_int8_quantized_sq_b200 as sq
from w8a8_int8_quantized_sq_b200 import build as sq_build

OK = ctypes.c_void_p(0x100000)   # aligned, never dereferenced: the checks fail first
BAD = ctypes.c_void_p(0x100008)  # 8-byte aligned only


@pytest.fixture(scope="module")
def lib():
    sq_build.build()
    return sq.lib()


@pytest.mark.parametrize("name", ["w8a8_grouped_mm", "fp8_block_grouped_mm"])
def test_grouped_checks(lib, name):
    f = getattr(lib, name)

    def call(p=(OK,) * 7, T=4, M=4, E=2, N=128, K=256):
        return f(*p, T, M, E, N, K, None)

    for i in (0, 1, 3, 4, 5, 6):  # rows (2) may be NULL
        assert call(tuple(None if j == i else OK for j in range(7))) == 1
    for i in range(7):
        assert call(tuple(BAD if j == i else OK for j in range(7))) == 3
    assert call(K=200) == 2 and call(K=0) == 2 and call(K=131072 + 128) == 2
    assert call(N=24) == 2 and call(N=0) == 2
    assert call(E=0) == 2 and call(E=1025) == 2
    assert call(T=-1) == 2 and call(M=-1) == 2 and call(M=0) == 2
    assert call((OK, OK, None, OK, OK, OK, OK), T=4, M=5) == 2   # no rows: M is T
    assert call(T=1 << 31) == 2 and call(M=1 << 31) == 2
    assert call(E=1024, N=1 << 22) == 2                          # E N past 32 bits
    assert call(T=(1 << 31) - 1000, N=1 << 20) == 2              # tiles past 32 bits
    assert call(T=1 << 30, M=1 << 30, N=65536) == 2              # with 128-row tiles
    assert call((None,) * 7, T=0, M=0) == 0                      # nothing to do
    assert f(*(OK,) * 7, 4, 4, 2, 144, 256, None) == 2 if name.startswith("fp8") else True


def test_add_rmsnorm_checks(lib):
    f, g = lib.sq_add_rmsnorm_quant, lib.sq_add_rmsnorm_quant_fp8

    def call(h=OK, r=OK, gamma=OK, eps=1e-6, group=0, out=OK, q=OK, s=OK, M=4, K=256):
        a = f(h, r, gamma, eps, group, out, q, s, None, M, K, None)
        if group == 0:
            assert g(h, r, gamma, eps, out, q, s, None, M, K, None) == a
        return a

    assert call(K=200) == 2 and call(K=24576 + 128) == 2 and call(M=-1) == 2
    assert call(eps=0.0) == 2 and call(eps=float("nan")) == 2 and call(eps=float("inf")) == 2
    assert call(group=64) == 2
    assert call(M=0, h=None) == 0
    shifted = ctypes.c_void_p(0x100000 + 256 * 2)
    far = ctypes.c_void_p(0x900000)
    assert call(out=shifted) == 2                                # overlaps h by all but a row
    assert call(h=far, out=shifted) == 2 and call(r=far, out=shifted) == 2
    for name in ("h", "r", "gamma", "out", "q", "s"):
        assert call(**{name: None}) == 1
        assert call(**{name: BAD}) == 3


def test_silu_mul_checks(lib):
    f, g = lib.sq_silu_mul_quant, lib.sq_silu_mul_quant_fp8

    def call(x=OK, inv=None, group=0, q=OK, s=OK, T=4, K=256):
        a = f(x, inv, group, q, s, T, K, None)
        if group == 0:
            assert g(x, inv, q, s, T, K, None) == a
        return a

    assert call(K=200) == 2 and call(K=24576 + 128) == 2 and call(T=-1) == 2 and call(group=64) == 2
    assert call(T=0, x=None) == 0
    for name in ("x", "q", "s"):
        assert call(**{name: None}) == 1
        assert call(**{name: BAD}) == 3
    assert call(inv=BAD) == 3


def test_binding_refuses_cpu_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sq.silu_mul_quant(x)
    with pytest.raises(ValueError):
        sq.add_rmsnorm_quant(x, x, torch.ones(256), 1e-6)
    with pytest.raises(ValueError):
        sq.w8a8_grouped_mm(torch.zeros(4, 256, dtype=torch.int8), torch.ones(4),
                           torch.zeros(1, 16, 256, dtype=torch.int8), torch.ones(1, 16),
                           torch.zeros(2, dtype=torch.int32))
