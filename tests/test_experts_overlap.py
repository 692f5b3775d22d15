"""The expert entry points refuse an output that overlaps an input or another output (status 2),
and a 1/rms output that no float can be stored to (3).  Checked before any CUDA call; the
addresses are never dereferenced, and every call here is one to refuse."""
from __future__ import annotations

import ctypes

import pytest

import w8a8_int8_quantized_sq_b200 as sq
from w8a8_int8_quantized_sq_b200 import build as sq_build


@pytest.fixture(scope="module")
def lib():
    sq_build.build()
    return sq.lib()


def at(i, byte=0):
    return ctypes.c_void_p((i + 1 << 32) + byte)


def hits(sizes, outs):
    """(output, other, address of the output) for starts at the other's first and last 16 bytes,
    and for an output that ends in its first 16."""
    for o in outs:
        for i in range(len(sizes)):
            if i == o:
                continue
            yield o, i, at(i)
            if sizes[i] > 16:
                yield o, i, at(i, (sizes[i] - 1) // 16 * 16)
            if sizes[o] > 16:
                yield o, i, at(i, -((sizes[o] - 1) // 16 * 16))


@pytest.mark.parametrize("name", ["w8a8_grouped_mm", "fp8_block_grouped_mm"])
def test_grouped(lib, name):
    T, M, E, N, K = 40, 24, 3, 256, 384
    f8 = name.startswith("fp8")
    sizes = [M * K, M * (K // 128 if f8 else 1) * 4, T * 4, E * N * K,
             E * (N // 128 * (K // 128) if f8 else N) * 4, (E + 1) * 4, T * N * 2]
    for o, i, where in hits(sizes, [6]):
        p = [at(j) for j in range(7)]
        p[o] = where
        assert getattr(lib, name)(*p, T, M, E, N, K, None) == 2, (o, i, hex(where.value))


@pytest.mark.parametrize("group", [0, 128, "fp8"])
def test_norm(lib, group):
    M, K = 6, 384
    sizes = [M * K * 2, M * K * 2, K * 4, M * K * 2, M * K, M * 4 * (K // 128 if group else 1), M * 4]

    def call(p):
        if group == "fp8":
            return lib.sq_add_rmsnorm_quant_fp8(*p[:3], 1e-6, *p[3:], M, K, None)
        return lib.sq_add_rmsnorm_quant(*p[:3], 1e-6, group, *p[3:], M, K, None)

    for o, i, where in hits(sizes, [3, 4, 5, 6]):
        if o == 3 and i < 2 and where.value == at(i).value:
            continue  # in place
        p = [at(j) for j in range(7)]
        p[o] = where
        assert call(p) == 2, (o, i, hex(where.value))
    for byte in (1, 2, 3):
        assert call([at(j) for j in range(6)] + [at(6, byte)]) == 3


@pytest.mark.parametrize("group", [0, 128, "fp8"])
def test_activation(lib, group):
    T, K = 6, 384
    sizes = [T * K * 4, K * 4, T * K, T * 4 * (K // 128 if group else 1)]
    for o, i, where in hits(sizes, [2, 3]):
        p = [at(j) for j in range(4)]
        p[o] = where
        if group == "fp8":
            rc = lib.sq_silu_mul_quant_fp8(*p, T, K, None)
        else:
            rc = lib.sq_silu_mul_quant(*p[:2], group, *p[2:], T, K, None)
        assert rc == 2, (o, i, hex(where.value))
