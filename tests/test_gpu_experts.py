"""Mixture-of-experts operators through the public binding, against plain 64-bit
(or exact integer) implementations: products grouped by expert (INT8 bit-exact,
FP8 within the fp32 accumulation bound), residual addition + RMSNorm with
8-bit output (codes and scales bit-exact given the kernel's 1/rms), the gated
activation with 8-bit output (within its stated error), and a run of them
together."""
from __future__ import annotations

import math
import os
import subprocess
import sys

import pytest
import torch

import oracle
import w8a8_int8_quantized_sq_b200 as sq
from tests.prep import bf16_ulp

pytestmark = pytest.mark.gpu

EPS = 1e-6


def gen(seed):
    return torch.Generator().manual_seed(seed)


def offsets_of(counts, first=0):
    return torch.tensor([first] + [first + sum(counts[: i + 1]) for i in range(len(counts))],
                        dtype=torch.int32)


def i8_case(counts, N, K, gather, seed):
    g = gen(seed)
    T = sum(counts)
    M = max(1, T // 3) if gather else T
    q_a = torch.randint(-127, 128, (M, K), generator=g, dtype=torch.int8)
    s_tok = torch.rand(M, generator=g) * 0.1 + 1e-3
    q_w = torch.randint(-127, 128, (len(counts), N, K), generator=g, dtype=torch.int8)
    s_ch = torch.rand(len(counts), N, generator=g) * 1e-3 + 1e-5
    rows = torch.randint(0, M, (T,), generator=g, dtype=torch.int32) if gather else None
    return q_a, s_tok, q_w, s_ch, offsets_of(counts), rows


def i8_reference(q_a, s_tok, q_w, s_ch, offsets, rows, out):
    """Exact int32 sums (fp64 products of integers below 2^53), then two fp32 roundings
    and one to bf16; rows outside the groups keep `out`, padding rows give 0."""
    M = q_a.shape[0]
    T = out.shape[0]
    ref = out.clone()
    idx = torch.arange(T) if rows is None else rows.long()
    for e in range(q_w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo >= hi:
            continue
        pick = idx[lo:hi]
        ok = (pick >= 0) & (pick < M)
        p = pick.clamp(0, M - 1)
        acc = (q_a[p].double() @ q_w[e].double().T).float()
        y = ((acc * s_tok[p][:, None]) * s_ch[e][None, :]).bfloat16()
        y[~ok] = 0
        ref[lo:hi] = y
    return ref


def cuda(*ts):
    return [t.cuda() if t is not None else None for t in ts]


def assert_bits(got, ref, what):
    g, r = got.cpu().view(torch.int16), ref.view(torch.int16)
    bad = (g != r) & ~((got.cpu() == 0) & (ref == 0))  # +0 and -0 are the same value
    assert not bad.any(), f"{what}: {int(bad.sum())} of {r.numel()} differ, first {bad.nonzero()[0].tolist()}"


COUNTS = [
    [1],
    [0, 5, 0],
    [31, 32, 33, 0, 1],
    [255, 256, 257],
    [0, 0, 300, 2, 513, 0],
    [7] * 40,
]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", [(16, 128), (272, 384), (512, 1024)])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: "-".join(map(str, c[:6])))
def test_grouped_i8_bit_exact(counts, N, K, gather):
    c = i8_case(counts, N, K, gather, 11 + N + len(counts))
    T = sum(counts)
    y = sq.w8a8_grouped_mm(*cuda(*c[:5]), rows=cuda(c[5])[0])
    assert y.shape == (T, N)
    assert_bits(y, i8_reference(*c, torch.zeros(T, N, dtype=torch.bfloat16)), "y")
    sq.check_device_error()


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", [(16, 512), (272, 1152), (1536, 2176), (5120, 640)])
@pytest.mark.parametrize("counts", [[1], [0, 0, 2], [3, 0, 29], [1] * 32])
def test_grouped_i8_few_rows(counts, N, K, gather):
    """Calls of at most 32 rows, whose tiles may share K among the pairs of a cluster."""
    c = i8_case(counts, N, K, gather, 12 + N + len(counts))
    y = sq.w8a8_grouped_mm(*cuda(*c[:5]), rows=cuda(c[5])[0])
    assert_bits(y, i8_reference(*c, torch.zeros(sum(counts), N, dtype=torch.bfloat16)), "y")
    sq.check_device_error()


def test_grouped_i8_many_tiles():
    """More tiles than CTA pairs, groups of several token tiles, a long K."""
    g = gen(5)
    counts = torch.randint(0, 700, (12,), generator=g).tolist()
    c = i8_case(counts, 1040, 2176, True, 6)
    y = sq.w8a8_grouped_mm(*cuda(*c[:5]), rows=cuda(c[5])[0])
    assert_bits(y, i8_reference(*c, torch.zeros(sum(counts), 1040, dtype=torch.bfloat16)), "y")


def test_grouped_i8_largest_sums():
    """All codes +-127 at K = 131072: sums at the edge of int32."""
    K, N = 131072, 32
    q_a = torch.full((3, K), 127, dtype=torch.int8)
    q_w = torch.full((2, N, K), -127, dtype=torch.int8)
    q_w[1] = 127
    s_tok, s_ch = torch.tensor([1e-4, 2e-4, 3e-4]), torch.full((2, N), 1e-3)
    off = offsets_of([2, 1])
    y = sq.w8a8_grouped_mm(*cuda(q_a, s_tok, q_w, s_ch, off))
    assert_bits(y, i8_reference(q_a, s_tok, q_w, s_ch, off, None,
                                torch.zeros(3, N, dtype=torch.bfloat16)), "y")


@pytest.mark.parametrize("kind", ["i8", "fp8"])
def test_grouped_rows_outside_the_groups_are_left(kind):
    c = i8_case([3, 0, 40], 128, 256, False, 21)
    q_a, s_tok, q_w, s_ch = c[:4]
    off = torch.tensor([2, 5, 5, 39], dtype=torch.int32)  # rows 0..1 and 39.. belong to nobody
    out = torch.full((43, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    if kind == "i8":
        y = sq.w8a8_grouped_mm(*cuda(q_a, s_tok, q_w, s_ch, off), out=out)
        ref = i8_reference(q_a, s_tok, q_w, s_ch, off, None,
                           torch.full((43, 128), 7.0, dtype=torch.bfloat16))
        assert_bits(y, ref, "y")
    else:
        f = fp8_case([3, 0, 40], 128, 256, False, 22)
        y = sq.fp8_block_grouped_mm(*cuda(*f[:4], off), out=out)
    assert y.data_ptr() == out.data_ptr()
    assert (out[:2] == 7).all() and (out[39:] == 7).all()
    assert not (out[2:39] == 7).all()


def test_grouped_i8_offsets_out_of_range_are_held():
    """Offsets that decrease, are negative or pass T are held to the range and to the
    largest before them."""
    c = i8_case([20, 20, 20, 20], 64, 128, False, 31)
    q_a, s_tok, q_w, s_ch = c[:4]
    wild = torch.tensor([-5, 30, 10, 60, 1 << 30], dtype=torch.int32)
    held = torch.tensor([0, 30, 30, 60, 80], dtype=torch.int32)
    y = sq.w8a8_grouped_mm(*cuda(q_a, s_tok, q_w, s_ch, wild))
    ref = i8_reference(q_a, s_tok, q_w, s_ch, held, None, torch.zeros(80, 64, dtype=torch.bfloat16))
    assert_bits(y, ref, "y")
    nothing = torch.zeros(5, dtype=torch.int32)
    out = torch.full((80, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    sq.w8a8_grouped_mm(*cuda(q_a, s_tok, q_w, s_ch, nothing), out=out)
    assert (out == 3).all()


@pytest.mark.parametrize("kind", ["i8", "fp8"])
def test_grouped_padding_rows_give_zero(kind):
    rows = torch.tensor([-1, 0, 5, 4, 1 << 30, 4, 4, -(1 << 31), 2, 6, 5], dtype=torch.int32)
    off = torch.tensor([0, 3, 11], dtype=torch.int32)
    pad = (rows < 0) | (rows >= 5)
    if kind == "i8":
        c = i8_case([5, 0], 128, 256, False, 41)
        y = sq.w8a8_grouped_mm(*cuda(*c[:4], off), rows=rows.cuda())
        assert_bits(y, i8_reference(*c[:4], off, rows, torch.zeros(11, 128, dtype=torch.bfloat16)), "y")
    else:
        c = fp8_case([5, 0], 128, 256, False, 42)
        c[0][0, :3] = 0x7F  # NaN codes in token 0 stay in the rows that read it
        y = sq.fp8_block_grouped_mm(*cuda(*c[:4], off), rows=rows.cuda())
        assert torch.isnan(y.cpu()[1]).all() and torch.isfinite(y.cpu()[2:]).all()
    assert (y.cpu()[pad] == 0).all()
    assert not (y.cpu()[~pad] == 0).any()


@pytest.mark.parametrize("T", [20, 90])
@pytest.mark.parametrize("kind", ["i8", "fp8"])
def test_grouped_padding_rows_give_zero_beside_nonfinite_weights(kind, T):
    """A padding row is zero even where its expert's scales are infinite or NaN (FP8: and its
    codes NaN); a token that no row reads and an expert without rows reach nothing."""
    g = gen(43)
    rows = torch.randint(0, 8, (T,), generator=g, dtype=torch.int32)
    rows[1::3] = 9
    rows[2::5] = -1
    off = torch.tensor([0, T // 2, T // 2, T], dtype=torch.int32)
    pad = (rows < 0) | (rows >= 8)
    make = i8_case if kind == "i8" else fp8_case
    mm = sq.w8a8_grouped_mm if kind == "i8" else sq.fp8_block_grouped_mm
    q_a, s_a, q_w, s_w, _, _ = make([8, 0, 0], 256, 512, False, 44)
    # token 5 unread, expert 1 without rows
    rows[rows == 5] = 4
    want = mm(*cuda(q_a, s_a, q_w, s_w, off), rows=rows.cuda()).cpu()
    s_a[5], s_w[1] = float("nan"), float("inf")
    if kind == "fp8":
        q_a[5], q_w[1] = 0x7F, 0xFF
    assert torch.equal(mm(*cuda(q_a, s_a, q_w, s_w, off), rows=rows.cuda()).cpu(), want)
    # expert 2: every scale infinite, or every code NaN
    s_w[2] = float("inf")
    y = mm(*cuda(q_a, s_a, q_w, s_w, off), rows=rows.cuda()).cpu()
    assert torch.equal(y[:T // 2], want[:T // 2])
    assert (y[pad] == 0).all() and not torch.isfinite(y[T // 2:][~pad[T // 2:]]).any()
    if kind == "fp8":
        s_w[2], q_w[2] = 1.0, 0x7F
        y = mm(*cuda(q_a, s_a, q_w, s_w, off), rows=rows.cuda()).cpu()
        assert (y[pad] == 0).all() and torch.isnan(y[T // 2:][~pad[T // 2:]]).all()


# ------------------------------------------------------------------------ FP8

def fp8_case(counts, N, K, gather, seed):
    g = gen(seed)
    E, T = len(counts), sum(counts)
    M = max(1, T // 3) if gather else T
    x = torch.randn(M, K, generator=g)
    x[:, :3] *= 30
    q_a, s_a = oracle.quant_fp8_per_group(x.bfloat16())
    w = [oracle.quant_fp8_block((torch.randn(N, K, generator=g) * 0.02).bfloat16()) for _ in range(E)]
    q_w, s_w = torch.stack([a for a, _ in w]), torch.stack([b for _, b in w])
    rows = torch.randint(0, M, (T,), generator=g, dtype=torch.int32) if gather else None
    return q_a, s_a, q_w, s_w, offsets_of(counts), rows


def check_fp8(y, c, what):
    """The bound of the dense FP8 product: one bf16 ulp plus an fp32 accumulation of
    K exact products in steps of 32 (K / 32 + 8 roundings of at most 2^-22 of the sum
    of magnitudes)."""
    q_a, s_a, q_w, s_w, off, rows = c
    K = q_a.shape[1]
    idx = torch.arange(y.shape[0]) if rows is None else rows.long()
    y = y.cpu()
    for e in range(q_w.shape[0]):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        p = idx[lo:hi]
        ref, mag = oracle.fp8_block_mm(q_a[p].contiguous(), s_a[p].contiguous(), q_w[e].contiguous(),
                                       s_w[e].contiguous(), with_bound=True)
        diff = (y[lo:hi].double() - ref.double()).abs()
        tol = bf16_ulp(ref) + (K / 32 + 8) * 2.0 ** -22 * mag
        assert (diff <= tol).all(), (what, e, float((diff - tol).max()))


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("counts,N,K", [([1], 128, 128), ([0, 5, 33], 128, 384),
                                        ([70, 0, 300, 130], 384, 1408), ([9] * 20, 256, 256),
                                        ([200, 520], 640, 640), ([1], 256, 512), ([0, 3, 0, 29], 384, 1152),
                                        ([2], 1536, 2176), ([1] * 32, 640, 640), ([32], 128, 1664)])
def test_grouped_fp8(counts, N, K, gather):
    c = fp8_case(counts, N, K, gather, 51 + N + K)
    y = sq.fp8_block_grouped_mm(*cuda(*c[:5]), rows=cuda(c[5])[0])
    check_fp8(y, c, f"counts {counts} N {N} K {K}")
    sq.check_device_error()


@pytest.mark.parametrize("K", [768, 1152, 2048, 3200, 4224, 5120])
@pytest.mark.parametrize("counts", [[0, 2, 0], [1, 1], [2]])
def test_grouped_few_rows_over_uneven_parts(counts, K):
    """Between 9 and 20 tiles, whose K is shared by two, three or four pairs, evenly or not."""
    for N in (1152, 2304, 2432):
        c = i8_case(counts, N - 16, K, True, 61 + K)
        y = sq.w8a8_grouped_mm(*cuda(*c[:5]), rows=cuda(c[5])[0])
        assert_bits(y, i8_reference(*c, torch.zeros(sum(counts), N - 16, dtype=torch.bfloat16)), "y")
        c = fp8_case(counts, N, K, True, 62 + K)
        y = sq.fp8_block_grouped_mm(*cuda(*c[:5]), rows=cuda(c[5])[0])
        check_fp8(y, c, (N, K))
    sq.check_device_error()


@pytest.mark.parametrize("kind", ["i8", "fp8"])
def test_grouped_answers_do_not_depend_on_timing(kind):
    """The same call many times, alone and under load on another stream: the same bits."""
    c = (i8_case if kind == "i8" else fp8_case)([2, 0, 7], 640, 2176, True, 62)
    mm = sq.w8a8_grouped_mm if kind == "i8" else sq.fp8_block_grouped_mm
    args, rows = cuda(*c[:5]), cuda(c[5])[0]
    want = mm(*args, rows=rows)
    load = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(20):
            load @ load
    got = [mm(*args, rows=rows) for _ in range(50)]
    torch.cuda.synchronize()
    assert all(torch.equal(want, g) for g in got)


def test_grouped_fp8_equals_the_dense_product():
    """One expert that owns every row against the dense entry point (both promote each K
    block in ascending order; block sums may differ in the tensor core's order)."""
    c = fp8_case([130], 256, 1024, False, 61)
    y = sq.fp8_block_grouped_mm(*cuda(*c[:5])).cpu()
    dense = sq.fp8_block_mm(*cuda(c[0], c[1], c[2][0], c[3][0])).cpu()
    check_fp8(dense, c, "dense")
    assert ((y.double() - dense.double()).abs() <= 2 * bf16_ulp(dense)).float().mean() > 0.999


# --------------------------------------------------------------- residual norm

def norm_reference(h, res, gamma, r, fmt):
    """IEEE fp32 operations in the documented order, given the kernel's r."""
    kept = (h.float() + res.float()).bfloat16()
    v = (kept.float() * r[:, None]) * gamma
    M, K = v.shape
    top = 448.0 if fmt == "fp8" else 127.0
    b = v.view(M, 1, K) if fmt == "i8" else v.view(M, K // 128, 128)
    amax = b.abs().amax(2, keepdim=True)
    mult = torch.where(amax > 0, torch.tensor(top) * (torch.ones(()) / amax), torch.zeros(()))
    mult = mult.clamp(max=torch.finfo(torch.float32).max)
    code = b * mult
    q = code.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8) if fmt == "fp8" else \
        code.round().clamp(-127, 127).to(torch.int8)
    scale = (amax * (torch.ones(()) / top)).view(M, -1)
    return kept, q.reshape(M, K), scale.view(M) if fmt == "i8" else scale


def call_norm(h, res, gamma, fmt, **kw):
    if fmt == "fp8":
        return sq.add_rmsnorm_quant_fp8(h, res, gamma, EPS, **kw)
    return sq.add_rmsnorm_quant(h, res, gamma, EPS, group=128 if fmt == "i8_group" else 0, **kw)


def norm_case(M, K, seed):
    g = gen(seed)
    h = torch.randn(M, K, generator=g)
    h[:, 1] *= 30
    h[::5] *= 50
    res = torch.randn(M, K, generator=g) * 4
    gamma = torch.rand(K, generator=g) + 0.25
    return h.bfloat16(), res.bfloat16(), gamma


@pytest.mark.parametrize("fmt", ["i8", "i8_group", "fp8"])
@pytest.mark.parametrize("M,K", [(1, 128), (7, 256), (130, 384), (5, 640), (3, 1024), (9, 1152),
                                 (300, 2048), (33, 4096), (2, 4224), (64, 5120), (3, 6272),
                                 (2, 8320), (17, 12416), (4, 17408), (3, 24576)])
def test_add_rmsnorm_quant(M, K, fmt):
    h, res, gamma = norm_case(M, K, 71 + M + K)
    if M > 2:
        h[M // 2] = 0
        res[M // 2] = 0   # an all-zero row: r = 1/sqrt(eps), zero codes and scales
        res[1] = -h[1]    # a sum that cancels to zeros
    kept, q, sc, r = call_norm(*cuda(h, res, gamma), fmt)
    x = (h.float() + res.float()).bfloat16().double()
    r64 = 1.0 / torch.sqrt(x.square().mean(1) + EPS)
    # ss, 1 / K, their product, + eps (half each under the root), sqrt, 1 / .: six roundings,
    # four effective; 5 leaves room for their cross terms
    assert ((r.cpu().double() - r64).abs() <= 5 * 2.0 ** -24 * r64).all()
    k_ref, q_ref, s_ref = norm_reference(h, res, gamma, r.cpu(), fmt)
    assert torch.equal(kept.cpu().view(torch.int16), k_ref.view(torch.int16))
    assert torch.equal(q.cpu(), q_ref)
    assert torch.equal(sc.cpu(), s_ref)


def test_add_rmsnorm_quant_agrees_with_the_norm_of_the_sum():
    """sq_rmsnorm_quant on the stored residual divides where this operator multiplies by
    rounded reciprocals.  In units of 2^-24, relative, the two sides' roundings add up to:
    the mean of squares 2 + 1, + eps 1 + 1, halved by the root 2.5; the root 1 + 1 and the
    reciprocal 1 + 1: r differs by at most 6.5.  A value v takes two more products on each
    side: 10.5; its scale a division or a reciprocal and a product: 13.5; its code's factor amax's 10.5 and
    three more roundings, then the product on each side: 10.5 + 13.5 + 2 = 26 on |v * factor|
    <= 127, a move of at most 2e-4, so codes differ by one at most, and in less than
    2 * 2e-4 of the places."""
    h, res, gamma = cuda(*norm_case(513, 5120, 81))
    for group in (0, 128):
        kept, q, sc, r = sq.add_rmsnorm_quant(h, res, gamma, EPS, group=group)
        q2, sc2, r2 = sq.rmsnorm_quant(kept, gamma, EPS, group=group)
        for a, b, steps in ((r, r2, 6.5), (sc, sc2, 13.5)):
            assert ((a.double() - b.double()).abs() <= steps * 2.0 ** -24 * b.double()).all()
        d = (q.int() - q2.int()).abs()
        assert d.max() <= 1 and d.sum() < q.numel() * 4e-4


@pytest.mark.parametrize("fmt", ["i8", "i8_group", "fp8"])
@pytest.mark.parametrize("target", ["residual", "h"])
def test_add_rmsnorm_quant_in_place(fmt, target):
    h, res, gamma = cuda(*norm_case(200, 2048, 82))
    want = call_norm(h, res, gamma, fmt)
    buf = {"residual": res, "h": h}[target]
    got = call_norm(h, res, gamma, fmt, residual_out=buf)
    assert got[0].data_ptr() == buf.data_ptr()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8) if a.dtype == torch.uint8 else a, b)


@pytest.mark.parametrize("fmt", ["i8", "i8_group", "fp8"])
def test_add_rmsnorm_quant_nonfinite_rows_stay_alone(fmt):
    h, res, gamma = norm_case(12, 1152, 83)
    clean = [t.cpu() for t in call_norm(*cuda(h, res, gamma), fmt)]
    h[3, 7], res[8, 1100], h[9, 0] = float("inf"), float("nan"), -float("inf")
    got = [t.cpu() for t in call_norm(*cuda(h, res, gamma), fmt)]
    keep = [i for i in range(12) if i not in (3, 8, 9)]
    for a, b in zip(got, clean):
        assert torch.equal(a[keep], b[keep])


# --------------------------------------------------------------- gated activation

def call_silu(gu, inv, fmt):
    if fmt == "fp8":
        return sq.silu_mul_quant_fp8(gu, inv)
    return sq.silu_mul_quant(gu, inv, group=128 if fmt == "i8_group" else 0)


def check_silu(gu, inv, fmt, q, sc):
    T, K = gu.shape[0], gu.shape[1] // 2
    g, u = gu.double().chunk(2, 1)
    v = g * torch.sigmoid(g) * u
    slack = v.abs() * 2.0 ** -20 + u.abs() * 2.0 ** -110  # the stated error of the activation
    if inv is not None:
        v, slack = v * inv.double(), slack * inv.double()
    per = K if fmt == "i8" else 128
    top = 448.0 if fmt == "fp8" else 127.0
    amax = v.view(T, -1, per).abs().amax(2)
    sc = sc.cpu().double().view(T, -1)
    far = slack.view(T, -1, per).amax(2) / top
    # scale: the activation's error at the largest value, the fold and the division
    assert ((sc - amax / top).abs() <= far + 3 * 2.0 ** -24 * amax / top + 2.0 ** -149).all()
    if fmt == "fp8":
        val = q.cpu().view(torch.float8_e4m3fn).double().view(T, -1, per)
        assert torch.isfinite(val).all()
        # half a step of E4M3: 2^-4 of the value, 2^-10 below the normal range
        half = torch.maximum(val.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10).double())
    else:
        val = q.cpu().double().view(T, -1, per)
        half = torch.tensor(0.5).double()
    s = sc[:, :, None]
    err = (val * s - v.view(T, -1, per)).abs()
    # code of v * (top / amax) against v / scale: the factors' roundings, relative to the value
    tol = half * s + slack.view(T, -1, per) + 6 * 2.0 ** -24 * v.view(T, -1, per).abs() + 2.0 ** -140
    # a largest magnitude below 2^-119 takes the finite factor: codes may be smaller than the value asks
    tiny = (amax < 2.0 ** -118)[:, :, None]
    assert ((err <= tol) | (tiny & (err <= v.view(T, -1, per).abs() + tol))).all(), float((err - tol).max())


@pytest.mark.parametrize("fmt", ["i8", "i8_group", "fp8"])
@pytest.mark.parametrize("fold", [False, True])
@pytest.mark.parametrize("T,K", [(1, 128), (3, 256), (130, 768), (9, 1024), (5, 1408), (65, 2048),
                                 (4, 5120), (3, 9216), (2, 24576)])
def test_silu_mul_quant(T, K, fold, fmt):
    g = gen(91 + T + K)
    gu = torch.randn(T, 2 * K, generator=g) * 3
    gu[T // 2, :K] = torch.linspace(-120, 120, K)  # the whole range of the exponential
    if T > 2:
        gu[0] = 0
        gu[1, :K] = -85.0                          # a row of tiny values
        gu[2, K:] = 0
    gu = gu.bfloat16()
    inv = torch.rand(K, generator=g) + 0.25 if fold else None
    q, sc = call_silu(gu.cuda(), cuda(inv)[0], fmt)
    check_silu(gu, inv, fmt, q, sc)
    if T > 2:
        assert (q[0] == 0).all() and (sc[0] == 0).all() and (sc[2] == 0).all()


@pytest.mark.parametrize("fmt", ["i8", "i8_group", "fp8"])
def test_silu_mul_quant_nonfinite_rows_stay_alone(fmt):
    gu = (torch.randn(9, 768, generator=gen(95)) * 2).bfloat16()
    clean = [t.cpu() for t in call_silu(gu.cuda(), None, fmt)]
    gu[2, 3], gu[5, 500], gu[6, 0] = float("inf"), float("nan"), -float("inf")
    got = [t.cpu() for t in call_silu(gu.cuda(), None, fmt)]
    keep = [0, 1, 3, 4, 7, 8]
    for a, b in zip(got, clean):
        assert torch.equal(a[keep], b[keep])


# ------------------------------------------------------------------ a run of them

def layer_inputs(M, E, top, K, I, fmt, seed):
    g = gen(seed)
    h, res, gamma = norm_case(M, K, seed)
    ids = torch.rand(M, E, generator=g).topk(top, 1).indices
    order = torch.sort(ids.flatten(), stable=True).indices
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.bincount(ids.flatten(), minlength=E).cumsum(0)
    rows = (order // top).to(torch.int32)
    w = {}
    for name, n, k in (("up", 2 * I, K), ("down", K, I)):
        full = [(torch.randn(n, k, generator=g) / math.sqrt(k)).bfloat16() for _ in range(E)]
        pack = [oracle.quant_fp8_block(t) if fmt == "fp8" else oracle.quant_weight(t, None) for t in full]
        w[name] = (torch.stack([a for a, _ in pack]), torch.stack([b for _, b in pack]))
    weight = torch.rand(M, top, generator=g)
    return h, res, gamma, rows, off, w, order, weight


def run_layer(h, res, gamma, rows, off, up, s_up, down, s_down, fmt):
    if fmt == "fp8":
        kept, q, s, _ = sq.add_rmsnorm_quant_fp8(h, res, gamma, EPS)
        y = sq.fp8_block_grouped_mm(q, s, up, s_up, off, rows=rows)
        q2, s2 = sq.silu_mul_quant_fp8(y)
        return kept, sq.fp8_block_grouped_mm(q2, s2, down, s_down, off)
    kept, q, s, _ = sq.add_rmsnorm_quant(h, res, gamma, EPS)
    y = sq.w8a8_grouped_mm(q, s, up, s_up, off, rows=rows)
    q2, s2 = sq.silu_mul_quant(y)
    return kept, sq.w8a8_grouped_mm(q2, s2, down, s_down, off)


def layer_reference(h, res, gamma, rows, off, w, fmt):
    """The layer in 64 bits on the dequantised weights, with no quantised activations."""
    kept = (h.double() + res.double()).bfloat16().double()
    x = kept / torch.sqrt(kept.square().mean(1, keepdim=True) + EPS) * gamma.double()

    def weights(name, e):
        q, s = w[name][0][e], w[name][1][e].double()
        if fmt == "fp8":
            return q.view(torch.float8_e4m3fn).double() * s.repeat_interleave(128, 0).repeat_interleave(128, 1)
        return q.double() * s[:, None]

    I = w["down"][0].shape[2]
    out = torch.zeros(rows.numel(), h.shape[1], dtype=torch.float64)
    for e in range(off.numel() - 1):
        lo, hi = int(off[e]), int(off[e + 1])
        if lo == hi:
            continue
        y = x[rows[lo:hi].long()] @ weights("up", e).T
        a = y[:, :I] * torch.sigmoid(y[:, :I]) * y[:, I:]
        out[lo:hi] = a @ weights("down", e).T
    return out


@pytest.mark.parametrize("fmt", ["i8", "fp8"])
@pytest.mark.parametrize("M,E,top,K,I", [(1, 8, 2, 256, 128), (37, 16, 4, 512, 256)])
def test_layer_run(M, E, top, K, I, fmt):
    h, res, gamma, rows, off, w, order, weight = layer_inputs(M, E, top, K, I, fmt, 101 + M)
    args = cuda(h, res, gamma, rows, off, *w["up"], *w["down"])
    kept, y = run_layer(*args, fmt)
    ref = layer_reference(h, res, gamma, rows, off, w, fmt)
    # two quantisations of the activations.  A code is off by at most half a step: INT8
    # amax / 254 of its row's largest value, E4M3 2^-4 of the value; the errors of a sum
    # of K products are independent, so the relative 2-norm error is near that of one
    # code: below 2 * (amax / rms) / 254 (amax / rms < 16 for these rows of at most 512
    # values with one column 30 times larger) and 2 * 2^-4
    rel = float((y.cpu().double() - ref).norm() / ref.norm())
    assert rel < (2 * 2.0 ** -4 if fmt == "fp8" else 2 * 16 / 254), rel
    # back to the tokens' order, weighted: as a layer would finish
    back = torch.empty(M * top, K, dtype=torch.float64)
    back[order] = y.cpu().double()
    assert torch.isfinite((back.view(M, top, K) * weight.double()[:, :, None]).sum(1)).all()
    sq.check_device_error()


@pytest.mark.parametrize("fmt", ["i8", "fp8"])
def test_layer_run_in_a_graph_and_on_streams(fmt):
    """A captured run replays with new inputs in the same buffers, and two runs on two
    streams at once give what they give alone."""
    a = layer_inputs(24, 8, 3, 512, 256, fmt, 111)
    b = layer_inputs(24, 8, 3, 512, 256, fmt, 112)
    args_a = cuda(*a[:5], *a[5]["up"], *a[5]["down"])
    args_b = cuda(*b[:5], *b[5]["up"], *b[5]["down"])
    want_a, want_b = run_layer(*args_a, fmt), run_layer(*args_b, fmt)
    torch.cuda.synchronize()

    live = [t.clone() for t in args_a]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run_layer(*live, fmt)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run_layer(*live, fmt)
    for args, want in ((args_a, want_a), (args_b, want_b), (args_a, want_a)):
        for d, s in zip(live, args):
            d.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    res = []
    for _ in range(4):
        with torch.cuda.stream(s1):
            x = run_layer(*args_a, fmt)
        with torch.cuda.stream(s2):
            y = run_layer(*args_b, fmt)
        res.append((x, y))
    torch.cuda.synchronize()
    for x, y in res:
        assert torch.equal(x[1], want_a[1]) and torch.equal(y[1], want_b[1])
    sq.check_device_error()


@pytest.mark.parametrize("fmt", ["i8", "fp8"])
def test_layer_run_after_joins_and_copies(fmt):
    """Eager and captured: the first call after a join of two streams, after a copy and after
    a fill sees what they wrote (every launch may overlap its predecessor's tail)."""
    a = layer_inputs(24, 8, 3, 512, 256, fmt, 113)
    args = cuda(*a[:5], *a[5]["up"], *a[5]["down"])
    want = run_layer(*args, fmt)
    torch.cuda.synchronize()
    live = [torch.zeros_like(t) for t in args]
    side = torch.cuda.Stream()

    def run():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for i in (0, 3, 4, 5, 7):
                live[i].copy_(args[i])
        for i in (1, 2, 6, 8):
            live[i].copy_(args[i])
        main.wait_stream(side)
        kept, y = run_layer(*live, fmt)
        live[0].zero_()             # after the run has read it
        live[0].add_(args[0])
        again = run_layer(*live, fmt)
        return kept, y, *again

    for _ in range(3):
        for t in live:
            t.zero_()
        got = run()
        torch.cuda.synchronize()
        for g, w in zip(got, want * 2):
            assert torch.equal(g, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for t in live:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for g, w in zip(got, want * 2):
            assert torch.equal(g, w)


@pytest.mark.parametrize("fmt", ["i8", "fp8"])
def test_layer_run_captured_as_the_first_calls_of_a_process(fmt):
    """Nothing has to be called before a capture."""
    code = f"""
import torch
import tests.test_gpu_experts as t
a = t.layer_inputs(3, 8, 2, 512, 256, {fmt!r}, 116)
args = t.cuda(*a[:5], *a[5]["up"], *a[5]["down"])
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = t.run_layer(*args, {fmt!r})
graph.replay()
torch.cuda.synchronize()
want = t.run_layer(*args, {fmt!r})
assert all(torch.equal(x, y) for x, y in zip(got, want))
t.sq.check_device_error()
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": os.pathsep.join(p for p in sys.path if p)})
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_two_graphs_replayed_at_once():
    """Nothing is shared between captured calls: two graphs replay on two streams together."""
    runs = []
    for seed in (114, 115):
        a = layer_inputs(3, 8, 2, 1024, 512, "i8", seed)
        args = cuda(*a[:5], *a[5]["up"], *a[5]["down"])
        want = run_layer(*args, "i8")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run_layer(*args, "i8")
        runs.append((graph, got, want, args, torch.cuda.Stream()))
    for _ in range(20):
        for graph, _, _, _, stream in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, got, want, _, _ in runs:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_layer_run_in_inference_mode_and_from_threads():
    """Under inference mode, and from two host threads on streams of their own."""
    from concurrent.futures import ThreadPoolExecutor
    a = layer_inputs(5, 8, 2, 512, 256, "i8", 117)
    args = cuda(*a[:5], *a[5]["up"], *a[5]["down"])
    want = run_layer(*args, "i8")
    torch.cuda.synchronize()
    with torch.inference_mode():
        got = run_layer(*args, "i8")
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

    def many(_):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            outs = [run_layer(*args, "i8") for _ in range(20)]
        stream.synchronize()
        return all(torch.equal(x, w) for o in outs for x, w in zip(o, want))

    with ThreadPoolExecutor(2) as pool:
        assert all(pool.map(many, range(2)))


@pytest.mark.parametrize("M", [3, 2000])
@pytest.mark.parametrize("fmt", ["i8", "i8_group", "fp8"])
def test_outputs_of_one_call_are_apart(fmt, M):
    """Aligned, not overlapping (small calls' outputs share an allocation), each with its own
    values after the others have been written and freed."""
    h = torch.randn(M, 768, generator=gen(118)).bfloat16().cuda()
    gamma = torch.rand(768, device="cuda") + 0.25
    for call in (lambda: call_norm(h, h, gamma, fmt), lambda: call_silu(h, None, fmt)):
        want = [t.clone() for t in call()]
        outs = list(call())
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in outs)
        assert all(lo % 16 == 0 for lo, _ in spans)
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
        for i in range(len(outs)):
            for t in outs[:i]:
                t.zero_()
            assert torch.equal(outs[i], want[i])
        last = outs.pop()
        del outs, t
        torch.empty(1 << 20, dtype=torch.uint8, device="cuda").fill_(7)
        call()
        assert torch.equal(last, want[-1])


# ------------------------------------------------------------------ large and many

def test_grouped_i8_thousand_experts():
    g = gen(131)
    counts = torch.randint(0, 4, (1024,), generator=g).tolist()
    c = i8_case(counts, 16, 128, True, 132)
    y = sq.w8a8_grouped_mm(*cuda(*c[:5]), rows=cuda(c[5])[0])
    assert_bits(y, i8_reference(*c, torch.zeros(sum(counts), 16, dtype=torch.bfloat16)), "y")


@pytest.mark.parametrize("kind", ["i8", "fp8"])
def test_grouped_output_past_32_bits(kind):
    """More than 2^31 outputs: every row against the product of its token and expert."""
    T, N = 1_100_003, 2048
    c = (i8_case if kind == "i8" else fp8_case)([2, 2], N, 128, False, 133)
    mm = sq.w8a8_grouped_mm if kind == "i8" else sq.fp8_block_grouped_mm
    q_a, s_a, q_w, s_w = cuda(*c[:4])
    cut = 700_001
    rows = torch.randint(0, 4, (T,), generator=gen(134), dtype=torch.int32).cuda()
    y = mm(q_a, s_a, q_w, s_w, torch.tensor([0, cut, T], dtype=torch.int32, device="cuda"), rows=rows)
    each = [mm(q_a, s_a, q_w, s_w, torch.tensor(o, dtype=torch.int32, device="cuda"))
            for o in ([0, 4, 4], [0, 0, 4])]
    for e, (lo, hi) in enumerate(((0, cut), (cut, T))):
        for at in range(lo, hi, 1 << 18):
            end = min(hi, at + (1 << 18))
            assert torch.equal(y[at:end], each[e][rows[at:end].long()])


def test_grouped_weights_past_32_bits():
    """More than 2^31 bytes of weights: the last experts' rows."""
    E, N, K = 64, 8192, 4352
    g = torch.Generator(device="cuda").manual_seed(135)
    q_w = torch.randint(-127, 128, (E, N, K), generator=g, dtype=torch.int8, device="cuda")
    q_a = torch.randint(-127, 128, (40, K), generator=g, dtype=torch.int8, device="cuda")
    s_a, s_w = torch.full((40,), 0.01, device="cuda"), torch.full((E, N), 1e-3, device="cuda")
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[E - 1], off[E] = 7, 40
    y = sq.w8a8_grouped_mm(q_a, s_a, q_w, s_w, off.cuda()).cpu()
    ref = i8_reference(q_a.cpu(), s_a.cpu(), q_w[E - 2:].cpu(), s_w[E - 2:].cpu(),
                       torch.tensor([0, 7, 40]), None, torch.zeros(40, N, dtype=torch.bfloat16))
    assert_bits(y, ref, "y")


@pytest.mark.parametrize("kind", ["i8", "fp8"])
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_tokens_past_32_bits(kind, gather):
    """More than 2^31 bytes of tokens: rows at the end, by index and in order."""
    M, N, K = 530_001, 128, 4096
    c = (i8_case if kind == "i8" else fp8_case)([64, 0], N, K, False, 136)
    mm = sq.w8a8_grouped_mm if kind == "i8" else sq.fp8_block_grouped_mm
    q_a, s_a, q_w, s_w = cuda(*c[:4])
    big = torch.zeros(M, K, dtype=q_a.dtype, device="cuda")
    big_s = torch.zeros(M, *s_a.shape[1:], device="cuda")
    big[-64:], big_s[-64:] = q_a, s_a
    off = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
    want = mm(q_a, s_a, q_w, s_w, off)
    if gather:
        rows = torch.arange(M - 64, M, dtype=torch.int32, device="cuda")
        y = mm(big, big_s, q_w, s_w, off, rows=rows)
    else:
        y = mm(big, big_s, q_w, s_w, off + torch.tensor([M - 64], dtype=torch.int32, device="cuda"))[-64:]
    assert torch.equal(y, want)


@pytest.mark.parametrize("fmt", ["i8", "fp8"])
def test_row_operators_past_32_bits(fmt):
    """More than 2^31 elements: the last rows equal the same rows alone."""
    M, K = 420_001, 5120
    h = torch.randn(64, K, device="cuda").bfloat16().repeat(M // 64 + 1, 1)[:M].contiguous()
    gamma = torch.rand(K, device="cuda") + 0.25
    got = call_norm(h, h, gamma, fmt)
    want = call_norm(h[-70:].contiguous(), h[-70:].contiguous(), gamma, fmt)
    for a, b in zip(got, want):
        assert torch.equal(a[-70:], b)
    del got, want
    q, sc = call_silu(h, None, fmt)
    q2, sc2 = call_silu(h[-70:].contiguous(), None, fmt)
    assert torch.equal(q[-70:], q2) and torch.equal(sc[-70:], sc2)


def test_refusals_on_the_gpu():
    q_a, s_tok, q_w, s_ch, off, rows = cuda(*i8_case([3, 2], 64, 256, True, 121))
    with pytest.raises(ValueError):
        sq.w8a8_grouped_mm(q_a, s_tok, q_w, s_ch, off.long(), rows=rows)
    with pytest.raises(ValueError):
        sq.w8a8_grouped_mm(q_a, s_tok, q_w, s_ch, off[:-1], rows=rows)
    with pytest.raises(ValueError):
        sq.w8a8_grouped_mm(q_a, s_tok, q_w, s_ch, off.cpu(), rows=rows)
    with pytest.raises(ValueError):
        sq.w8a8_grouped_mm(q_a, s_tok, q_w.transpose(1, 2), s_ch, off, rows=rows)
    with pytest.raises(ValueError):
        sq.fp8_block_grouped_mm(q_a, s_tok, q_w, s_ch, off, rows=rows)
    with pytest.raises(sq.SqError) as e:
        sq.w8a8_grouped_mm(q_a[:, :192].contiguous(), s_tok, q_w[:, :, :192].contiguous(), s_ch, off, rows=rows)
    assert e.value.code == 2
    h = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    gamma = torch.ones(256, device="cuda")
    with pytest.raises(ValueError):
        sq.add_rmsnorm_quant(h, h.float(), gamma, EPS)
    with pytest.raises(sq.SqError) as e:
        sq.add_rmsnorm_quant(h, h, gamma, 0.0)
    assert e.value.code == 2
    with pytest.raises(sq.SqError) as e:
        sq.silu_mul_quant(h, group=64)
    assert e.value.code == 2
    # no rows: empty outputs
    assert sq.w8a8_grouped_mm(q_a[:0], s_tok[:0], q_w, s_ch, torch.zeros_like(off)).shape == (0, 64)
    assert sq.silu_mul_quant(h[:0])[0].shape == (0, 128)
