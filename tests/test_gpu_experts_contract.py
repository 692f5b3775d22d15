"""What a caller of the mixture-of-experts operators may rely on beside their values."""
from __future__ import annotations

import io
import threading
import time

import pytest
import torch

import w8a8_int8_quantized_sq_b200 as sq
from tests.test_gpu_experts import (EPS, assert_bits, call_norm, call_silu, check_fp8, check_silu, cuda,
                                    fp8_case, gen, i8_case, i8_reference, layer_inputs, norm_case, norm_reference,
                                    run_layer)

pytestmark = pytest.mark.gpu


def test_layer_run_repeats_itself():
    """The same FP8 run many times, alone and under load on another stream: the same bits."""
    a = layer_inputs(333, 8, 4, 1024, 512, "fp8", 208)
    args = cuda(*a[:5], *a[5]["up"], *a[5]["down"])
    want = run_layer(*args, "fp8")
    load = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(40):
            load @ load
    got = [run_layer(*args, "fp8") for _ in range(60)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for g in got for x, y in zip(g, want))


@pytest.mark.parametrize("fmt", ["i8", "fp8"])
@pytest.mark.parametrize("M,E,top,K,I", [(1, 8, 2, 256, 128), (50, 16, 4, 512, 384)])
def test_layer_run_step_by_step(M, E, top, K, I, fmt):
    """Each operator of a run against its definition on what the one before it gave."""
    h, res, gamma, rows, off, w, _, _ = layer_inputs(M, E, top, K, I, fmt, 209 + M)
    d = cuda(h, res, gamma, rows, off, *w["up"], *w["down"])
    mm = sq.w8a8_grouped_mm if fmt == "i8" else sq.fp8_block_grouped_mm
    kept, q, s, r = call_norm(*d[:3], fmt)
    k_ref, q_ref, s_ref = norm_reference(h, res, gamma, r.cpu(), fmt)
    assert torch.equal(kept.cpu(), k_ref) and torch.equal(q.cpu(), q_ref) and torch.equal(s.cpu(), s_ref)
    gu = mm(q, s, d[5], d[6], d[4], rows=d[3])
    q2, s2 = call_silu(gu, None, fmt)
    check_silu(gu.cpu(), None, fmt, q2, s2)
    y = mm(q2, s2, d[7], d[8], d[4])
    if fmt == "fp8":
        check_fp8(gu, (q.cpu(), s.cpu(), *w["up"], off, rows), "up")
        check_fp8(y, (q2.cpu(), s2.cpu(), *w["down"], off, None), "down")
    else:
        empty = torch.zeros(M * top, 2 * I, dtype=torch.bfloat16)
        assert_bits(gu, i8_reference(q.cpu(), s.cpu(), *w["up"], off, rows, empty), "up")
        empty = torch.zeros(M * top, K, dtype=torch.bfloat16)
        assert_bits(y, i8_reference(q2.cpu(), s2.cpu(), *w["down"], off, None, empty), "down")


@pytest.mark.parametrize("between", ["norm", "activation"])
def test_a_product_under_overlap_sees_weights_written_two_kernels_before(between):
    """sq_set_overlap lets a product read its weights before the kernel directly ahead of it is
    over, if that kernel does not write them.  A norm or an activation does not, and the
    kernel that it follows is over when the product starts."""
    N, K = 5120, 5120
    w = [(torch.randn(N, K, generator=gen(210 + i)) * 0.02).bfloat16().cuda() for i in range(2)]
    x = torch.randn(8, K, generator=gen(212)).bfloat16().cuda()
    small = torch.randn(8, 512, generator=gen(213)).bfloat16().cuda()
    gamma = torch.ones(512, device="cuda")
    q_a, s_tok = sq.quant_per_token(x)
    want = [sq.w8a8_scaled_mm(q_a, s_tok, *sq.quant_weight(v, None)) for v in w]
    assert not torch.equal(*want)
    q_w, s_ch = sq.quant_weight(w[1], None)
    torch.cuda.synchronize()
    write = sq.lib().sq_quant_weight
    sq.set_overlap(True)
    try:
        for i in range(40):
            rc = write(w[i % 2].data_ptr(), None, q_w.data_ptr(), s_ch.data_ptr(), N, K, 0,
                       torch.cuda.current_stream().cuda_stream)
            assert rc == 0
            if between == "norm":
                sq.add_rmsnorm_quant(small, small, gamma, EPS)
            else:
                sq.silu_mul_quant(small)
            y = sq.w8a8_scaled_mm(q_a, s_tok, q_w, s_ch)
            assert torch.equal(y, want[i % 2]), i
    finally:
        sq.set_overlap(False)
    sq.check_device_error()


def products(q, sc, fmt):
    """The codes and scales through a grouped product of one expert (weights of ones)."""
    T, K = q.shape
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    if fmt == "fp8":
        w = torch.full((1, 128, K), 0x38, dtype=torch.uint8, device="cuda")
        return sq.fp8_block_grouped_mm(q, sc, w, torch.ones(1, 1, K // 128, device="cuda"), off)
    w = torch.ones(1, 128, K, dtype=torch.int8, device="cuda")
    return sq.w8a8_grouped_mm(q, sc, w, torch.ones(1, 128, device="cuda"), off)


@pytest.mark.parametrize("fmt", ["i8", "i8_group", "fp8"])
@pytest.mark.parametrize("K", [256, 1152, 2048, 5120, 17408])
def test_norm_of_a_nonfinite_row_has_a_nonfinite_scale(K, fmt):
    h, res, gamma = norm_case(9, K, 201)
    clean = [t.cpu() for t in call_norm(*cuda(h, res, gamma), fmt)]
    h[1, 7], res[3, K - 9], h[5, 0], res[7, K // 2] = float("nan"), float("inf"), -float("inf"), float("nan")
    got = call_norm(*cuda(h, res, gamma), fmt)
    sc = got[2].cpu().view(9, -1)
    at = {1: slice(None), 7: slice(None)}           # a NaN is in every value of its row
    at |= {3: -1, 5: 0}                             # 1 / rms is 0: zeros beside the infinity's NaN
    for row, where in at.items():
        assert not torch.isfinite(sc[row][where]).any(), (row, sc[row])
    for a, b in zip(got, clean):
        assert torch.equal(a.cpu()[[0, 2, 4, 6, 8]], b[[0, 2, 4, 6, 8]])
    if fmt != "i8_group":
        bad = torch.isfinite(products(got[1], got[2], fmt).cpu()).sum(1)
        assert bad.tolist() == [128, 0] * 4 + [128]


@pytest.mark.parametrize("fmt", ["i8", "i8_group", "fp8"])
@pytest.mark.parametrize("K", [256, 768, 1408, 5120, 17408])
def test_activation_of_a_nonfinite_row_has_a_nonfinite_scale(K, fmt):
    gu = (torch.randn(9, 2 * K, generator=gen(202)) * 2).bfloat16()
    gu[:, [3, K - 100]] = 2.0
    gu[:, [K + 3, 2 * K - 100]] = 1.5
    clean = [t.cpu() for t in call_silu(gu.cuda(), None, fmt)]
    gu[1, 3], gu[2, K + 3] = float("nan"), float("nan")
    gu[3, 3], gu[4, K + 3] = float("inf"), -float("inf")   # silu(inf) = inf
    gu[5, K - 100], gu[6, 3] = -float("inf"), 3e38
    gu[6, K + 3] = 3e38                                    # a product past the range
    got = call_silu(gu.cuda(), None, fmt)
    sc, ref = got[1].cpu().view(9, -1), clean[1].view(9, -1)
    bad = {1: 0, 2: 0, 3: 0, 4: 0, 5: (K - 100) // 128 if fmt != "i8" else 0, 6: 0}
    for row, g in bad.items():
        assert not torch.isfinite(sc[row, g]), row
        keep = torch.ones(sc.shape[1], dtype=torch.bool)
        keep[g] = False
        assert torch.equal(sc[row][keep], ref[row][keep])
    for row in (1, 2):
        assert torch.isnan(sc[row, 0])
    for row in (3, 4, 6):
        assert sc[row, 0] == float("inf")
    for a, b in zip(got, clean):
        assert torch.equal(a.cpu()[[0, 7, 8]], b[[0, 7, 8]])
    if fmt != "i8_group":
        ok = torch.isfinite(products(got[0], got[1], fmt).cpu()).sum(1)
        assert ok.tolist() == [128] + [0] * 6 + [128] * 2


def test_activation_of_an_infinite_gate():
    """silu(inf) u = inf u, and the largest finite gates are not touched by what guards it."""
    K = 128
    gu = torch.ones(4, 2 * K)
    gu[0, :K], gu[1, :K], gu[2, :K], gu[3, :K] = float("inf"), 3e38, 2.0 ** 17, 2.0 ** 18
    gu = gu.bfloat16()
    q, sc = call_silu(gu.cuda(), None, "i8")
    assert sc[0] == float("inf")
    check_silu(gu[1:], None, "i8", q[1:], sc[1:])


@pytest.mark.parametrize("M", [1, 3, 2000])
@pytest.mark.parametrize("fmt", ["i8", "i8_group", "fp8"])
def test_outputs_of_one_call_have_storages_of_their_own(fmt, M):
    """Growing one output, freeing its memory or saving it touches no other."""
    h = torch.randn(M, 768, generator=gen(203)).bfloat16().cuda()
    gamma = torch.rand(768, device="cuda") + 0.25
    for call in (lambda: call_norm(h, h, gamma, fmt), lambda: call_silu(h, None, fmt),
                 lambda: call_norm(h, h, gamma, fmt, residual_out=h.clone())):
        want = [t.clone() for t in call()]
        for i in range(len(want)):
            outs = call()
            assert outs[i].untyped_storage().nbytes() == want[i].numel() * want[i].element_size()
            outs[i].resize_(outs[i].numel() + 70000).fill_(1)
            assert all(torch.equal(a, b) for j, (a, b) in enumerate(zip(outs, want)) if j != i)
            outs = call()
            outs[i].untyped_storage().resize_(0)
            assert all(torch.equal(a, b) for j, (a, b) in enumerate(zip(outs, want)) if j != i)
            file = io.BytesIO()
            torch.save(call()[i], file)
            assert file.tell() < want[i].numel() * want[i].element_size() + 4096


def test_a_full_launch_queue_stops_no_other_host_thread():
    """While a call waits for room in the launch queue (behind work that lasts a good second),
    another thread goes on.  A thread that holds the interpreter's lock would stop it."""
    x = torch.randn(4, 256, device="cuda").bfloat16()
    q_a, s_a, q_w, s_w, off, _ = cuda(*i8_case([4], 128, 128, False, 204))
    gamma = torch.ones(256, device="cuda")
    for call in (lambda: sq.silu_mul_quant(x), lambda: sq.add_rmsnorm_quant(x, x, gamma, EPS),
                 lambda: sq.w8a8_grouped_mm(q_a, s_a, q_w, s_w, off)):
        call()
        torch.cuda.synchronize()
        gaps, stop = [], threading.Event()

        def tick():
            last = time.perf_counter()
            while not stop.is_set():
                time.sleep(0.001)
                now = time.perf_counter()
                gaps.append(now - last)
                last = now

        t = threading.Thread(target=tick)
        t.start()
        torch.cuda._sleep(2_000_000_000)
        longest = 0.0
        for _ in range(3000):
            t0 = time.perf_counter()
            call()
            longest = max(longest, time.perf_counter() - t0)
            if longest > 0.2:
                break
        stop.set()
        t.join()
        torch.cuda.synchronize()
        assert longest > 0.2, "the launch queue never filled"
        assert max(gaps) < longest / 2, (max(gaps), longest)


def shifted(t, by=1):
    """The same values in a view that starts `by` elements into its storage."""
    flat = torch.empty(t.numel() + by, dtype=t.dtype, device=t.device)
    view = flat[by:].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("kind,K", [("i8", 256), ("fp8", 640), ("fp8", 512)])
def test_grouped_operands_that_start_anywhere(kind, K):
    """Scales, offsets and row indexes may be views at any element."""
    counts = [5, 0, 40, 7, 300]
    c = (i8_case if kind == "i8" else fp8_case)(counts, 256, K, True, 205)
    mm = sq.w8a8_grouped_mm if kind == "i8" else sq.fp8_block_grouped_mm
    q_a, s_a, q_w, s_w, off, rows = cuda(*c)
    want = mm(q_a, s_a, q_w, s_w, off, rows=rows)
    for by in (1, 2, 3):
        assert shifted(off, by).data_ptr() % 16
        assert torch.equal(mm(q_a, s_a, q_w, s_w, shifted(off, by), rows=rows), want)
        assert torch.equal(mm(q_a, s_a, q_w, s_w, off, rows=shifted(rows, by)), want)
        assert torch.equal(mm(q_a, shifted(s_a, by), q_w, s_w, off, rows=rows), want)
        assert torch.equal(mm(q_a, s_a, q_w, shifted(s_w, by), off, rows=rows), want)
        assert torch.equal(mm(q_a, shifted(s_a, by), q_w, shifted(s_w, by), shifted(off, by),
                              rows=shifted(rows, by)), want)
    sq.check_device_error()


@pytest.mark.parametrize("kind", ["i8", "fp8"])
def test_grouped_call_on_a_range_of_experts(kind):
    """offsets[e0 : e1 + 1] with the range's weights: its rows as in the whole call, the others
    left; eager and captured."""
    counts = [5, 0, 40, 7, 3, 20, 0, 9]
    c = (i8_case if kind == "i8" else fp8_case)(counts, 128, 384, True, 206)
    mm = sq.w8a8_grouped_mm if kind == "i8" else sq.fp8_block_grouped_mm
    q_a, s_a, q_w, s_w, off, rows = cuda(*c)
    want = mm(q_a, s_a, q_w, s_w, off, rows=rows)
    bounds = off.tolist()
    out = torch.empty_like(want)
    for e0 in range(len(counts)):
        for e1 in range(e0 + 1, len(counts) + 1):
            graph = torch.cuda.CUDAGraph()
            call = lambda: mm(q_a, s_a, q_w[e0:e1], s_w[e0:e1], off[e0:e1 + 1], rows=rows, out=out)
            with torch.cuda.graph(graph):
                call()
            for go in (call, graph.replay):
                out.fill_(7.0)
                go()
                lo, hi = bounds[e0], bounds[e1]
                assert torch.equal(out[lo:hi], want[lo:hi])
                assert (out[:lo] == 7).all() and (out[hi:] == 7).all()
    sq.check_device_error()


@pytest.mark.parametrize("fmt", ["i8", "i8_group", "fp8"])
def test_factors_that_start_anywhere(fmt):
    """gamma and inv_s may be views at any element; a gradient that they ask for is not recorded."""
    h, res, gamma = cuda(*norm_case(5, 768, 214))
    want, act = call_norm(h, res, gamma, fmt), call_silu(h, gamma[:384].clone(), fmt)
    for by in (1, 2, 3):
        got = call_norm(h, res, shifted(gamma, by).requires_grad_(), fmt)
        got += call_silu(h, shifted(gamma[:384], by).requires_grad_(), fmt)
        assert all(torch.equal(a, b) and not a.requires_grad for a, b in zip(got, (*want, *act)))
    sq.check_device_error()


@pytest.mark.parametrize("kind", ["i8", "fp8"])
def test_an_output_over_an_input_is_refused(kind):
    q_a, s_a, q_w, s_w, off, _ = cuda(*(i8_case if kind == "i8" else fp8_case)([40, 24], 128, 256, False, 215))
    mm = sq.w8a8_grouped_mm if kind == "i8" else sq.fp8_block_grouped_mm
    kept = q_a.clone()
    with pytest.raises(sq.SqError) as e:
        mm(q_a, s_a, q_w, s_w, off, out=q_a.view(torch.bfloat16))
    assert e.value.code == 2 and torch.equal(q_a, kept)
    h, gamma = torch.randn(64, 256, device="cuda").bfloat16(), torch.ones(256, device="cuda")
    big = torch.zeros(65, 256, dtype=torch.bfloat16, device="cuda")
    big[1:] = h
    with pytest.raises(sq.SqError) as e:
        sq.add_rmsnorm_quant(big[1:], h, gamma, EPS, residual_out=big[:-1])
    assert e.value.code == 2


def test_fp8_rows_of_a_call_of_32_are_those_of_a_call_of_31():
    """Calls of 31 and of 32 rows over 4 experts make the same tiles, so they share K among as
    many pairs, and their common rows have the same bits."""
    for counts in ([8, 8, 8, 8], [1, 29, 1, 1], [32]):
        c = fp8_case(counts, 2048, 5120, False, 207)
        q_a, s_a, q_w, s_w, off = cuda(*c[:5])
        y = sq.fp8_block_grouped_mm(q_a, s_a, q_w, s_w, off)
        less = sq.fp8_block_grouped_mm(q_a[:31].contiguous(), s_a[:31].contiguous(), q_w, s_w,
                                       off.clamp(max=31))
        assert torch.equal(y[:31], less), int((y[:31] != less).sum())
        check_fp8(y, c, counts)


@pytest.mark.parametrize("kind", ["i8", "fp8"])
def test_grouped_tiles_fill_their_bound(kind):
    """The most token tiles that T rows over E experts can make: one row in every expert but
    one, which has the rest.  Row counts around the tile heights."""
    for T in (31, 32, 33, 127, 128, 129, 255, 256, 257, 258, 512, 513):
        for E in (1, 2, 5):
            c = (i8_case if kind == "i8" else fp8_case)([1] * (E - 1) + [T - E + 1], 128, 256, False, 216)
            mm = sq.w8a8_grouped_mm if kind == "i8" else sq.fp8_block_grouped_mm
            y = mm(*cuda(*c[:5]))
            if kind == "i8":
                assert_bits(y, i8_reference(*c, torch.zeros(T, 128, dtype=torch.bfloat16)), (T, E))
            else:
                check_fp8(y, c, (T, E))
    sq.check_device_error()


def test_the_accumulator_wait_gives_up_too():
    """The self-test runs one wait of each kind to its limit (two limits' time in all), and the
    expert operators answer as before once the error word is cleared."""
    c = i8_case([3, 0, 29, 200], 256, 640, True, 217)
    args, rows = cuda(*c[:5]), cuda(c[5])[0]
    want = sq.w8a8_grouped_mm(*args, rows=rows)
    sq.check_device_error()
    limit = 100_000_000
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    assert sq.selftest_wait_timeout(limit) == 1
    end.record()
    end.synchronize()
    # a clock of at most 2 GHz; one limit alone would be over in 50 ms at 2 GHz
    took, clock = start.elapsed_time(end) * 1e-3, 2.0e9
    assert took >= 2 * limit / clock, took
    with pytest.raises(sq.SqError) as e:
        sq.check_device_error(reset=True)
    assert e.value.code == 6
    assert torch.equal(sq.w8a8_grouped_mm(*args, rows=rows), want)
    sq.check_device_error()
