// rowquant.cuh -- HBM-bound kernels that fuse a row operation with 8-bit
// quantisation: residual addition + RMSNorm, and the gated activation
// silu(gate) * up.  Codes are INT8 with one scale per row or per 128 columns, or
// E4M3 with one scale per 128 columns (as quant.cuh, with the divisions by amax,
// by 127 or 448 and by K formed as products with one rounded reciprocal).
//
// One pass over HBM: TPR threads own a row and hold it in registers (NV vectors
// of 8 columns per thread) from the loads to the codes, so nothing is read
// twice and no shared memory but the reduction slots is touched.  The grid is
// what fits on the device (twice that for the activation); a block walks its rows with
// the next one's loads in flight.  Bound by HBM: 7 bytes per element (norm) and
// 5 (activation).  Measured:
//   norm, INT8 per token, 8192 x 5120: 47.9 us, 6130 GB/s; one row per block and no
//     prefetch 52.9 us; 512 threads per row 69 us.  8 x 5120: 2.9 us.
//   activation, E4M3, 32768 x 1024: 29.4 us, 5710 GB/s (64 threads x 2 vectors).  Without
//     the guard of an infinite gate 28.7 us, and against that: 32 x 4 31.0 us, 128 x 1
//     29.9 us; with __expf and __fdividef 31.1 us; one row per warp, none ahead, 47 us.
//     8192 x 17408 (512 x 5: one block holds an SM's registers, with small spills): E4M3
//     134 us, 5330 GB/s; INT8 per row 169 us, 4220 GB/s.
#pragma once
#include "quant.cuh"

namespace sq {

enum : int { RQ_ADD_NORM = 0, RQ_SILU = 1 };           // row operation
enum : int { RQ_I8_ROW = 0, RQ_I8_GROUP = 1, RQ_E4M3_GROUP = 2 };  // output format

struct RowQuantArgs {
  const __nv_bfloat16* a;   // h [M, K], or gate_up [M, 2 K]
  const __nv_bfloat16* b;   // residual [M, K] (may be b_out)
  __nv_bfloat16* b_out;     // residual' [M, K]
  const float* vec;         // gamma [K], or 1/s [K] (may be NULL)
  uint8_t* q;               // codes [M, K]
  float* scales;            // [M] or [M, K / 128]
  float* r_out;             // 1/rms [M] or NULL
  int64_t M;
  int K;
  float eps, inv_k;         // inv_k = f32(1 / K)
};

// silu(g) * u = g / (1 + exp(-g)) * u with the hardware's base-2 exponential and
// reciprocal (maximum relative errors 2^-22 and 2^-23, subnormals flushed to zero).
// log2(e) = H + L with H of 16 bits, so that g H is exact for a bf16 g, and
// 2^(-g log2 e) = 2^(-g H) (1 - g L ln 2 + ...), where the next term is below 2^-23 for g
// >= -87.  With the roundings of the product, the sum and the last two products (2^-24
// each) the result is within 2^-20 of its value for g >= -87; below, the value and its
// error are less than 2^-110 |u|.  L > 0 keeps an overflowed exponential infinite, and
// -g L ln 2 is held at -1, where the exponential has long been zero (g > 2^17), so that
// an infinite g does not make it 0 * inf: silu(inf) = inf.  (That guard costs 0.6 us of
// 29.4, E4M3 32768 x 1024; the arithmetic on pairs of values, with it, took the same.)
// (Without it: g log2(e) rounded to fp32 took the same time: 28.2 and 28.3 us, E4M3 32768 x 1024;
// a division in place of the reciprocal and expf 44 us.  Codes on the other side of a
// rounding border than in 64 bits, of 33.5 M: 25 to 33; with the division and expf 27 to 32.)
__device__ __forceinline__ float silu_mul(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(g, -1.44268798828125f)));
  e = __fmaf_rn(e, fmaxf(__fmul_rn(g, -4.888495152e-06f), -1.0f), e);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__fadd_rn(1.0f, e)));
  return __fmul_rn(__fmul_rn(g, r), u);
}

// The larger, NaN if either is (fmaxf would drop it): a row that holds NaN has scale NaN, so
// what is computed from it is NaN, not a plausible number.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// Codes per value: f32(QMAX * f32(1 / amax)), held finite (a largest magnitude
// below 2^-119 would make it infinite, and zeros NaN; 0 gives the largest finite
// factor too, which leaves zeros zero).  With |v| <=
// amax the product stays below QMAX (1 + 2^-24)^4: INT8 rounds it to at most 127,
// E4M3 saturates at 448.
__device__ __forceinline__ float code_factor(float amax, float qmax) {
  return fminf(__fmul_rn(qmax, __frcp_rn(amax)), 3.402823466e38f);
}

template <int TPR, int NV, int OP, int FMT>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
    row_quant_kernel(const RowQuantArgs p) {
  constexpr int BLOCK = TPR < 128 ? 128 : TPR;
  constexpr int RPB = BLOCK / TPR;     // rows per block
  constexpr int NW = TPR / 32;         // warps per row
  constexpr bool GROUP = FMT != RQ_I8_ROW;
  constexpr bool FP8 = FMT == RQ_E4M3_GROUP;
  constexpr float QMAX = FP8 ? 448.0f : 127.0f;
  // two slots, taken in turn: a row's sums are read while the next row's are written
  __shared__ double red_d[2][RPB][NW];
  __shared__ float red[2][RPB][NW];
  const int rib = threadIdx.x / TPR;
  const int t = threadIdx.x % TPR;
  const int lane = threadIdx.x & 31;
  const int wig = t >> 5;
  const int K = p.K;
  griddep_wait();  // nothing above touches global memory: the launch may overlap any kernel
  // The next kernel may start from here on, not before the wait: a product under
  // sq_set_overlap reads its weights as soon as it starts, and only the kernel directly
  // before it is known not to write them; the one before that has to be over.
  griddep_launch_dependents();

  // The next row is requested as soon as this one is unpacked, so its loads are in
  // flight during the arithmetic (in the registers that this row's just left).
  uint4 x[NV], y[NV];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + t) * 8;
      x[j] = y[j] = make_uint4(0, 0, 0, 0);
      if (row < p.M && c < K) {
        // plain loads: b_out may be one of the inputs, and a kernel that this launch
        // overlaps may have written any of them
        if constexpr (OP == RQ_ADD_NORM) {
          x[j] = *reinterpret_cast<const uint4*>(p.a + row * K + c);
          y[j] = *reinterpret_cast<const uint4*>(p.b + row * K + c);
        } else {
          x[j] = *reinterpret_cast<const uint4*>(p.a + row * 2 * K + c);
          y[j] = *reinterpret_cast<const uint4*>(p.a + row * 2 * K + K + c);
        }
      }
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * RPB;
  int64_t row = static_cast<int64_t>(blockIdx.x) * RPB + rib;
  load(row);
  int slot = 0;
  for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * RPB; row0 < p.M; row0 += step, row += step, slot ^= 1) {
    const bool active = row < p.M;
    float v[NV][8];
    // ---- the row, in fp32 registers
    if constexpr (OP == RQ_ADD_NORM) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + t) * 8;
        float f[8];
        bf16x8_to_f32(x[j], v[j]);
        bf16x8_to_f32(y[j], f);
        uint32_t s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)  // the sum is kept in bf16: what is stored is what is normalised
          s[i] = pack_bf16x2(__fadd_rn(v[j][2 * i], f[2 * i]), __fadd_rn(v[j][2 * i + 1], f[2 * i + 1]));
        const uint4 sum = make_uint4(s[0], s[1], s[2], s[3]);
        if (active && c < K) *reinterpret_cast<uint4*>(p.b_out + row * K + c) = sum;
        bf16x8_to_f32(sum, v[j]);
      }
      load(row + step);
      double ss = 0.0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double d = static_cast<double>(v[j][i]);
          ss = __fma_rn(d, d, ss);
        }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      if constexpr (NW > 1) {
        if (lane == 0) red_d[slot][rib][wig] = ss;
        __syncthreads();
        ss = 0.0;
#pragma unroll
        for (int w = 0; w < NW; ++w) ss += red_d[slot][rib][w];
      }
      const float ms = __fmul_rn(__double2float_rn(ss), p.inv_k);
      const float rn = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(ms, p.eps)));
      if (active && p.r_out && t == 0) p.r_out[row] = rn;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + t) * 8;
        if (c < K) {
          const float4 g0 = *reinterpret_cast<const float4*>(p.vec + c);
          const float4 g1 = reinterpret_cast<const float4*>(p.vec + c)[1];
          const float gm[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] = __fmul_rn(__fmul_rn(v[j][i], rn), gm[i]);
        }
      }
    } else {
      float u[NV][8];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        bf16x8_to_f32(x[j], v[j]);
        bf16x8_to_f32(y[j], u[j]);
      }
      load(row + step);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * TPR + t) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] = silu_mul(v[j][i], u[j][i]);
        if (p.vec && c < K) {
          const float4 g0 = *reinterpret_cast<const float4*>(p.vec + c);
          const float4 g1 = reinterpret_cast<const float4*>(p.vec + c)[1];
          const float gm[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] = __fmul_rn(v[j][i], gm[i]);
        }
      }
    }
    // ---- largest magnitude: of the row, or of each 128 columns (16 adjacent lanes)
    float amax = 0.0f, gmax[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float m = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(v[j][i]));
      if constexpr (GROUP) {
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
      }
      gmax[j] = m;
      amax = max_nan(amax, m);
    }
    if constexpr (!GROUP) {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, off));
      if constexpr (NW > 1) {
        if (lane == 0) red[slot][rib][wig] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NW; ++w) amax = max_nan(amax, red[slot][rib][w]);
      }
      if (active && t == 0) p.scales[row] = __fmul_rn(amax, 1.0f / QMAX);
    }
    // ---- codes
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TPR + t) * 8;
      const float am = GROUP ? gmax[j] : amax;
      const float mult = code_factor(am, QMAX);
      if (!active || c >= K) continue;
      if (GROUP && (t & 15) == 0) p.scales[row * (K >> 7) + (c >> 7)] = __fmul_rn(am, 1.0f / QMAX);
      uint32_t pk[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float* f = &v[j][4 * i];
        if constexpr (FP8) {
          const uint32_t lo = e4m3x2_bits(__fmul_rn(f[0], mult), __fmul_rn(f[1], mult));
          const uint32_t hi = e4m3x2_bits(__fmul_rn(f[2], mult), __fmul_rn(f[3], mult));
          pk[i] = am > 0.0f ? (lo | (hi << 16)) : 0u;  // an all-zero group: zero codes, not -0
        } else {
          pk[i] = pack_code_bytes(quant_byte_bits(f[0], mult), quant_byte_bits(f[1], mult),
                                  quant_byte_bits(f[2], mult), quant_byte_bits(f[3], mult));
        }
      }
      *reinterpret_cast<uint2*>(p.q + row * K + c) = make_uint2(pk[0], pk[1]);
    }
  }
}

}  // namespace sq
