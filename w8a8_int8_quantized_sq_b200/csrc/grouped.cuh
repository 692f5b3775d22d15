// grouped.cuh -- matrix products grouped by expert with ragged sizes, on CTA
// pairs (tcgen05 cta_group::2): W8A8 with per-token x per-channel scales, and
// FP8 (E4M3) with 1x128 activation and [128, 128] weight scales.
//
// Rows are in the experts' order: expert e owns rows offsets[e] ..
// offsets[e+1] - 1 and multiplies them by its own weights q_w[e] (N x K).  Row t
// reads token rows[t] (or token t when rows is NULL).  The offsets live on the
// device, so every CTA works the tile list out for itself: expert e has
// ceil(r_e / 256) token tiles of nearly equal size times ceil(N / 256) channel
// tiles; clusters take tiles round-robin, token tiles of one weight tile
// next to each other so that the weights come from L2 after the first.
//
// Operand roles: the weights fill the 256 MMA rows (128 channels in each CTA's
// tensor memory) and the tokens are the MMA's N, which is an operand of the
// instruction descriptor and so follows each tile's row count in steps of 32.
// A group of 20 rows therefore costs an N = 32 product and loads 32 token rows,
// not a full tile; a 256-row tile has the shared-memory traffic of a dense
// 256 x 256 pair tile.
//
// INT8: acc int32 over the whole of K, y = bf16((f32(acc) * s_tok) * s_ch).
// FP8: every 128-wide K block is a fresh accumulator and is promoted into fp32
// registers, acc = fmaf(P_kb, f32(s_a * s_w), acc).  A CTA's 128 channels are
// one weight block, so s_w is uniform and the products s_a * s_w of a K block are
// one vector over the tile's tokens: a scale warp writes it to a shared-memory
// ring one K block ahead.  Its arrival counts on the barrier on which the K
// block's MMAs report, so the epilogue waits once for both.
//
// Roles per CTA: warp 0 TMA producer, warp 1 tensor-memory allocation (pair)
// and, in the leader CTA, the MMA issuer, warp 2 scales (FP8 only), the others
// epilogue.  Token rows are fetched by tile loads when rows is NULL and by
// four-row gather loads otherwise.  No load uses multicast.
#pragma once
#include "gemm3.cuh"

namespace sq {

constexpr int kMaxExperts = 1024;

struct GroupedArgs {
  const int32_t* offsets;  // [E + 1]
  const int32_t* rows;     // [T] or NULL
  const float* s_a;        // INT8: [M]; FP8: [M, kb_total]
  const float* s_w;        // INT8: [E, N]; FP8: [E, N / 128, kb_total]
  __nv_bfloat16* out;      // [T, N]
  int T, M, E, N;
  int kb_total;            // K / 128
  int tiles_n;             // ceil(N / 256)
};

template <bool F8_>
struct GroupedCfg {
  static constexpr bool F8 = F8_;
  static constexpr int BT = 256;                 // most tokens per tile
  static constexpr int STAGES = F8 ? 5 : 6;
  static constexpr int A_BYTES = 128 * 128;      // weights staged by each CTA per K block
  static constexpr int B_BYTES = BT / 2 * 128;   // tokens staged by each CTA per K block
  static constexpr int NACC = 2;
  static constexpr int TMEM_COLS = 512;
  static constexpr int NE = F8 ? 16 : 8;         // epilogue warps
  static constexpr int EPI0 = F8 ? 3 : 2;        // first epilogue warp
  static constexpr int THREADS = (EPI0 + NE) * 32;
  static constexpr int SRING = 8;                // FP8: scale vectors in the ring
  static constexpr int OFF_B = STAGES * A_BYTES;
  static constexpr int OFF_SC = OFF_B + STAGES * B_BYTES;
  static constexpr int OFF_LO = OFF_SC + (F8 ? SRING * BT * 4 : 0);
  static constexpr int OFF_CUM = OFF_LO + (kMaxExperts + 1) * 4;
  static constexpr int OFF_BAR = (OFF_CUM + (kMaxExperts + 1) * 4 + 7) & ~7;
  static constexpr int NUM_BARS = 2 * STAGES + 2 * NACC + 1;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int smem_bytes() { return 1024 + OFF_MISC + 16; }
  static_assert(1024 + OFF_MISC + 16 <= 232448, "shared memory");
};

// 2-D four-row gather load (rows r.x .. r.w of the tensor, 128 bytes each at
// innermost coordinate x) into this CTA's shared memory; bytes counted on the
// pair leader's barrier.  A row outside the tensor reads as zero.
__device__ __forceinline__ void tma_gather4_pair(void* dst, const CUtensorMap* m, int32_t x, int4 r,
                                                 uint32_t bar_cluster) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      ".cta_group::2 [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(r.x), "r"(r.y), "r"(r.z), "r"(r.w),
      "r"(bar_cluster)
      : "memory");
}

// A tile of the list: expert, channel tile, first row and row count.
struct GroupedTile {
  int e, ct, row0, nrows;
};

// Walks this cluster's tiles in order; cum[e] counts the token tiles of the
// experts before e.
struct GroupedWalk {
  const int* lo;
  const int* cum;
  int tiles_n, e;
  __device__ __forceinline__ GroupedWalk(const int* lo_, const int* cum_, int tiles_n_)
      : lo(lo_), cum(cum_), tiles_n(tiles_n_), e(0) {}
  __device__ __forceinline__ GroupedTile at(int t) {
    while (t >= cum[e + 1] * tiles_n) ++e;
    const int nt = cum[e + 1] - cum[e];
    const int i = t - cum[e] * tiles_n;
    const int r = lo[e + 1] - lo[e];
    const int w = ((r + nt - 1) / nt + 31) & ~31;  // rows per token tile, at most BT
    GroupedTile g;
    g.e = e;
    g.ct = i / nt;
    const int tt = i - g.ct * nt;
    g.row0 = lo[e] + tt * w;
    g.nrows = min(w, r - tt * w);
    return g;
  }
};

// Two tokens' values of this lane's channel -> 32-bit stores of two channels:
// even lanes store token a (channels l, l + 1), odd lanes token b (l - 1, l).
__device__ __forceinline__ void grouped_store2(__nv_bfloat16* oa, __nv_bfloat16* ob, float a,
                                               float b, int lane, bool ok_a, bool ok_b) {
  const bool odd = lane & 1;
  const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
  const uint32_t v = odd ? pack_bf16x2(got, b) : pack_bf16x2(a, got);
  if (odd ? ok_b : ok_a) *reinterpret_cast<uint32_t*>(odd ? ob - 1 : oa) = v;
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmW,    // weights [E N, K], 128-row boxes
                   const __grid_constant__ CUtensorMap tmX,    // tokens [M, K]: 16-row boxes, or
                                                               // one-row boxes for the gather
                   const __grid_constant__ CUtensorMap tmX64,  // tokens, 64-row boxes
                   const GroupedArgs g) {
  constexpr int STAGES = Cfg::STAGES, NACC = Cfg::NACC, NE = Cfg::NE, BT = Cfg::BT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* smA = smem;
  uint8_t* smB = smem + Cfg::OFF_B;
  float* ring = reinterpret_cast<float*>(smem + Cfg::OFF_SC);
  int* lo = reinterpret_cast<int*>(smem + Cfg::OFF_LO);
  int* cum = reinterpret_cast<int*>(smem + Cfg::OFF_CUM);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* full = bars;                 // leader: pair's tiles of a stage have landed
  uint64_t* empty = bars + STAGES;       // both: the pair's MMAs are done with a stage
  uint64_t* tfull = bars + 2 * STAGES;   // both: an accumulator (FP8: and its scales) is complete
  uint64_t* tempty = tfull + NACC;       // leader: both epilogues released an accumulator
  uint64_t* drain = tempty + NACC;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int cluster = blockIdx.x >> 1;
  const int nclusters = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int a = 0; a < NACC; ++a) {
      mbar_init(tfull + a, Cfg::F8 ? 2 : 1);
      mbar_init(tempty + a, 2 * NE);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, Cfg::TMEM_COLS);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  griddep_wait();  // nothing above touches global memory: the launch may overlap any kernel
  // offsets, held inside [0, T] and non-decreasing whatever the caller wrote
  for (int e = threadIdx.x; e <= g.E; e += Cfg::THREADS) lo[e] = min(max(__ldg(g.offsets + e), 0), g.T);
  __syncthreads();
  if (warp == 0) {
    int top = 0, tiles = 0;
    for (int b = 0; b <= g.E; b += 32) {
      const int e = b + lane;
      int v = e <= g.E ? lo[e] : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, off);
        if (lane >= off) v = max(v, o);
      }
      v = max(v, top);
      const int prev = __shfl_up_sync(0xffffffffu, v, 1);
      // token tiles of expert e - 1 end where expert e begins
      int n = lane == 0 ? (b == 0 ? 0 : v - top) : v - prev;
      n = e <= g.E ? (n + BT - 1) / BT : 0;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, n, off);
        if (lane >= off) n += o;
      }
      n += tiles;
      if (e <= g.E) {
        lo[e] = v;
        cum[e] = n;
      }
      top = __shfl_sync(0xffffffffu, v, 31);
      tiles = __shfl_sync(0xffffffffu, n, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers of both CTAs initialised, tensor memory allocated in both
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  const int num_tiles = cum[g.E] * g.tiles_n;
  const int kbt = g.kb_total;
  griddep_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    const uint32_t full_leader = mapa_shared(smem_u32(full), 0);
    const uint64_t pol = policy_evict_normal();
    GroupedWalk walk(lo, cum, g.tiles_n);
    uint32_t stage = 0, phase = 0;
    long long fills = 0;
    bool ok = true;
    for (int t = cluster; ok && t < num_tiles; t += nclusters) {
      const GroupedTile tile = walk.at(t);
      const int half = ((tile.nrows + 31) & ~31) >> 1;  // token rows staged by this CTA
      const int w_row = tile.e * g.N + tile.ct * 256 + static_cast<int>(rank) * 128;
      const int first = static_cast<int>(rank) * half;
      int4 r4 = make_int4(g.M, g.M, g.M, g.M);
      if (g.rows && lane * 4 < half) {
        // rows past the tile or outside the tokens are fetched as zeros
        auto token = [&](int i) {
          if (first + i >= tile.nrows) return g.M;
          const int r = __ldg(g.rows + tile.row0 + first + i);
          return static_cast<unsigned>(r) < static_cast<unsigned>(g.M) ? r : g.M;
        };
        r4 = make_int4(token(lane * 4), token(lane * 4 + 1), token(lane * 4 + 2), token(lane * 4 + 3));
      }
      for (int kb = 0; kb < kbt; ++kb) {
        if (!warp_wait_bounded(empty + stage, phase ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        uint8_t* dst = smB + stage * Cfg::B_BYTES;
        if (lane == 0) {
          if (leader) mbar_arrive_expect_tx(full + stage, 2 * (Cfg::A_BYTES + half * 128));
          tma_load_2d_pair(smA + stage * Cfg::A_BYTES, &tmW, kb * 128, w_row,
                           full_leader + stage * 8, pol);
          if (!g.rows) {
            int i = 0;
            for (; i + 64 <= half; i += 64)
              tma_load_2d_pair(dst + i * 128, &tmX64, kb * 128, tile.row0 + first + i,
                               full_leader + stage * 8, pol);
            for (; i < half; i += 16)
              tma_load_2d_pair(dst + i * 128, &tmX, kb * 128, tile.row0 + first + i,
                               full_leader + stage * 8, pol);
          }
        }
        if (g.rows && lane * 4 < half)
          tma_gather4_pair(dst + lane * 512, &tmX, kb * 128, r4, full_leader + stage * 8);
        __syncwarp();
        ++fills;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (leader && lane == 0) {
      // the pair's copies (both CTAs' bytes count here) have all landed
      for (int st = 0; st < STAGES; ++st) {
        const long long n = fills / STAGES + (st < fills % STAGES ? 1 : 0);
        if (n > 0) wait_drain(full + st, static_cast<uint32_t>((n - 1) & 1));
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------- MMA issuer (leader)
    if (leader) {
      GroupedWalk walk(lo, cum, g.tiles_n);
      uint32_t stage = 0, phase = 0, local = 0;
      bool ok = true;
      for (int t = cluster; ok && t < num_tiles; t += nclusters) {
        const GroupedTile tile = walk.at(t);
        const int n = (tile.nrows + 31) & ~31;
        const uint32_t idesc = Cfg::F8 ? idesc_e4m3_f32_m256(n) : idesc_i8_s32_m256(n);
        uint32_t d = 0;
        for (int kb = 0; kb < kbt; ++kb) {
          if (Cfg::F8 || kb == 0) {  // a free accumulator: per K block (FP8) or per tile
            const uint32_t a = local % NACC, u = local / NACC;
            ++local;
            if (!warp_wait_bounded(tempty + a, (u & 1u) ^ 1u, abort_flag)) { ok = false; break; }
            d = tmem + a * BT;
          }
          if (!warp_wait_bounded(full + stage, phase, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sa = smem_u32(smA + stage * Cfg::A_BYTES);
          const uint32_t sb = smem_u32(smB + stage * Cfg::B_BYTES);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t acc = (k > 0 || (!Cfg::F8 && kb > 0)) ? 1u : 0u;
              if constexpr (Cfg::F8)
                mma_f8_pair(d, smem_desc_sw128(sa + k * 32), smem_desc_sw128(sb + k * 32), idesc, acc);
              else
                mma_i8_pair(d, smem_desc_sw128(sa + k * 32), smem_desc_sw128(sb + k * 32), idesc, acc);
            }
            mma_commit_pair_both(empty + stage);
            if (Cfg::F8 || kb == kbt - 1) mma_commit_pair_both(tfull + (local - 1) % NACC);
          }
          __syncwarp();
          if (++stage == STAGES) { stage = 0; phase ^= 1u; }
        }
      }
      if (elect_one()) {
        mma_commit_pair(drain);
        wait_drain(drain, 0);
      }
    }
    __syncwarp();
  } else if (Cfg::F8 && warp == 2) {
    // ------------------------------------------------------------- scales
    // Vector kb of the ring slot kb % SRING: s_a[token, kb] * s_w[block, kb] for the
    // tile's tokens (0 for rows outside).  A slot is rewritten SRING K blocks
    // later; by then this warp has seen the accumulator of K block kb - 3
    // complete, whose buffer the epilogue released (after using its scales) for
    // K block kb - 5, so slots up to kb - 6 are free.
    GroupedWalk walk(lo, cum, g.tiles_n);
    uint32_t local = 0;
    bool ok = true;
    for (int t = cluster; ok && t < num_tiles; t += nclusters) {
      const GroupedTile tile = walk.at(t);
      const int nch = (tile.nrows + 31) >> 5;  // 32-token chunks
      const int ch0 = tile.ct * 256 + static_cast<int>(rank) * 128;
      const bool ch_ok = ch0 < g.N;
      const float* sw = g.s_w + (static_cast<size_t>(tile.e) * (g.N >> 7) + (ch_ok ? ch0 >> 7 : 0)) * kbt;
      const float* sa[BT / 32];
#pragma unroll
      for (int i = 0; i < BT / 32; ++i) {
        sa[i] = nullptr;
        const int c = i * 32 + lane;
        if (c < tile.nrows) {
          const int r = g.rows ? __ldg(g.rows + tile.row0 + c) : tile.row0 + c;
          if (static_cast<unsigned>(r) < static_cast<unsigned>(g.M))
            sa[i] = g.s_a + static_cast<size_t>(r) * kbt;
        }
      }
      float v[BT / 32], w = __ldg(sw);
#pragma unroll
      for (int i = 0; i < BT / 32; ++i) v[i] = i < nch && sa[i] ? __ldg(sa[i]) : 0.0f;
      for (int kb = 0; kb < kbt; ++kb, ++local) {
        float* slot = ring + (local % Cfg::SRING) * BT;
#pragma unroll
        for (int i = 0; i < BT / 32; ++i)
          if (i < nch) slot[i * 32 + lane] = __fmul_rn(v[i], w);
        if (kb + 1 < kbt) {
          w = __ldg(sw + kb + 1);
#pragma unroll
          for (int i = 0; i < BT / 32; ++i)
            if (i < nch) v[i] = sa[i] ? __ldg(sa[i] + kb + 1) : 0.0f;
        }
        const uint32_t a = local % NACC, u = local / NACC;
        // the previous use of this barrier must be over before its next arrival
        if (u > 0 && !warp_wait_bounded(tfull + a, (u - 1u) & 1u, abort_flag)) { ok = false; break; }
        __syncwarp();
        if (lane == 0) mbar_arrive(tfull + a);
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int ew = warp - Cfg::EPI0;
    const int q = warp & 3;                 // tensor-memory lane quadrant
    const int grp = ew >> 2;                // which columns of the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t tempty_leader = mapa_shared(smem_u32(tempty), 0);
    auto release = [&](uint32_t a) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(tempty + a);
        else mbar_arrive_remote(tempty_leader + a * 8);
      }
    };
    GroupedWalk walk(lo, cum, g.tiles_n);
    uint32_t local = 0;
    bool ok = true;
    for (int t = cluster; ok && t < num_tiles; t += nclusters) {
      const GroupedTile tile = walk.at(t);
      const int ch = tile.ct * 256 + static_cast<int>(rank) * 128 + q * 32 + lane;
      const bool ch_ok = ch < g.N;
      const int n = (tile.nrows + 31) & ~31;
      __nv_bfloat16* out = g.out + static_cast<size_t>(tile.row0) * g.N + ch;
      if constexpr (!Cfg::F8) {
        const float s_ch = ch_ok ? __ldg(g.s_w + static_cast<size_t>(tile.e) * g.N + ch) : 0.0f;
        const uint32_t a = local % NACC, u = local / NACC;
        ++local;
        if (!warp_wait_bounded(tfull + a, u & 1u, abort_flag)) { ok = false; break; }
        tc_fence_after();
#pragma unroll 1
        for (int c = grp * 32; c < n; c += (NE / 4) * 32) {
          // lane j holds the scale of column c + j (0: no such token)
          float st = 0.0f;
          if (c + lane < tile.nrows) {
            const int r = g.rows ? __ldg(g.rows + tile.row0 + c + lane) : tile.row0 + c + lane;
            if (static_cast<unsigned>(r) < static_cast<unsigned>(g.M)) st = __ldg(g.s_a + r);
          }
          uint32_t v[32];
          tmem_ld32(lane_base + a * BT + c, v);
          __nv_bfloat16* o = out + static_cast<size_t>(c) * g.N;
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float s0 = __shfl_sync(0xffffffffu, st, j), s1 = __shfl_sync(0xffffffffu, st, j + 1);
            const float y0 = __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(v[j])), s0), s_ch);
            const float y1 = __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(v[j + 1])), s1), s_ch);
            grouped_store2(o, o + g.N, y0, y1, lane, ch_ok && c + j < tile.nrows,
                           ch_ok && c + j + 1 < tile.nrows);
            o += 2 * static_cast<size_t>(g.N);
          }
        }
        release(a);
      } else {
        // this warp's columns: a quarter of the tile's, in steps of 16
        const int wcol = ((n >> 2) + 15) & ~15;
        const int col0 = grp * wcol;
        const int ncol = max(0, min(wcol, n - col0));
        float acc[64];
#pragma unroll
        for (int j = 0; j < 64; ++j) acc[j] = 0.0f;
        for (int kb = 0; kb < kbt; ++kb, ++local) {
          const uint32_t a = local % NACC, u = local / NACC;
          if (!warp_wait_bounded(tfull + a, u & 1u, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const float4* sc = reinterpret_cast<const float4*>(ring + (local % Cfg::SRING) * BT + col0);
#pragma unroll
          for (int c = 0; c < 64; c += 16) {
            if (c < ncol) {
              uint32_t v[16];
              tmem_ld16(lane_base + a * BT + col0 + c, v);
              if (c + 16 >= ncol) release(a);
#pragma unroll
              for (int j = 0; j < 16; j += 4) {
                const float4 s = sc[(c + j) >> 2];
                acc[c + j] = __fmaf_rn(__uint_as_float(v[j]), s.x, acc[c + j]);
                acc[c + j + 1] = __fmaf_rn(__uint_as_float(v[j + 1]), s.y, acc[c + j + 1]);
                acc[c + j + 2] = __fmaf_rn(__uint_as_float(v[j + 2]), s.z, acc[c + j + 2]);
                acc[c + j + 3] = __fmaf_rn(__uint_as_float(v[j + 3]), s.w, acc[c + j + 3]);
              }
            }
          }
          if (ncol == 0) release(a);
        }
        if (!ok) break;
        __nv_bfloat16* o = out + static_cast<size_t>(col0) * g.N;
#pragma unroll
        for (int j = 0; j < 64; j += 2) {
          if (j < ncol)
            grouped_store2(o, o + g.N, acc[j], acc[j + 1], lane, ch_ok && col0 + j < tile.nrows,
                           ch_ok && col0 + j + 1 < tile.nrows);
          o += 2 * static_cast<size_t>(g.N);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs are done with the pair's tensor memory and barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, Cfg::TMEM_COLS);
  }
}

}  // namespace sq
