// grouped.cuh -- matrix products grouped by expert with ragged sizes, on CTA
// pairs (tcgen05 cta_group::2): W8A8 with per-token x per-channel scales, and
// FP8 (E4M3) with 1x128 activation and [128, 128] weight scales.
//
// Rows are in the experts' order: expert e owns rows offsets[e] ..
// offsets[e+1] - 1 and multiplies them by its own weights q_w[e] (N x K).  Row t
// reads token rows[t] (or token t when rows is NULL).  The offsets live on the
// device, so every CTA works the tile list out for itself: expert e has
// ceil(r_e / BT) token tiles of nearly equal size times ceil(N / 256) channel
// tiles; clusters take tiles round-robin, token tiles of one weight tile
// next to each other so that the weights come from L2 after the first.  (Giving each
// cluster a contiguous range of equal cost instead made a 32768-row prefill 35 %
// slower: the ranges' weight tiles no longer meet in L2.)
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
// one vector over the tile's tokens, which scale warps write to a shared-memory ring.
//
// Roles per CTA: warp 0 loads weights and, when rows is NULL, tokens (TMA tiles);
// warp 1 allocates the tensor memory (pair), issues the MMAs in the leader CTA and in
// the other relays the epilogue's releases; then the scale warps, the warps that issue
// four-row gather loads when rows is given, and the epilogue.  The epilogue reads the
// accumulators as matrix fragments (a lane sees a quarter of the tokens, hence few scale
// reads) and stores through a transposing matrix store.  No load uses multicast.
//
// What bounds it, measured on one B200 (INT8 codes of normal values unless said):
//   INT8, 8 experts x 1024 rows, N = 8192: K = 5120 225-232 us (3000 TOPS; 4030 with zero
//     codes, so the power limit, not the pipeline), K = 2048 98-102 us (2750 TOPS).
//   INT8, 32768 rows over 64 experts, K = N = 2048: 122-126 us, gathered 124-130 us (104 us
//     with zero codes; 152 us in a long sequence, at lower clocks).  Token tiles that are not
//     full and the uneven last wave cost the rest.
//   INT8, 128 rows over 53 of 64 experts, K = 2048, N = 1536: 33.6 us, 5.0 TB/s in all.
//   FP8, 8198 rows over 8 experts, K = 5120, N = 2048: 119 us, 1440 TOPS (127 us
//     gathered, 148 us in a long sequence).  Of the gathered call's 127, with the
//     promotion's fused multiply-adds left out 105 us, with the tensor-memory reads too 102:
//     the hand-offs between loads, MMAs and releases.  L2 is at 24 % of its rate to the
//     SMs.  With branches on the warp's chunks inside the K loop and
//     both chunks read before either was added it took 139 us.
//     Slower variants, each against the kernel of its time (138-146 us): lanes as channels
//     with broadcast scales (220 us), 192- and 256-token tiles with two accumulators
//     (240-400 us); 16 epilogue warps of 32 columns gained nothing (143 us, decode 6 % slower)
//     and were not measured again on the present K loop.
//   FP8, 222 rows over 60 of 64 experts, K = 1408, N = 2048: 33.2 us, 5.2 TB/s in all.
//   Token rows copied by cp.async threads instead of TMA ran 2-3 times slower (the
//   proxy fences wait for every copy in flight).
#pragma once
#include <type_traits>
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
  int split;               // CTA pairs that share a tile's K: 2 to 4 with tiles of 32 tokens, else 1
};

// Tensor maps of the token rows: boxes of 16, 32, 64 and 128 rows, of which a tile
// takes the smallest that holds its half (one load per stage and CTA: a load's cost
// is mostly its own, a 96-row half fetched as 64 + 16 + 16 rows made the prefill of
// 32768 rows over 64 experts, K = N = 2048, take 167 us); [0] has one-row
// boxes when the tokens are gathered.
struct GroupedMaps {
  CUtensorMap m[4];
};

// BT: most tokens per tile.  256 (INT8, two accumulators for a tile each) and 128 (FP8,
// four for a K block each) fill the tensor memory.  32 is for calls of at most 32 rows
// with so few tiles that most SMs would idle (an SM pair reads about 100 bytes/ns, and
// a deeper ring does not change that): there a tile's K is split over the 2 to 4 CTA
// pairs of one cluster.  The other pairs' partial sums meet in the first's shared
// memory and are added in the order of K, so the answer does not depend on timing.
// Measured with one row per expert, N = 2048 (8 tiles per expert), us (32 rows in all: up to
// 0.5 us more with two pairs and more, the rest alike), on 1, 2, 3 and 4 pairs per tile:
//   tiles, K      INT8                       FP8
//    8, 1024       5.6   6.1   6.1   6.6      6.1   6.5   6.5   7.0
//    8, 2048       8.0   7.7   7.3   7.8      8.6   8.0   7.6   7.9
//    8, 5120      13.7  10.5   9.2   9.3     14.5  11.1   9.8   9.8
//   16, 1536       7.3   7.5   7.8            7.9   8.0   8.1
//   16, 2048       8.2   8.0   8.2            8.9   8.4   8.6
//   16, 5120      13.8  10.7  10.3           14.6  11.5  10.9
//   24, 2048       8.3   8.7                  9.0   9.2
//   24, 2560       9.3   9.3                 10.0   9.9
//   24, 3584      11.1  10.3                 11.9  11.0
//   32, 2048       8.5   9.5                  9.2  10.0
//   32, 2560       9.4  10.1                 10.1  10.7
//   32, 3584      11.3  11.4                 12.1  11.9
//   32, 5120      14.2  13.3                 15.0  13.8
// With more tiles than resident clusters the 32-token tiles on one pair are no faster
// than the wide ones (8 to 64 rows: 0 to 4 % slower), so those run the wide ones.
template <bool F8_, int BT_>
struct GroupedCfg {
  static constexpr bool F8 = F8_;
  static constexpr int BT = BT_;
  static constexpr int NACC = F8 ? 4 : 2;        // accumulators (BT tensor-memory columns each)
  static constexpr bool SPLIT = BT == 32;        // K is split over the cluster's pairs
  static constexpr int STAGES = BT == 32 || F8 ? 8 : 6;
  static constexpr int PART_BYTES = 128 * 32 * 4;  // one CTA's partial sums of a split tile
  static constexpr int A_BYTES = 128 * 128;      // weights staged by each CTA per K block
  static constexpr int B_BYTES = BT / 2 * 128;   // tokens staged by each CTA per K block, at most
  static constexpr int TMEM_COLS = 512;
  static constexpr int NS = F8 ? 2 : 1;          // scale warps
  static constexpr int NG = F8 ? 4 : 8;          // warps that issue gather loads
  static constexpr int NE = 8;                   // epilogue warps
  static constexpr int EPI0 = 2 + NS + NG;       // first epilogue warp
  static constexpr int THREADS = (EPI0 + NE) * 32;
  static constexpr int SV = F8 ? 4 : 1;          // scale vectors per ring slot: K blocks, or a tile's
  static constexpr int SSLOTS = 4;               // ring slots
  // FP8: registers move from the first eight warps to the epilogue's eight, which hold 64
  // sums and 64 partials per thread: 512 threads launch with 128 each, 8 * 80 + 8 *
  // 176 = 16 * 128 (no spills; at 72 and 184 the scale warps spilled).
  static constexpr int CONTROL_REGS = 80, EPI_REGS = 176;
  static constexpr int PITCH = 80;               // bytes per token in a warp's store staging
  static constexpr int OFF_B = STAGES * A_BYTES;
  static constexpr int OFF_SC = OFF_B + STAGES * B_BYTES;
  static constexpr int OFF_VALID = OFF_SC + SSLOTS * SV * BT * 4;  // a bit per token and slot
  static constexpr int OFF_INFO = OFF_VALID + SSLOTS * ((BT / 32 * 4 + 15) & ~15);  // a slot's tile
  static constexpr int OFF_ST = OFF_INFO + SSLOTS * 16;
  static constexpr int OFF_PART = OFF_ST + NE * 16 * PITCH;
  static constexpr int OFF_ROWS = OFF_PART + (SPLIT ? 3 * PART_BYTES : 0);
  static constexpr int OFF_LO = OFF_ROWS + (SPLIT ? BT * 4 : 0);
  static constexpr int OFF_CUM = OFF_LO + (kMaxExperts + 1) * 4;
  static constexpr int OFF_BAR = (OFF_CUM + (kMaxExperts + 1) * 4 + 7) & ~7;
  static constexpr int NUM_BARS = 2 * STAGES + 2 * NACC + 2 * SSLOTS + 4;
  static constexpr int OFF_MISC = OFF_BAR + NUM_BARS * 8;
  static constexpr int smem_bytes() { return 1024 + OFF_MISC + 16; }
  static_assert(1024 + OFF_MISC + 16 <= 232448, "shared memory");
  static_assert(!F8 || (EPI0 == 8 && THREADS == 512 && CONTROL_REGS + EPI_REGS <= 2 * 128),
                "the register split stays within what the block launches with");
  static_assert(NACC * BT <= 512, "tensor memory");
  static_assert(!F8 || BT <= 128, "FP8 epilogue: two groups of at most 64 columns");
};

// Asynchronous load of 32 columns of 16 tensor-memory lanes (taddr: lane 0 or 16 of
// the warp's quadrant) as matrix fragments: lane l gets, for columns 8 i + 2 (l % 4)
// and the next, rows l / 4 (r[4 i], r[4 i + 1]) and l / 4 + 8 (r[4 i + 2], r[4 i + 3]).
// A lane sees a quarter of the columns, so the per-token scales are four times fewer
// reads than with one lane per channel.
__device__ __forceinline__ void tmem_frag32_async(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// 32 columns of all 32 lanes of the quadrant: v[h] rows 16 h ..
__device__ __forceinline__ void tmem_frags_async(uint32_t taddr, uint32_t (&v)[2][16]) {
  tmem_frag32_async(taddr, v[0]);
  tmem_frag32_async(taddr + (16u << 16), v[1]);
}
// Completes this thread's tensor-memory loads; v's values may be used after it.
__device__ __forceinline__ void tmem_frags_wait(uint32_t (&v)[2][16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 16; i += 8)  // orders the uses after the wait
      asm volatile(""
                   : "+r"(v[h][i]), "+r"(v[h][i + 1]), "+r"(v[h][i + 2]), "+r"(v[h][i + 3]),
                     "+r"(v[h][i + 4]), "+r"(v[h][i + 5]), "+r"(v[h][i + 6]), "+r"(v[h][i + 7]));
}

// Two fp32 fused multiply-adds, each rounded as fmaf: (a0, a1) * f + c.
__device__ __forceinline__ uint64_t fma2(uint32_t a0, uint32_t a1, uint64_t f, uint64_t c) {
  uint64_t d;
  asm("{\n\t.reg .b64 a;\n\tmov.b64 a, {%1, %2};\n\tfma.rn.f32x2 %0, a, %3, %4;\n\t}"
      : "=l"(d)
      : "r"(a0), "r"(a1), "l"(f), "l"(c));
  return d;
}

// Arrive (once the pair's MMAs issued so far are done) on the mbarrier at this offset in
// both CTAs of the pair led by cluster rank `lead`.
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .b16 m;\n\tcvt.u16.u32 m, %1;\n\t"
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], m;\n\t}" ::"r"(smem_u32(bar)),
      "r"(3u << lead)
      : "memory");
}

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

// The tile list: expert by expert, channel tile by channel tile, the token tiles of a
// weight tile next to each other.  cum[e] counts the token tiles of the experts before e.
// Working a tile out takes a few hundred cycles, so only the warps that run ahead do (loads,
// MMA, scales); the epilogue finds its tile with the first scales.  (With every warp
// searching expert by expert, 1200 cycles of the epilogue's 13400 per tile, FP8 K = 2048,
// went there: 4100 rows over 32 experts, K = 1024, 27.2 us against 26.0.)
struct GroupedWalk {
  const int* lo;
  const int* cum;
  int tiles_n, E, e;
  __device__ __forceinline__ GroupedWalk(const int* lo_, const int* cum_, int tiles_n_, int E_)
      : lo(lo_), cum(cum_), tiles_n(tiles_n_), E(E_), e(0) {}
  // tile t of the list, for the whole warp; t must not decrease from call to call
  __device__ __forceinline__ GroupedTile at(int t) {
    const int lane = threadIdx.x & 31;
    for (;; e += 32) {  // the first expert whose tiles end after t, 32 at a time
      const int next = min(e + 1 + lane, E);
      const uint32_t after = __ballot_sync(0xffffffffu, cum[next] * tiles_n > t);
      if (after) {
        e += __ffs(after) - 1;
        break;
      }
    }
    const int nt = cum[e + 1] - cum[e];
    const int i = t - cum[e] * tiles_n;
    const int r = lo[e + 1] - lo[e];
    GroupedTile g;
    g.e = e;
    g.ct = i;
    g.row0 = lo[e];
    g.nrows = r;
    if (nt > 1) {
      const int w = ((r + nt - 1) / nt + 31) & ~31;  // rows per token tile, at most BT
      g.ct = i / nt;
      const int tt = i - g.ct * nt;
      g.row0 += tt * w;
      g.nrows = min(w, r - tt * w);
    }
    return g;
  }
};

// Stores 16 tokens x 32 channels of one warp as bf16.  p[b][k]: this lane's fragment
// of tokens 8 b .. 8 b + 7 and channels 8 k .. 8 k + 7 (its row is the channel, its two
// values two tokens).  A transposing matrix store puts every token's 32 channels
// side by side in the warp's staging rows, which leave in 16-byte pieces.
// out: token 0, channel 0 of the block; the first ntok tokens are stored, as zeros
// where their bit in `valid` is clear (a padding row is zero whatever the expert's
// weights and scales hold); ch_ok: channels 8 (lane % 4) .. + 7 exist.
template <int PITCH>
__device__ __forceinline__ void grouped_store(uint32_t st, __nv_bfloat16* out, size_t N, int lane,
                                              const uint32_t (&p)[2][4], int ntok, uint32_t valid,
                                              bool ch_ok) {
  const uint32_t to = st + (lane & 7) * PITCH + (lane >> 3) * 16;
  __syncwarp();  // the previous block has been read
#pragma unroll
  for (int b = 0; b < 2; ++b)
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                     to + b * 8 * PITCH),
                 "r"(p[b][0]), "r"(p[b][1]), "r"(p[b][2]), "r"(p[b][3])
                 : "memory");
  __syncwarp();
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int t = b * 8 + (lane >> 2);
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(st + t * PITCH + (lane & 3) * 16)
                 : "memory");
    if (!(valid >> t & 1u)) v = make_uint4(0, 0, 0, 0);
    if (t < ntok && ch_ok) *reinterpret_cast<uint4*>(out + t * N + (lane & 3) * 8) = v;
  }
}

template <class Cfg>
__global__ void __launch_bounds__(Cfg::THREADS, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmW,   // weights [E N, K], 128-row boxes
                   const __grid_constant__ GroupedMaps tmX,   // tokens
                   const GroupedArgs g) {
  constexpr int STAGES = Cfg::STAGES, NACC = Cfg::NACC, NE = Cfg::NE, BT = Cfg::BT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* smA = smem;
  uint8_t* smB = smem + Cfg::OFF_B;
  float* ring = reinterpret_cast<float*>(smem + Cfg::OFF_SC);
  uint32_t* valid = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_VALID);
  int4* info = reinterpret_cast<int4*>(smem + Cfg::OFF_INFO);
  int* lo = reinterpret_cast<int*>(smem + Cfg::OFF_LO);
  int* cum = reinterpret_cast<int*>(smem + Cfg::OFF_CUM);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Cfg::OFF_BAR);
  uint64_t* full = bars;                 // leader: pair's tiles of a stage have landed
  uint64_t* empty = bars + STAGES;       // both: the pair's MMAs are done with a stage
  uint64_t* tfull = bars + 2 * STAGES;   // both: an accumulator is complete
  uint64_t* tfree = tfull + NACC;        // both: this CTA's epilogue (leader: both CTAs') released one
  uint64_t* sfull = tfree + NACC;        // both: a slot of the scale ring is written
  uint64_t* sfree = sfull + Cfg::SSLOTS; // both: the epilogue is done with it
  uint64_t* pfull = sfree + Cfg::SSLOTS; // first pair: another pair's partial sums have arrived
  uint64_t* drain = pfull + 3;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + Cfg::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cfg::OFF_MISC + 4);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t crank = cluster_ctarank();
  const uint32_t rank = crank & 1u;      // within the CTA pair
  const uint32_t lead = crank & ~1u;     // the pair's leader
  const bool leader = rank == 0;
  const int split = Cfg::SPLIT ? g.split : 1;
  const int pair = Cfg::SPLIT ? static_cast<int>(crank >> 1) : 0;
  const int cluster = blockIdx.x / (2 * split);
  const int nclusters = gridDim.x / (2 * split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int a = 0; a < NACC; ++a) {
      mbar_init(tfull + a, 1);
      mbar_init(tfree + a, leader ? NE + 1 : NE);
    }
    for (int i = 0; i < Cfg::SSLOTS; ++i) {
      mbar_init(sfull + i, 1);
      mbar_init(sfree + i, NE);
    }
    for (int i = 0; i < 3; ++i) mbar_init(pfull + i, 4);
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
    tma_prefetch_desc(&tmX.m[0]);
  }
  tc_fence_before();
  cluster_sync();  // barriers of every CTA initialised, tensor memory allocated in both of a pair
  tc_fence_after();
  // Nothing above touches global memory, so the launch may overlap any kernel.  What that
  // kernel may have written is read below through L2, not through the read-only path.
  griddep_wait();
  // A call of at most 32 rows fetches their indexes with the offsets (one latency, not two).
  int* near_rows = reinterpret_cast<int*>(smem + Cfg::OFF_ROWS);
  if constexpr (Cfg::SPLIT) {
    const int i = static_cast<int>(threadIdx.x) - (Cfg::THREADS - BT);
    if (g.rows && i >= 0 && i < g.T) near_rows[i] = __ldcg(g.rows + i);
  }
  auto row_index = [&](int t) {
    if constexpr (Cfg::SPLIT) return near_rows[t];
    else return __ldcg(g.rows + t);
  };
  // offsets, held inside [0, T] and non-decreasing whatever the caller wrote
  for (int e = threadIdx.x; e <= g.E; e += Cfg::THREADS) lo[e] = min(max(__ldcg(g.offsets + e), 0), g.T);
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
  __syncthreads();
  const uint32_t tmem = *tmem_holder;
  const int num_tiles = cum[g.E] * g.tiles_n;
  const int kbt = g.kb_total;
  // this pair's K blocks: nk of them from k0
  const int k0 = Cfg::SPLIT ? kbt * pair / split : 0;
  const int nk = Cfg::SPLIT ? kbt * (pair + 1) / split - k0 : kbt;
  griddep_launch_dependents();

  if (warp < Cfg::EPI0) {
    if constexpr (Cfg::F8) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::CONTROL_REGS));
    if (warp == 0) {
      // ------------------------------- weights, and tokens in row order (TMA)
      const uint32_t full_leader = mapa_shared(smem_u32(full), lead);
      const uint64_t pol = policy_evict_normal();
      GroupedWalk walk(lo, cum, g.tiles_n, g.E);
      uint32_t stage = 0, phase = 0;
      long long fills = 0;
      bool ok = true;
      for (int t = cluster; ok && t < num_tiles; t += nclusters) {
        const GroupedTile tile = walk.at(t);
        const int n = (tile.nrows + 31) & ~31;
        const int half = n >> 1;  // token rows staged by this CTA
        const int w_row = tile.e * g.N + tile.ct * 256 + static_cast<int>(rank) * 128;
        const int x_row = tile.row0 + static_cast<int>(rank) * half;
        // the smallest box of 16 << box rows that holds the half
        const int box = half <= 16 ? 0 : half <= 32 ? 1 : half <= 64 ? 2 : 3;
        const uint32_t bytes = 2 * (Cfg::A_BYTES + (g.rows ? half : 16 << box) * 128);
        if (lane == 0) {
          for (int kb = 0; kb < nk; ++kb) {
            if (!wait_bounded(empty + stage, phase ^ 1u, abort_flag)) {
              ok = false;
              break;
            }
            if (leader) {
              mbar_arrive_expect_tx(full + stage, bytes);
            }
            tma_load_2d_pair(smA + stage * Cfg::A_BYTES, &tmW, (k0 + kb) * 128, w_row,
                             full_leader + stage * 8, pol);
            if (!g.rows)
              tma_load_2d_pair(smB + stage * Cfg::B_BYTES, &tmX.m[box], (k0 + kb) * 128, x_row,
                               full_leader + stage * 8, pol);
            ++fills;
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (lane == 0 && leader) {
        // the pair's copies (both CTAs' bytes count here) have all landed
        for (int st = 0; st < STAGES; ++st) {
          const long long n = fills / STAGES + (st < fills % STAGES ? 1 : 0);
          if (n > 0) wait_drain(full + st, static_cast<uint32_t>((n - 1) & 1));
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------ MMA issuer (leader), relay (other CTA)
      // The other CTA's releases of an accumulator reach the leader as one arrival: its
      // epilogue warps arrive on their own CTA's barrier and this warp passes it on.
      if (!leader) {
        const uint32_t tfree_leader = mapa_shared(smem_u32(tfree), lead);
        uint32_t local = 0;
        bool ok = true;
        for (int t = cluster; ok && t < num_tiles; t += nclusters)
          for (int i = 0; i < (Cfg::F8 ? nk : 1); ++i, ++local) {
            const uint32_t a = local % NACC, u = local / NACC;
            if (!prompt_wait(tfree + a, u & 1u, abort_flag)) { ok = false; break; }
            if (lane == 0) mbar_arrive_remote(tfree_leader + a * 8);
            __syncwarp();
          }
      }
      if (leader) {
        GroupedWalk walk(lo, cum, g.tiles_n, g.E);
        uint32_t stage = 0, phase = 0, local = 0;
        bool ok = true;
        for (int t = cluster; ok && t < num_tiles; t += nclusters) {
          const int n = (walk.at(t).nrows + 31) & ~31;
          const uint32_t idesc = Cfg::F8 ? idesc_e4m3_f32_m256(n) : idesc_i8_s32_m256(n);
          uint32_t d = 0;
          for (int kb = 0; kb < nk; ++kb) {
            if (Cfg::F8 || kb == 0) {  // a free accumulator: per K block (FP8) or per tile
              const uint32_t a = local % NACC, u = local / NACC;
              ++local;
              ok = prompt_wait2(tfree + a, (u & 1u) ^ 1u, full + stage, phase, abort_flag);
              d = tmem + a * BT;
            } else {
              ok = prompt_wait(full + stage, phase, abort_flag);
            }
            if (!ok) break;
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
              commit_pair(empty + stage, lead);
              if (Cfg::F8 || kb == nk - 1) commit_pair(tfull + (local - 1) % NACC, lead);
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
    } else if (warp >= 2 + Cfg::NS) {
      // ---------------------------------------------------- gathered tokens
      // Warps take the stages in turn, NG / 4 of them to a stage, and each lane fetches four
      // rows; the warps of a stage share the loads evenly.  A load takes its warp about
      // 80 cycles to issue and a stage's wait over 100, so the loads are spread over
      // warps and the waits are not repeated by all of them: the prefill of 32768 rows
      // over 64 experts, K = N = 2048, took 346 us with one warp, 152 with four and 138
      // with eight on every stage, 130 and 127 us with eight on every second and fourth.
      if (g.rows) {
        const uint32_t full_leader = mapa_shared(smem_u32(full), lead);
        constexpr int TURNS = 4, WARPS = Cfg::NG / TURNS;  // warps of a stage
        // A parity wait tells a phase from the next only.  Before fill f (which waits until fill
        // f - STAGES is consumed) this warp saw fill f - TURNS - STAGES consumed, and so
        // fill f - 2 STAGES: the wait cannot take that phase for its own.
        static_assert(TURNS <= STAGES && WARPS * TURNS == Cfg::NG, "gather warps");
        const int gw = warp - 2 - Cfg::NS;
        const int j = (lane * WARPS + gw / TURNS) * 4;
        int skip = gw % TURNS;  // stages until this warp's next
        GroupedWalk walk(lo, cum, g.tiles_n, g.E);
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        for (int t = cluster; ok && t < num_tiles; t += nclusters) {
          const GroupedTile tile = walk.at(t);
          const int half = ((tile.nrows + 31) & ~31) >> 1;
          const int first = static_cast<int>(rank) * half + j;
          // rows past the tile or outside the tokens are fetched as zeros
          auto token = [&](int i) {
            if (first + i >= tile.nrows) return g.M;
            const int r = row_index(tile.row0 + first + i);
            return static_cast<unsigned>(r) < static_cast<unsigned>(g.M) ? r : g.M;
          };
          const bool mine = j < half;
          int4 r4 = make_int4(g.M, g.M, g.M, g.M);
          if (mine) r4 = make_int4(token(0), token(1), token(2), token(3));
          for (int kb = 0; kb < nk; ++kb) {
            if (skip == 0) {
              if (!warp_wait_bounded(empty + stage, phase ^ 1u, abort_flag)) {
                ok = false;
                break;
              }
              if (mine)
                tma_gather4_pair(smB + stage * Cfg::B_BYTES + j * 128, &tmX.m[0], (k0 + kb) * 128, r4,
                                 full_leader + stage * 8);
              __syncwarp();
            }
            skip = skip == 0 ? TURNS - 1 : skip - 1;
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
    } else {
      // ------------------------------------------------------------- scales
      // A ring slot holds SV vectors over the tile's tokens: INT8 the tile's s_tok; FP8 s_a *
      // s_w of four K blocks (0 for rows outside).  FP8: two warps fill slots in turn,
      // each with its next slot's loads in flight.  One warp that loaded, wrote and
      // then loaded again gave four K blocks per L2 latency, and decode of 222
      // rows over 64 experts (K = 1408, N = 2048) took 55 us.
      constexpr int NV = BT / 32;
      GroupedWalk walk(lo, cum, g.tiles_n, g.E);
      uint32_t slot = 0, phase = 0;
      const uint32_t mine = warp - 2;  // FP8: the slots of this parity
      bool ok = true;
      for (int t = cluster; ok && t < num_tiles; t += nclusters) {
        const GroupedTile tile = walk.at(t);
        int tok[NV];  // token of column 32 i + lane, -1: none
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = i * 32 + lane;
          tok[i] = -1;
          if (c < tile.nrows) {
            const int r = g.rows ? row_index(tile.row0 + c) : tile.row0 + c;
            if (static_cast<unsigned>(r) < static_cast<unsigned>(g.M)) tok[i] = r;
          }
        }
        // word i of a slot's bits: which of columns 32 i .. 32 i + 31 have a token
        auto write_valid = [&]() {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const uint32_t has = __ballot_sync(0xffffffffu, tok[i] >= 0);
            if (lane == 0) valid[slot * NV + i] = has;
          }
        };
        auto next_slot = [&]() {
          if (++slot == Cfg::SSLOTS) { slot = 0; phase ^= 1u; }
        };
        if constexpr (!Cfg::F8) {
          float v[NV];
#pragma unroll
          for (int i = 0; i < NV; ++i) v[i] = tok[i] >= 0 ? __ldcg(g.s_a + tok[i]) : 0.0f;
          if (!warp_wait_bounded(sfree + slot, phase ^ 1u, abort_flag)) { ok = false; break; }
#pragma unroll
          for (int i = 0; i < NV; ++i) ring[slot * BT + i * 32 + lane] = v[i];
          write_valid();
          if (lane == 0) info[slot] = make_int4(tile.row0, tile.nrows, tile.e, tile.ct);
          __syncwarp();
          if (lane == 0) mbar_arrive(sfull + slot);
          next_slot();
        } else {
          const int ch0 = tile.ct * 256 + static_cast<int>(rank) * 128;
          const float* sw =
              g.s_w + (static_cast<size_t>(tile.e) * (g.N >> 7) + (ch0 < g.N ? ch0 >> 7 : 0)) * kbt + k0;
          const bool wide = ((kbt | k0) & 3) == 0;  // a token's scales can be loaded four K blocks at a time
          // scales of K blocks kb .. kb + 3 (0 past the last)
          auto load4 = [&](const float* p, int kb) {
            if (wide) return __ldcg(reinterpret_cast<const float4*>(p + kb));
            return make_float4(__ldcg(p + kb), kb + 1 < nk ? __ldcg(p + kb + 1) : 0.0f,
                               kb + 2 < nk ? __ldcg(p + kb + 2) : 0.0f,
                               kb + 3 < nk ? __ldcg(p + kb + 3) : 0.0f);
          };
          float4 w, v[NV];
          auto fetch = [&](int kb) {
            w = load4(sw, kb);
#pragma unroll
            for (int i = 0; i < NV; ++i)
              v[i] = tok[i] >= 0 ? load4(g.s_a + static_cast<size_t>(tok[i]) * kbt + k0, kb)
                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          };
          int kb = (slot & 1u) == mine ? 0 : 4;  // this warp's first batch of the tile
          if (kb < nk) fetch(kb);
          for (int b = 0; b < nk; b += 4, next_slot()) {
            if ((slot & 1u) != mine) continue;
            if (!warp_wait_bounded(sfree + slot, phase ^ 1u, abort_flag)) { ok = false; break; }
            float* to = ring + slot * (Cfg::SV * BT) + lane;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
              to[i * 32] = __fmul_rn(v[i].x, w.x);
              to[BT + i * 32] = __fmul_rn(v[i].y, w.y);
              to[2 * BT + i * 32] = __fmul_rn(v[i].z, w.z);
              to[3 * BT + i * 32] = __fmul_rn(v[i].w, w.w);
            }
            if (b == 0 && lane == 0) info[slot] = make_int4(tile.row0, tile.nrows, tile.e, tile.ct);
            if (b + 4 >= nk) write_valid();  // the epilogue reads them with the tile's last slot
            __syncwarp();
            if (lane == 0) mbar_arrive(sfull + slot);
            kb += 8;
            if (kb < nk) fetch(kb);
          }
        }
      }
    }
  } else {
    if constexpr (Cfg::F8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::EPI_REGS));
    // ------------------------------------------------------------ epilogue
    const int ew = warp - Cfg::EPI0;
    const int q = warp & 3;                 // tensor-memory lane quadrant: 32 channels
    const int grp = ew >> 2;                // which columns of the tile
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const uint32_t st = smem_u32(smem + Cfg::OFF_ST + ew * 16 * Cfg::PITCH);
    const size_t N = static_cast<size_t>(g.N);
    auto release = [&](uint32_t a) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tfree + a);
    };
    // Split tiles: the other pairs hand their 32 values per thread to the same thread of
    // the first pair, which adds them in the order of the pairs (a cluster has at
    // most one tile then, so no buffer is used twice).  False: a wait gave up.
    auto combine = [&](auto&& value, auto&& add) {
      uint8_t* mine = smem + Cfg::OFF_PART + q * 4096 + lane * 16;
      if (pair > 0) {
        const uint32_t to = mapa_shared(smem_u32(mine + (pair - 1) * Cfg::PART_BYTES), rank);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_cluster_v4(to + i * 512, value(4 * i), value(4 * i + 1), value(4 * i + 2), value(4 * i + 3));
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(pfull + pair - 1), rank));
        return true;
      }
      for (int p = 0; p < split - 1; ++p) {
        if (!__all_sync(0xffffffffu, wait_bounded_cluster(pfull + p, 0, abort_flag))) return false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 x = *reinterpret_cast<const uint4*>(mine + p * Cfg::PART_BYTES + i * 512);
          add(4 * i, x.x);
          add(4 * i + 1, x.y);
          add(4 * i + 2, x.z);
          add(4 * i + 3, x.w);
        }
      }
      return true;
    };
    uint32_t local = 0, sslot = 0, sphase = 0;
    bool ok = true;
    for (int t = cluster; ok && t < num_tiles; t += nclusters) {
      if (!warp_wait_bounded(sfull + sslot, sphase, abort_flag)) break;
      const int4 in = info[sslot];  // row0, nrows, e, ct
      const GroupedTile tile = {in.z, in.w, in.x, in.y};
      const int n = (tile.nrows + 31) & ~31;
      const int ch = tile.ct * 256 + static_cast<int>(rank) * 128 + q * 32;  // this warp's channels
      const bool ch_ok = ch + (lane & 3) * 8 < g.N;
      __nv_bfloat16* out = g.out + static_cast<size_t>(tile.row0) * N + ch;
      auto next_scales = [&]() {  // done with the slot's vectors
        __syncwarp();
        if (lane == 0) mbar_arrive(sfree + sslot);
        if (++sslot == Cfg::SSLOTS) { sslot = 0; sphase ^= 1u; }
      };
      if constexpr (!Cfg::F8) {
        float s_ch[4];  // of channels 8 k + lane / 4
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = ch + 8 * k + (lane >> 2);
          s_ch[k] = c < g.N ? __ldcg(g.s_w + static_cast<size_t>(tile.e) * N + c) : 0.0f;
        }
        const uint32_t a = local % NACC, u = local / NACC;
        const float* slot = ring + sslot * BT;
        ++local;
        if (!warp_wait_bounded(tfull + a, u & 1u, abort_flag)) break;
        tc_fence_after();
        const uint32_t src = lanes + a * BT;
#pragma unroll 1
        for (int c = grp * 32; c < n; c += (NE / 4) * 32) {
          uint32_t v[2][16];
          tmem_frags_async(src + c, v);
          tmem_frags_wait(v);
          if constexpr (Cfg::SPLIT) {
            ok = combine([&](int i) { return v[i >> 4][i & 15]; },
                         [&](int i, uint32_t x) { v[i >> 4][i & 15] += x; });
            if (pair > 0 || !ok) break;
          }
          const uint32_t bits = valid[sslot * (BT / 32) + (c >> 5)];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t pk[2][4];
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const float2 s = *reinterpret_cast<const float2*>(slot + c + i * 16 + b * 8 + (lane & 3) * 2);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint32_t* x = &v[k >> 1][8 * i + 4 * b + 2 * (k & 1)];
                pk[b][k] = pack_bf16x2(
                    __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(x[0])), s.x), s_ch[k]),
                    __fmul_rn(__fmul_rn(__int2float_rn(static_cast<int>(x[1])), s.y), s_ch[k]));
              }
            }
            grouped_store<Cfg::PITCH>(st, out + (c + i * 16) * N, N, lane, pk,
                                      tile.nrows - c - i * 16, bits >> (i * 16), ch_ok);
          }
        }
        release(a);
        next_scales();
      } else {
        // this warp's columns: 64 or, of a tile of at most 64, 32; in two chunks of 32
        const int wcol = n > 64 ? 64 : 32;
        const int col0 = grp * wcol;
        const bool has0 = col0 < n, has1 = wcol == 64 && col0 + 32 < n;
        uint64_t acc[2][2][8];  // pairs of fp32 sums of neighbouring tokens
#pragma unroll
        for (int j = 0; j < 32; ++j) (&acc[0][0][0])[j] = 0;
        uint32_t v[2][2][16];   // one K block's partials
        uint64_t f[2][4] = {};  // and scales (pairs)
        const uint32_t src = lanes + col0;
        // acc += partials * scales of one chunk
        auto add = [&](uint64_t (&x)[2][8], const uint32_t (&y)[2][16], const uint64_t (&f)[4]) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int r = 2 * i; r < 2 * i + 2; ++r)
                x[h][r] = fma2(y[h][2 * r], y[h][2 * r + 1], f[i], x[h][r]);
        };
        // The tile's K blocks for a warp with this many chunks, without a branch on
        // them inside the loop.  K blocks are taken in pairs on one poll (a poll takes over
        // 100 cycles even when it succeeds; commits arrive in order, so the second is
        // complete after the first).  With two chunks, one's partials are read while the
        // other's are added.  False: a wait gave up.
        auto k_blocks = [&](auto chunks) -> bool {
          constexpr int CH = decltype(chunks)::value;
          auto load_scales = [&](int kb) {
            const float* s = ring + (sslot * Cfg::SV + (kb & 3)) * BT + col0 + (lane & 3) * 2;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
              for (int i = 0; i < 4; ++i) f[c][i] = *reinterpret_cast<const uint64_t*>(s + c * 32 + i * 8);
          };
          auto load = [&](uint32_t l, int c) {
            if (c < CH) tmem_frags_async(src + l % NACC * BT + 32 * c, v[c]);
          };
          // one K block, whose first chunk is on its way
          auto block = [&](uint32_t l) {
            if constexpr (CH > 0) tmem_frags_wait(v[0]);
            if constexpr (CH == 2) load(l, 1);
            else release(l % NACC);
            if constexpr (CH > 0) add(acc[0], v[0], f[0]);
            if constexpr (CH == 2) {
              tmem_frags_wait(v[1]);
              release(l % NACC);
            }
          };
          auto rest = [&]() {  // after the next block's load
            if constexpr (CH == 2) add(acc[1], v[1], f[1]);
          };
          const uint32_t l1 = local + (nk > 1 ? 1 : 0);
          if (!prompt_wait(tfull + l1 % NACC, l1 / NACC & 1u, abort_flag)) return false;
          tc_fence_after();
          load(local, 0);
          for (int kb = 0; kb < nk; kb += 2) {
            // (at kb = 0 for the second time: a branch around it cost more)
            if ((kb & 3) == 0 && !prompt_wait(sfull + sslot, sphase, abort_flag)) return false;
            load_scales(kb);
            const bool two = kb + 1 < nk, more = kb + 2 < nk;
            const uint32_t l2 = local + 2, l3 = kb + 3 < nk ? local + 3 : l2;  // the next pair
            block(local);
            const bool polled = more && prompt_try_wait(smem_u32(tfull + l3 % NACC), l3 / NACC & 1u);
            if (two) {
              load(local + 1, 0);
              rest();
              load_scales(kb + 1);
              block(local + 1);
            }
            const bool early = __all_sync(0xffffffffu, polled);
            if (early) {
              tc_fence_after();
              load(l2, 0);
            }
            rest();
            if ((kb & 2) && more) next_scales();
            local += two ? 2 : 1;
            if (more && !early) {
              if (!prompt_wait(tfull + l3 % NACC, l3 / NACC & 1u, abort_flag)) return false;
              tc_fence_after();
              load(l2, 0);
            }
          }
          return true;
        };
        if constexpr (BT > 32) {
          if (has1) ok = k_blocks(std::integral_constant<int, 2>());
        }
        if (!has1)
          ok = has0 ? k_blocks(std::integral_constant<int, 1>()) : k_blocks(std::integral_constant<int, 0>());
        if (!ok) break;
        // the last slot is held until the stores: its bits, read earlier, cost a spill
        const uint32_t* bits = valid + sslot * (BT / 32) + (col0 >> 5);
        if constexpr (Cfg::SPLIT) {
          if (has0) {
            float sum[32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
              sum[i] = __uint_as_float(static_cast<uint32_t>(acc[0][i >> 4][(i >> 1) & 7] >> (32 * (i & 1))));
            ok = combine([&](int i) { return __float_as_uint(sum[i]); },
                         [&](int i, uint32_t x) { sum[i] = __fadd_rn(sum[i], __uint_as_float(x)); });
#pragma unroll
            for (int i = 0; i < 16; ++i)
              acc[0][i >> 3][i & 7] = static_cast<uint64_t>(__float_as_uint(sum[2 * i + 1])) << 32 |
                                      __float_as_uint(sum[2 * i]);
            if (pair > 0 || !ok) break;  // the cluster's only tile
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < 2 ? has0 : has1) {
            uint32_t pk[2][4];
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const uint64_t x = acc[i >> 1][k >> 1][4 * (i & 1) + 2 * b + (k & 1)];
                pk[b][k] = pack_bf16x2(__uint_as_float(static_cast<uint32_t>(x)),
                                       __uint_as_float(static_cast<uint32_t>(x >> 32)));
              }
            grouped_store<Cfg::PITCH>(st, out + (col0 + i * 16) * N, N, lane, pk,
                                      tile.nrows - col0 - i * 16, bits[i >> 1] >> (16 * (i & 1)), ch_ok);
          }
        next_scales();
      }
    }
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");  // a wait may have given up before it
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
