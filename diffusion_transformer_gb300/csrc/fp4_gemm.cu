// Product of two microscaled 4-bit matrices on the block-scaled tcgen05 MMA: out = A B^T, A [M, K], B
// [N, K] in the layout of fp4_layout.h, fp32 accumulators in tensor memory, the NV format's row scales applied
// to the accumulator as it is drained.
//
// A 128-byte swizzled shared-memory row holds 256 codes, so a pipeline stage is K = 256: four MMAs of
// K = 64, preceded by the copies of the stage's scale chunks from shared to tensor memory.
//
// Two kernels:
//   pair   tiles of 256 rows of one operand by up to 256 of the other on CTA pairs (cta_group::2),
//          persistent, for products with enough tiles
//   split  128 rows of B against up to 128 rows of A per CTA, a cluster of CTAs sharing the K loop and
//          adding their partial tiles through distributed shared memory, for few rows or few tiles
//
// What bounds the pair kernel. A stage of a 256 x 256 tile takes each SM 512 cycles of MMA (247 ns at 2070 MHz).
// Measured per stage, 4096 x 24320 x 3072: 327 ns without an epilogue, 348 with all of it but the stores, 394
// in all (94.5 us; 32-value blocks, with half the scales and no factors: 87); 4096 x 4864 x 12288: 330 ns. What the 80
// ns over the MMA's own time are is not shown. A stage's 38 KB go into shared memory and out of it again: 152
// bytes per cycle at the MMA's pace, 115 at the measured one, where it moves 128; but tiles of 128 and 192 rows,
// with 31 and 35 KB and 124 and 185 ns of MMA, take 215 and 250 ns, about the same 65 to 90 more, so a wait in each
// stage (its scale copies for the MMAs before them, its MMAs for the copies) may be the cause as well. The output
// counts beside it: 32-byte stores from registers 94.5 us, staged in shared memory and stored by TMA 104, lanes
// exchanging pieces to store whole 128-byte lines 99.8, evict-first hints 96, four epilogue warps in place
// of eight 93 (104 when staged). 4224 x 24576 x 3072 with data that toggles bits: 104 us (6.1 PFLOP/s, tensor
// pipe 72 % active) in a burst, 112 to 123 back to back, where the power limit lowers the clock; 8192^3:
// 151 us, 7.3 PFLOP/s.
// What bounds the split kernel: B's bytes where rows are few (1 x 18432 x 3072: 6.2 us, 5.1 TB/s with B partly
// in L2), else the fixed 2 to 4 us of start, first loads and epilogue.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "fp4.cuh"
#include "fp4.h"
#include "fp4_choice.h"
#include "fp4_ptx.cuh"
#include "internal.h"
#include "tmap.h"

namespace dit {
namespace {

constexpr int kStageK = kFp4StageK;           // codes per stage and row: 128 bytes
constexpr uint32_t kTileBytes = 128 * 128;    // 128 rows of a stage
template <int FMT>
struct Scales {
  static constexpr bool kNv = FMT == DIT_FP4_NV;
  static constexpr int kGroups = kNv ? 4 : 2;             // 512-byte scale chunks per stage and 128 rows
  static constexpr uint32_t kBytes = kGroups * 512;
};

struct Fp4Params {
  int M, N, K;
  int* err;
  void* out;
  long long ldo;
  const float* a_scale;  // NV: row scales
  const float* b_scale;
  int early;             // B was complete before the kernel ahead of this one in the stream began
  int n_fast;            // tile order
  int bn, stages;        // rows of the narrow operand per tile (see each kernel), pipeline depth
};

__device__ __forceinline__ int stage_steps(int K, int kb) { return min(4, (K - kb * kStageK + 63) / 64); }

// ---------------------------------------------------------------------------------------------
// pair kernel
// ---------------------------------------------------------------------------------------------
// D [256 rows of P, bn rows of Q] per tile: P and Q are A and B, or (SWAP) B and A. Each CTA of the pair
// brings its 128 rows of P, half of the rows of Q, and the scales of its P rows and of all Q rows.
//
// Tensor memory, 512 columns: two accumulators and 48 columns of scales from 464 on. With bn = 256 the
// accumulators overlap by 48 columns ([0, 256) and [208, 464)): the overlapped columns are drained first
// and then handed over, so the next tile's MMAs wait for a quarter of an epilogue, not for all of it.
constexpr int kOverlapAt = 208, kSfCol = 464, kMaxStages = 8;
constexpr int kEpiWarps = 8, kPairThreads = 64 + 32 * kEpiWarps;
constexpr uint32_t kPairFixed = 1024 + kEpiWarps * 256 + 8 * (2 * kMaxStages + 5) + 16;

template <int FMT>
__host__ __device__ constexpr uint32_t pair_stage_bytes(int bn) {
  return kTileBytes + uint32_t(bn) * 64 + 3 * Scales<FMT>::kBytes;
}

// Four neighbouring products of one row times the row's factor, then times their columns' (two at a time,
// each product rounded by itself).
__device__ __forceinline__ void scale4(uint32_t* x, uint64_t row2, const float4& f) {
  const uint64_t lo = f2_mul(f2_mul(f2_pack(__uint_as_float(x[0]), __uint_as_float(x[1])), row2), f2_pack(f.x, f.y));
  const uint64_t hi = f2_mul(f2_mul(f2_pack(__uint_as_float(x[2]), __uint_as_float(x[3])), row2), f2_pack(f.z, f.w));
  x[0] = uint32_t(lo);
  x[1] = uint32_t(lo >> 32);
  x[2] = uint32_t(hi);
  x[3] = uint32_t(hi >> 32);
}
// Row factors of any size, so that a product is finite wherever its value is. An accumulator that is not zero lies
// between 2^-20 (the smallest codes and scales) and 2^53 (2688^2 times the longest K), a factor between 2^-112 and
// 2^117. The first factor as it is between 2^-100 and 2^64 makes neither an infinity nor a subnormal of any
// accumulator; a larger one is taken by 2^44 smaller, a smaller one by 2^44 larger, which is exact and keeps the
// products with the second factor in range too (past 2^128 the value itself is), and the result is put back after.
__device__ __forceinline__ float factor_back(float f) { return f > 0x1p64f ? 0x1p44f : (f > 0.f && f < 0x1p-100f ? 0x1p-44f : 1.f); }
__device__ __forceinline__ float factor_first(float f) {
  return f > 0x1p64f ? f * 0x1p-44f : (f > 0.f && f < 0x1p-100f ? f * 0x1p44f : f);
}
template <int N>
__device__ __forceinline__ void put_back(uint32_t* x, float back) {
#pragma unroll
  for (int c = 0; c < N; ++c) x[c] = __float_as_uint(__uint_as_float(x[c]) * back);
}

// z / (1 + e^-z); the approximate division is within two units of the fp32 result, which goes on to bf16 (for z from
// -88.7 to -87.3, where 1 + e^-z passes 2^126, it gives 0 in place of -5e-37 at most)
__device__ __forceinline__ float silu_bf16(float z) { return __fdividef(z, 1.f + __expf(-z)); }

// The QKV epilogue's part of one warp (the gizai:dit reference's prepOf; klein article, section 4.4): 128
// columns of the product, one head of 128 or two of 64, in the registers of the lanes that own the rows.
// Query and key heads are RMS-normed, weighted, rotated by the row's tables and stored head-major; value
// heads are transposed through the warp's 4 KB of shared memory (chunks of 32 columns: 64 bytes per row,
// 16-byte pieces swizzled by (row >> 1) & 3), so that a lane stores 32 rows of one value as 64 bytes.
// 128 columns in registers are more than the 168 that ten warps leave a thread: 88 bytes of them spill (16-value
// blocks; 144 for 32-value ones), and a lane per row makes a warp's access 32 pieces of 32 bytes in 32 lines. Both hold
// the QKV linear of 4224 x 9216 x 3072 at 83 us (78 for 32-value blocks), where its operations take 31.
template <int D>
__device__ __forceinline__ void qkv_store(const GemmParams& g, const uint32_t* w, int row0, int lane, int n0,
                                          uint8_t* scratch) {
  const int row = row0 + lane, H = g.H, R = g.M;
  const int which = n0 / H, head = (n0 - which * H) / D;
  auto val = [&](int c) { return __uint_as_float(w[c]); };
  if (which == 2) {
#pragma unroll
    for (int c = 0; c < D; c += 32) {
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t u[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) u[e] = pack_bf16x2(val(c + 8 * q + 2 * e), val(c + 8 * q + 2 * e + 1));
        *reinterpret_cast<uint4*>(scratch + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
      }
      __syncwarp();
      uint32_t col[16];
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        const int at = r * 64 + (((lane >> 3) ^ ((r >> 1) & 3)) << 4) + (lane & 7) * 2;
        const uint32_t x = *reinterpret_cast<const uint16_t*>(scratch + at);
        col[r >> 1] = r & 1 ? col[r >> 1] | x << 16 : x;
      }
      uint16_t* dst = g.vt + ((long long)head * D + c + lane) * g.Rp + row0;  // row0 % 32 == 0, Rp % 8 == 0
      if (row0 + 32 <= R) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          reinterpret_cast<uint4*>(dst)[q] = make_uint4(col[4 * q], col[4 * q + 1], col[4 * q + 2], col[4 * q + 3]);
      } else {
#pragma unroll
        for (int r = 0; r < 32; ++r)
          if (row0 + r < R) dst[r] = uint16_t(r & 1 ? col[r >> 1] >> 16 : col[r >> 1]);
      }
    }
    return;
  }
  if (row >= R) return;
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < D; ++c) ss = fmaf(val(c), val(c), ss);
  const float rstd = rsqrtf(ss / float(D) + g.qk_eps);
  const float* wn = which == 0 ? g.q_norm : g.k_norm;
  const int tw = g.rope_split ? 3 * D / 8 : D / 2;
  const float* cs = row < g.L ? g.txt_cos + (long long)row * tw : g.img_cos + (long long)(row - g.L) * tw;
  const float* sn = row < g.L ? g.txt_sin + (long long)row * tw : g.img_sin + (long long)(row - g.L) * tw;
  uint16_t* dst = (which == 0 ? g.q : g.k) + ((long long)head * R + row) * D;
  auto normed = [&](int c) { return wn ? val(c) * rstd * __ldg(wn + c) : val(c) * rstd; };
  if (!g.rope_split) {
    const bool whole = on_32(cs) && on_32(sn);  // the lanes are on different rows: fewer, wider accesses
#pragma unroll
    for (int c = 0; c < D; c += 16) {
      float cc[8], ss8[8];
      ld_global_8(cc, cs + c / 2, whole);
      ld_global_8(ss8, sn + c / 2, whole);
      uint32_t u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = normed(c + 2 * e), y = normed(c + 2 * e + 1);
        u[e] = pack_bf16x2(x * cc[e] - y * ss8[e], x * ss8[e] + y * cc[e]);
      }
      st_global_256(dst + c, u);
    }
  } else {
    constexpr int hr = 3 * D / 8;  // values i and i + hr by angle i; the last quarter only normed
#pragma unroll
    for (int c = 0; c < hr; c += 8) {
      float x[8], y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p = normed(c + e), q = normed(c + hr + e), t = __ldg(cs + c + e), s = __ldg(sn + c + e);
        x[e] = p * t - q * s;
        y[e] = p * s + q * t;
      }
      *reinterpret_cast<uint4*>(dst + c) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                      pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      *reinterpret_cast<uint4*>(dst + c + hr) = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                                                           pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
    }
#pragma unroll
    for (int c = 2 * hr; c < D; c += 8)
      *reinterpret_cast<uint4*>(dst + c) =
          make_uint4(pack_bf16x2(normed(c), normed(c + 1)), pack_bf16x2(normed(c + 2), normed(c + 3)),
                     pack_bf16x2(normed(c + 4), normed(c + 5)), pack_bf16x2(normed(c + 6), normed(c + 7)));
  }
}

// EPI: kEpiStoreF32 / kEpiStoreBF16 store the products; kEpiSwiGLU takes pairs of columns through SwiGLU,
// kEpiGated adds gate * product to the residual rows, kEpiQKV prepares queries, keys and values: a block's
// linears, with bn = 256, whole tiles of columns, and `ep` holding what their epilogues need.
struct NoParams {};
template <int EPI>
using EpiParams = typename std::conditional<EPI == kEpiQKV || EPI == kEpiGated, GemmParams, NoParams>::type;

template <int FMT, int EPI, bool SWAP>
__global__ void __launch_bounds__(kPairThreads, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
                    const __grid_constant__ CUtensorMap tmSP, const __grid_constant__ CUtensorMap tmSQ,
                    const Fp4Params p, const __grid_constant__ EpiParams<EPI> ep) {
  using T = typename std::conditional<EPI == kEpiStoreF32, float, __nv_bfloat16>::type;
  using SC = Scales<FMT>;
  const int S = p.stages, bn = p.bn;
  const uint32_t qBytes = uint32_t(bn) * 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sP = smem;
  uint8_t* sQ = sP + S * kTileBytes;
  uint8_t* sSP = sQ + S * qBytes;
  uint8_t* sSQ = sSP + S * SC::kBytes;
  // per epilogue warp: 64 column factors, or (QKV) 128 of them and then 4 KB to transpose values in
  uint8_t* sC = sSQ + S * 2 * SC::kBytes;
  constexpr int kScratch = EPI == kEpiQKV ? 4096 : 256;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sC + kEpiWarps * kScratch);
  uint64_t *full = bars, *empty = bars + S, *tfull = bars + 2 * S, *tempty = tfull + 2, *drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x >> 5, lane = lane_id();
  const uint32_t rank = cluster_ctarank();
  const int unit = int(blockIdx.x >> 1), units = int(gridDim.x >> 1);
  const int rowsP = SWAP ? p.N : p.M, rowsQ = SWAP ? p.M : p.N;
  const int num_p = (rowsP + 255) / 256, num_q = (rowsQ + bn - 1) / bn, tiles = num_p * num_q;
  const int KB = (p.K + kStageK - 1) / kStageK;
  const bool overlap = bn == 256;
  const uint32_t acc1 = overlap ? kOverlapAt : bn;
  auto tile_pq = [&](int tile, int& pb, int& qb) {
    pb = p.n_fast ? tile / num_q : tile % num_p;
    qb = p.n_fast ? tile % num_q : tile / num_p;
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(smem_u32(&tfull[a]), 1);
      mbar_init(smem_u32(&tempty[a]), 2 * 32 * kEpiWarps);  // both CTAs' epilogue threads
    }
    mbar_init(smem_u32(drain), 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmP);
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmSP);
    tma_prefetch_desc(&tmSQ);
  }
  __syncthreads();
  cluster_barrier();  // barriers of both CTAs are up
  const uint32_t full0 = mapa_shared(smem_u32(&full[0]), 0);  // both CTAs' copies count on the first's barriers
  auto load_p = [&](int stage, int kb, int pb) {
    const uint32_t fb = full0 + uint32_t(stage) * 8u;
    tma_load_2d_pair(smem_u32(sP + stage * kTileBytes), &tmP, fb, kb * 128, pb * 256 + int(rank) * 128);
    tma_load_3d_pair(smem_u32(sSP + stage * SC::kBytes), &tmSP, fb, 0, kb * SC::kGroups, pb * 2 + int(rank));
  };
  auto load_q = [&](int stage, int kb, int qb) {
    const uint32_t fb = full0 + uint32_t(stage) * 8u;
    tma_load_2d_pair(smem_u32(sQ + stage * qBytes), &tmQ, fb, kb * 128, qb * bn + int(rank) * (bn / 2));
    tma_load_3d_pair(smem_u32(sSQ + stage * 2 * SC::kBytes), &tmSQ, fb, 0, kb * SC::kGroups, (qb * bn) >> 7);
  };
  auto expect = [&](int stage) {
    if (rank == 0) mbar_arrive_expect_tx(smem_u32(&full[stage]), 2 * pair_stage_bytes<FMT>(bn));
  };
  // B's part of the first stages does not wait for the kernel that writes A
  const int ahead = p.early ? min(S, KB) : 0;
  if (warp == 0 && ahead > 0 && elect_one()) {
    int pb, qb;
    tile_pq(unit, pb, qb);
    for (int s = 0; s < ahead; ++s) {
      expect(s);
      if constexpr (SWAP) load_p(s, s, pb);
      else load_q(s, s, qb);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, parity = 0;
      bool ok = true;
      int done = 0;  // stages filled so far
      for (int tile = unit; tile < tiles && ok; tile += units) {
        int pb, qb;
        tile_pq(tile, pb, qb);
        for (int kb = 0; kb < KB; ++kb, ++done) {
          if (done < ahead) {
            if constexpr (SWAP) load_q(stage, kb, qb);
            else load_p(stage, kb, pb);
          } else {
            if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1, p.err, kErrTimeoutProducer)) { ok = false; break; }
            expect(stage);
            load_p(stage, kb, pb);
            load_q(stage, kb, qb);
          }
          issued |= 1u << stage;
          parity = (parity & ~(1u << stage)) | (phase << stage);
          if (++stage == S) { stage = 0; phase ^= 1; }
        }
      }
      // Every copy has landed before the CTAs leave: the first CTA's barriers count both CTAs' copies, but not those
      // that one of them issued after the other gave up
      if (aborted(p.err)) outlast_copies();
      else if (rank == 0)
        for (int s = 0; s < S; ++s)
          if (issued & (1u << s)) mbar_drain(smem_u32(&full[s]), (parity >> s) & 1u, p.err);
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int it = 0;
      for (int tile = unit; tile < tiles && ok; tile += units, ++it) {
        int pb, qb;
        tile_pq(tile, pb, qb);
        // this accumulator is free: the tile before last was drained (overlap: the last one's shared
        // columns are, and it drained the tile before it first)
        const int prev = overlap ? it - 1 : it - 2;
        if (prev >= 0 &&
            !mbar_wait_cluster(smem_u32(&tempty[prev & 1]), uint32_t(prev >> 1) & 1u, p.err, kErrTimeoutMma))
          break;
        tc_fence_after();
        const uint32_t d = tmem + ((it & 1) ? acc1 : 0);
        // Q rows may start in the middle of a band of 128: two columns per 64 rows
        const uint32_t sfp = tmem + kSfCol, sfq = sfp + SC::kGroups * 4, sub = uint32_t((qb * bn) & 127) >> 5;
        for (int kb = 0; kb < KB; ++kb) {
          if (!mbar_wait(smem_u32(&full[stage]), phase, p.err, kErrTimeoutMma)) { ok = false; break; }
          tc_fence_after();
          const int steps = stage_steps(p.K, kb);
          const uint64_t dp = scale_chunk_desc(smem_u32(sSP + stage * SC::kBytes));
          const uint64_t dq = scale_chunk_desc(smem_u32(sSQ + stage * 2 * SC::kBytes));
          const uint64_t pd = sw128_desc(smem_u32(sP + stage * kTileBytes));
          const uint64_t qd = sw128_desc(smem_u32(sQ + stage * qBytes));
#pragma unroll
          for (int g = 0; g < SC::kGroups; ++g) {
            tmem_cp_scales<true>(sfp + 4 * g, dp + uint64_t(32 * g));
            tmem_cp_scales<true>(sfq + 8 * g, dq + uint64_t(32 * g));
            if (bn > 128) tmem_cp_scales<true>(sfq + 8 * g + 4, dq + uint64_t(32 * (SC::kGroups + g)));
          }
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk < steps) {
              const int g = SC::kNv ? kk : kk >> 1;
              umma_fp4<SC::kNv, true>(d, pd + uint64_t(2 * kk), qd + uint64_t(2 * kk),
                                      idesc_fp4(SC::kNv, 256, bn, SC::kNv ? 0 : (kk & 1) * 2), sfp + 4 * g,
                                      sfq + 8 * g + sub, kb != 0 || kk != 0);
            }
          }
          umma_commit_pair_both(smem_u32(&empty[stage]));
          if (++stage == S) { stage = 0; phase ^= 1; }
        }
        if (!ok) break;
        umma_commit_pair_both(smem_u32(&tfull[it & 1]));
      }
      umma_commit_pair(smem_u32(drain));
      mbar_drain(smem_u32(drain), 0, p.err);
    }
  } else if constexpr (EPI == kEpiQKV) {
    // two warps to each quadrant of 32 lanes, 128 columns each, all of them in registers at once: the
    // accumulator is free as soon as every warp has loaded its part
    const int quad = warp & 3, half = (warp - 2) >> 2;
    uint8_t* scratch = sC + (warp - 2) * kScratch;
    float* cf = reinterpret_cast<float*>(scratch);
    const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[0]), 0);
    int it = 0;
    for (int tile = unit; tile < tiles; tile += units, ++it) {
      int pb, qb;
      tile_pq(tile, pb, qb);
      const int acc = it & 1, row0 = pb * 256 + int(rank) * 128 + quad * 32, row = row0 + lane;
      const int n0 = qb * 256 + half * 128;
      float rp = 1.f;
      if constexpr (SC::kNv) {
        rp = row < rowsP ? __ldg(p.a_scale + row) : 0.f;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 4; ++c) cf[c * 32 + lane] = __ldg(p.b_scale + n0 + c * 32 + lane);
        __syncwarp();
      }
      if (!mbar_wait_warp(smem_u32(&tfull[acc]), uint32_t(it >> 1) & 1u, p.err, kErrTimeoutEpilogue)) break;
      tc_fence_after();
      const uint32_t taddr = tmem + (uint32_t(quad * 32) << 16) + (acc ? acc1 : 0) + half * 128;
      uint32_t w[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(taddr + c * 32, w[c]);
      tmem_ld_wait();
      tc_fence_before();
      mbar_arrive_cluster(tempty0 + uint32_t(acc) * 8u);
      if (row0 >= rowsP) continue;
      if constexpr (SC::kNv) {
        const float first = factor_first(rp), back = factor_back(rp);
        const uint64_t rp2 = f2_pack(first, first);
#pragma unroll
        for (int c = 0; c < 128; c += 4) scale4(w[c >> 5] + (c & 31), rp2, *reinterpret_cast<const float4*>(cf + c));
        if (__any_sync(0xffffffffu, back != 1.f)) put_back<128>(w[0], back);
      }
      if (ep.head_dim == 128) {
        qkv_store<128>(ep, w[0], row0, lane, n0, scratch);
      } else {
        qkv_store<64>(ep, w[0], row0, lane, n0, scratch);
        qkv_store<64>(ep, w[2], row0, lane, n0 + 64, scratch);
      }
      __syncwarp();
    }
  } else {
    // two warps to each quadrant of 32 lanes, taking its 64-column groups in turn
    const int quad = warp & 3, half = (warp - 2) >> 2, groups = bn / 64;
    float* cf = reinterpret_cast<float*>(sC + (warp - 2) * kScratch);
    const uint32_t tempty0 = mapa_shared(smem_u32(&tempty[0]), 0);
    const float* p_scale = SWAP ? p.b_scale : p.a_scale;
    const float* q_scale = SWAP ? p.a_scale : p.b_scale;
    int it = 0;
    for (int tile = unit; tile < tiles; tile += units, ++it) {
      int pb, qb;
      tile_pq(tile, pb, qb);
      const int acc = it & 1;
      const int row0 = pb * 256 + int(rank) * 128 + quad * 32, row = row0 + lane;  // P rows of this warp
      float rp = 1.f, f0 = 1.f, f1 = 1.f;
      // 64 columns at a time, overlapped ones first; a group's factors are fetched a group ahead
      auto group_at = [&](int j) { return overlap && acc == 0 ? groups - 1 - j : j; };
      auto fetch = [&](int j) {
        const int q = qb * bn + group_at(j) * 64 + lane;
        f0 = q < rowsQ ? __ldg(q_scale + q) : 0.f;
        f1 = q + 32 < rowsQ ? __ldg(q_scale + q + 32) : 0.f;
      };
      if constexpr (SC::kNv) {
        rp = row < rowsP ? __ldg(p_scale + row) : 0.f;
        fetch(half);
      }
      if (!mbar_wait_warp(smem_u32(&tfull[acc]), uint32_t(it >> 1) & 1u, p.err, kErrTimeoutEpilogue)) break;
      tc_fence_after();
      const uint32_t taddr = tmem + (uint32_t(quad * 32) << 16) + (acc ? acc1 : 0);
      // what this warp holds back from the next tile: nothing of the overlapped columns (group 0), or nothing at all.
      // Its arrival also stands for its reads of the tile before, which end ahead of the fence
      if (overlap && half == 1) {
        tc_fence_before();
        mbar_arrive_cluster(tempty0 + uint32_t(acc) * 8u);
      }
#pragma unroll 1
      for (int j = half; j < groups; j += 2) {
        const int g = group_at(j), q0 = qb * bn + g * 64;
        uint32_t w[2][32];
        tmem_ld32(taddr + g * 64, w[0]);
        tmem_ld32(taddr + g * 64 + 32, w[1]);
        tmem_ld_wait();
        if (overlap ? j == 0 : j + 2 >= groups) {
          tc_fence_before();
          mbar_arrive_cluster(tempty0 + uint32_t(acc) * 8u);
        }
        if constexpr (SC::kNv) {
          __syncwarp();
          cf[lane] = f0;
          cf[lane + 32] = f1;
          if (j + 2 < groups) fetch(j + 2);
          __syncwarp();
        }
        if (q0 >= rowsQ || row0 >= rowsP) continue;
        if constexpr (SC::kNv) {
          const float first = factor_first(rp), back = factor_back(rp);
          const uint64_t rp2 = f2_pack(first, first);
#pragma unroll
          for (int c = 0; c < 64; c += 4) {
            const float4 f = *reinterpret_cast<const float4*>(cf + c);
            scale4(w[c >> 5] + (c & 31), rp2, f);
          }
          if (__any_sync(0xffffffffu, back != 1.f)) put_back<64>(w[0], back);
        }
        auto val = [&](int c) { return __uint_as_float(w[c >> 5][c & 31]); };
        if constexpr (SWAP) {
          // out[q][p]: the lanes hold 32 consecutive values of each output row
          if (row < rowsP) {
            T* o = static_cast<T*>(p.out) + (long long)q0 * p.ldo + row;
            if (q0 + 64 <= rowsQ) {
#pragma unroll
              for (int c = 0; c < 64; ++c) o[c * p.ldo] = T(val(c));
            } else {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (q0 + c < rowsQ) o[c * p.ldo] = T(val(c));
            }
          }
        } else if constexpr (EPI == kEpiSwiGLU) {
          // out[p][q / 2] = silu(even column) * odd column (whole 64-column groups: N is a multiple of 256)
          if (row < rowsP) {
            T* o = static_cast<T*>(p.out) + (long long)row * p.ldo + q0 / 2;
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
              uint32_t u[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                u[e] = pack_bf16x2(silu_bf16(val(c + 4 * e)) * val(c + 4 * e + 1),
                                   silu_bf16(val(c + 4 * e + 2)) * val(c + 4 * e + 3));
              st_global_256(o + c / 2, u);
            }
          }
        } else if constexpr (EPI == kEpiGated) {
          // x[p][q] += gate[map[p]][q] * product (the gizai:dit reference's gatedInto). A lane per row: 32 pieces
          // of 32 bytes in 32 lines per access, which hold 4224 x 3072 x 3072 at 39 us (15 by its bytes)
          if (row < rowsP) {
            float* x = (row < ep.L ? ep.txt + (long long)row * ep.N : ep.img + (long long)(row - ep.L) * ep.N) + q0;
            const float* gate = ep.gate + (ep.map ? __ldg(ep.map + row) : 0) * ep.gate_stride + q0;
            const bool wx = on_32(x), wg = on_32(gate);
#pragma unroll
            for (int h = 0; h < 64; h += 32) {
              float xv[4][8], gv[4][8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                ld_global_8(xv[e], x + h + 8 * e, wx);
                ld_global_8(gv[e], gate + h + 8 * e, wg);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t u[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) u[k] = __float_as_uint(fmaf(gv[e][k], val(h + 8 * e + k), xv[e][k]));
                if (wx) {
                  st_global_256(x + h + 8 * e, u);
                } else {
                  reinterpret_cast<uint4*>(x + h + 8 * e)[0] = make_uint4(u[0], u[1], u[2], u[3]);
                  reinterpret_cast<uint4*>(x + h + 8 * e)[1] = make_uint4(u[4], u[5], u[6], u[7]);
                }
              }
            }
          }
        } else if (row < rowsP) {
          // out[p][q]: a lane holds 64 consecutive values of its row, stored 32 bytes at a time
          T* o = static_cast<T*>(p.out) + (long long)row * p.ldo + q0;
          constexpr int kPer = 32 / sizeof(T);
#pragma unroll
          for (int c = 0; c < 64; c += kPer) {
            if (q0 + c + kPer <= rowsQ) {
              uint32_t u[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                u[e] = sizeof(T) == 2 ? pack_bf16x2(val(c + 2 * e), val(c + 2 * e + 1)) : w[(c + e) >> 5][(c + e) & 31];
              st_global_256(o + c, u);
            } else {
#pragma unroll
              for (int e = 0; e < kPer; ++e)
                if (q0 + c + e < rowsQ) o[c + e] = T(val(c + e));
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_barrier();  // no CTA frees or leaves what the other may still use
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ---------------------------------------------------------------------------------------------
// split kernel: D [128 rows of B, bn rows of A], so that few rows of A still fill the MMA's 128 lanes
// ---------------------------------------------------------------------------------------------
constexpr int kSplitThreads = 192;
constexpr uint32_t kSplitMinSmem = 116 * 1024;
constexpr int kSplitMaxStages = 12;
constexpr uint32_t kSplitFixed = 1024 + 2 * 128 * 4 + 8 * (2 * kSplitMaxStages + 1) + 16;
__host__ __device__ constexpr uint32_t split_stage_bytes(int bn, uint32_t sf) { return kTileBytes + uint32_t(bn) * 128 + 2 * sf; }

template <int FMT, typename T>
__global__ void __launch_bounds__(kSplitThreads, 1)
    fp4_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
                     const Fp4Params p) {
  using SC = Scales<FMT>;
  const int S = p.stages, bn = p.bn;
  const uint32_t aBytes = uint32_t(bn) * 128;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* sFa = reinterpret_cast<float*>(smem);  // row factors of the tile's A and B rows (1 KB)
  float* sFb = sFa + 128;
  uint8_t* sB = smem + 1024;               // 128 rows of B per stage (the MMA's A side)
  uint8_t* sA = sB + S * kTileBytes;       // bn rows of A (multiples of 16: 1024-byte swizzle atoms stay whole)
  uint8_t* sSB = sA + S * aBytes;
  uint8_t* sSA = sSB + S * SC::kBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sSA + S * SC::kBytes);
  uint64_t *full = bars, *empty = bars + S, *tfull = bars + 2 * S;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);

  const int warp = threadIdx.x >> 5, lane = lane_id();
  const int parts = int(cluster_nctarank()), part = int(cluster_ctarank());
  const int n0 = int(blockIdx.x / parts) * 128, m0 = int(blockIdx.y) * bn;
  const int KB = (p.K + kStageK - 1) / kStageK;
  const int k0 = int((long long)KB * part / parts), k1 = int((long long)KB * (part + 1) / parts);
  const uint32_t cols = bn <= 32 ? 64 : (bn <= 64 ? 128 : 256);  // bn accumulator columns, then the scales
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(tfull), 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmSA);
    tma_prefetch_desc(&tmSB);
  }
  auto load_b = [&](int stage, int kb) {
    const uint32_t fb = smem_u32(&full[stage]);
    mbar_arrive_expect_tx(fb, kTileBytes + aBytes + 2 * SC::kBytes);
    tma_load_2d(smem_u32(sB + stage * kTileBytes), &tmB, fb, kb * 128, n0);
    tma_load_3d(smem_u32(sSB + stage * SC::kBytes), &tmSB, fb, 0, kb * SC::kGroups, n0 >> 7);
  };
  // B's part of the first stages does not wait for the kernel that writes A
  const int ahead = p.early ? min(S, k1 - k0) : 0;
  if (threadIdx.x == 0)
    for (int s = 0; s < ahead; ++s) load_b(s, k0 + s);
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  bool far = false;  // one of the tile's A factors goes first as another (factor_first)

  if (warp == 0) {
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0, issued = 0, parity = 0;
      for (int kb = k0; kb < k1; ++kb) {
        if (kb - k0 >= ahead) {
          if (!mbar_wait(smem_u32(&empty[stage]), phase ^ 1, p.err, kErrTimeoutProducer)) break;
          load_b(stage, kb);
        }
        const uint32_t fb = smem_u32(&full[stage]);
        tma_load_2d(smem_u32(sA + stage * aBytes), &tmA, fb, kb * 128, m0);
        tma_load_3d(smem_u32(sSA + stage * SC::kBytes), &tmSA, fb, 0, kb * SC::kGroups, m0 >> 7);
        issued |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == S) { stage = 0; phase ^= 1; }
      }
      for (int s = 0; s < S; ++s)  // every copy has landed before the CTA leaves
        if (issued & (1u << s)) mbar_drain(smem_u32(&full[s]), (parity >> s) & 1u, p.err);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      const uint32_t sfb = tmem + bn, sfa = sfb + SC::kGroups * 4;  // B's scales (MMA A side), A's scales
      for (int kb = k0; kb < k1; ++kb) {
        if (!mbar_wait(smem_u32(&full[stage]), phase, p.err, kErrTimeoutMma)) break;
        tc_fence_after();
        const int steps = stage_steps(p.K, kb);
        const uint64_t db = scale_chunk_desc(smem_u32(sSB + stage * SC::kBytes));
        const uint64_t da = scale_chunk_desc(smem_u32(sSA + stage * SC::kBytes));
        const uint64_t bd = sw128_desc(smem_u32(sB + stage * kTileBytes));
        const uint64_t ad = sw128_desc(smem_u32(sA + stage * aBytes));
#pragma unroll
        for (int g = 0; g < SC::kGroups; ++g) {
          tmem_cp_scales<false>(sfb + 4 * g, db + uint64_t(32 * g));
          tmem_cp_scales<false>(sfa + 4 * g, da + uint64_t(32 * g));
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (kk < steps) {
            const int g = SC::kNv ? kk : kk >> 1;
            umma_fp4<SC::kNv, false>(tmem, bd + uint64_t(2 * kk), ad + uint64_t(2 * kk),
                                     idesc_fp4(SC::kNv, 128, bn, SC::kNv ? 0 : (kk & 1) * 2), sfb + 4 * g,
                                     sfa + 4 * g, kb != k0 || kk != 0);
          }
        }
        umma_commit(smem_u32(&empty[stage]));
        if (++stage == S) { stage = 0; phase ^= 1; }
      }
      umma_commit(smem_u32(tfull));
      mbar_drain(smem_u32(tfull), 0, p.err);
    }
  } else {
    if constexpr (SC::kNv) {
      const int i = int(threadIdx.x) - 64;
      const float ra = i < bn && m0 + i < p.M ? __ldg(p.a_scale + m0 + i) : 0.f;
      far = factor_back(ra) != 1.f;
      sFa[i] = factor_first(ra);
      sFb[i] = n0 + i < p.N ? __ldg(p.b_scale + n0 + i) : 0.f;
    }
    (void)mbar_wait_warp(smem_u32(tfull), 0, p.err, kErrTimeoutEpilogue);
    tc_fence_after();
  }
  // Epilogue. A lone CTA stores its tile; the CTAs of a cluster put their partial tiles into shared
  // memory ([column of A][128 rows of B] fp32, the pipeline's memory), and each adds up its share of the
  // columns, part by part in order.
  const int quad = warp & 3;
  const uint32_t taddr = tmem + (uint32_t(quad * 32) << 16);
  const int n = n0 + quad * 32 + lane;
  T* out = static_cast<T*>(p.out);
  float* tile = reinterpret_cast<float*>(sB);
  if constexpr (SC::kNv) far = __syncthreads_or(far);
  else __syncthreads();
  tc_fence_after();
  const int live = min(bn, p.M - m0);
  auto drain = [&](auto back) {  // back: A factors that were taken smaller or larger are put back (a loop of its own)
    const float rb = SC::kNv ? sFb[quad * 32 + lane] : 1.f;
    T* o = out + (long long)m0 * p.ldo + n;
    for (int c = 0; c < live; c += 16, o += 16 * p.ldo) {
      uint32_t w[16];
      tmem_ld16(taddr + c, w);
      tmem_ld_wait();
      if (parts > 1) {
#pragma unroll
        for (int e = 0; e < 16; ++e) tile[(c + e) * 128 + quad * 32 + lane] = __uint_as_float(w[e]);
        continue;
      }
      // every value first, then the stores: a store between them would hold back the next factor's load
      T v[16];
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const float4 f = SC::kNv ? *reinterpret_cast<const float4*>(sFa + c + e) : make_float4(1.f, 1.f, 1.f, 1.f);
        const float* ff = &f.x;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x = __uint_as_float(w[e + k]);
          float y = SC::kNv ? x * ff[k] * rb : x;
          if constexpr (back.value)
            if (c + e + k < live) y *= factor_back(__ldg(p.a_scale + m0 + c + e + k));
          v[e + k] = T(y);
        }
      }
      if (n < p.N) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (c + e < live) o[e * p.ldo] = v[e];
      }
    }
  };
  if (warp >= 2) {
    if (SC::kNv && far) drain(std::true_type{});
    else drain(std::false_type{});
  }
  if (parts > 1) {
    cluster_barrier();
    const uint32_t base = smem_u32(tile);
    // four rows of B per thread, 32 threads to a column; all parts of two columns in flight together
    constexpr int kMaxParts = 8;
    const int step = parts * kSplitThreads;
    const bool whole = n0 + 128 <= p.N && p.ldo % 4 == 0 && reinterpret_cast<uintptr_t>(out) % (4 * sizeof(T)) == 0;
    for (int i0 = part * kSplitThreads + int(threadIdx.x); i0 < live * 32; i0 += 2 * step) {
      float4 v[2][kMaxParts];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int q = 0; q < kMaxParts; ++q)
          if (q < parts && i0 + u * step < live * 32)
            v[u][q] = ld_shared_cluster_v4(mapa_shared(base + uint32_t(i0 + u * step) * 16u, uint32_t(q)));
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = i0 + u * step;
        if (i >= live * 32) continue;
        float4 s = v[u][0];
#pragma unroll
        for (int q = 1; q < kMaxParts; ++q)
          if (q < parts) {
            s.x += v[u][q].x;
            s.y += v[u][q].y;
            s.z += v[u][q].z;
            s.w += v[u][q].w;
          }
        const int c = i >> 5, r4 = (i & 31) * 4;
        if constexpr (SC::kNv) {
          const float ra = sFa[c];
          const float4 f = *reinterpret_cast<const float4*>(sFb + r4);
          s = make_float4(s.x * ra * f.x, s.y * ra * f.y, s.z * ra * f.z, s.w * ra * f.w);
          if (far) {
            const float back = factor_back(__ldg(p.a_scale + m0 + c));
            s = make_float4(s.x * back, s.y * back, s.z * back, s.w * back);
          }
        }
        T* o = out + (long long)(m0 + c) * p.ldo + n0 + r4;
        if (whole) {
          if constexpr (sizeof(T) == 2)
            *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
          else
            *reinterpret_cast<float4*>(o) = s;
        } else {
          const float* sv = &s.x;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n0 + r4 + e < p.N) o[e] = T(sv[e]);
        }
      }
    }
    cluster_barrier();  // no CTA leaves while another reads its shared memory
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, cols);
}

// ---------------------------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------------------------
// All of an SM's shared memory for `kern`; asked for once per device (a bit of `ready`), since a call here
// takes microseconds and the library's table of kernels is searched under a lock.
bool allow_smem(const void* kern, std::atomic<uint64_t>& ready) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (ready.load(std::memory_order_acquire) & bit) return true;
  if (!smem_attr_once(kern, 227 * 1024)) return false;
  ready.fetch_or(bit, std::memory_order_release);
  return true;
}

// CTA pairs that are resident at once, asked for once per kernel and device (`cached`, by device).
int resident_pairs(const void* kern, unsigned smem, std::atomic<int>* cached) {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return num_sms() / 2;
  if ((n = cached[dev].load(std::memory_order_relaxed)) > 0) return n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(num_sms() & ~1));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 2;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n <= 0) {
    cudaGetLastError();
    n = num_sms() / 2;
  }
  n = std::min(n, num_sms() / 2);
  cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Scale tiles as a 3-D map: chunks of 512 bytes (as 128 words) x groups of four blocks x bands of 128 rows; box
// = one chunk x box_groups x box_bands.
bool make_tmap_scales(CUtensorMap* m, const void* base, long long groups, long long bands, int box_groups, int box_bands) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {128, cuuint64_t(groups), cuuint64_t(bands)};
  cuuint64_t strides[2] = {512, cuuint64_t(groups) * 512};
  cuuint32_t box[3] = {128, cuuint32_t(box_groups), cuuint32_t(box_bands)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool tmap_codes(CUtensorMap* m, const uint8_t* codes, int rows, int K, int box_rows) {
  return make_tmap_2d(m, codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, fp4_code_row_bytes(K), rows, fp4_code_row_bytes(K), 128,
                      box_rows, true);
}
bool tmap_sf(CUtensorMap* m, const dit_fp4_matrix& x, int box_groups, int box_bands) {
  return make_tmap_scales(m, x.scales, fp4_groups(x.format, x.cols), (x.rows + 127) / 128, box_groups, box_bands);
}

template <int FMT, int EPI, bool SWAP>
int launch_pair(const dit_fp4_matrix& a, const dit_fp4_matrix& b, Fp4Params p, const EpiParams<EPI>& g, int bn,
                cudaStream_t st) {
  const dit_fp4_matrix &P = SWAP ? b : a, &Q = SWAP ? a : b;
  CUtensorMap mp, mq, msp, msq;
  constexpr int G = Scales<FMT>::kGroups;
  p.bn = bn;
  const uint32_t fixed = kPairFixed + (EPI == kEpiQKV ? kEpiWarps * (4096 - 256) : 0);
  p.stages = std::min(kMaxStages, int((227 * 1024 - fixed) / pair_stage_bytes<FMT>(bn)));
  const uint32_t smem = fixed + uint32_t(p.stages) * pair_stage_bytes<FMT>(bn);
  if (!tmap_codes(&mp, P.codes, P.rows, p.K, 128) || !tmap_codes(&mq, Q.codes, Q.rows, p.K, bn / 2) ||
      !tmap_sf(&msp, P, G, 1) || !tmap_sf(&msq, Q, G, 2))
    return DIT_ECUDA;
  p.n_fast = P.rows > Q.rows;  // consecutive tiles share the smaller operand's rows, which stay in L2
  auto kern = fp4_pair_kernel<FMT, EPI, SWAP>;
  static std::atomic<uint64_t> ready{0};
  if (!allow_smem(reinterpret_cast<const void*>(kern), ready)) return DIT_ECUDA;
  const long long tiles = (long long)((P.rows + 255) / 256) * ((Q.rows + bn - 1) / bn);
  if (tiles > 0x7fffffffLL - num_sms()) return DIT_EUNSUPPORTED;
  static std::atomic<int> pairs[64];  // one smem size counts for all: more than half an SM's, so a CTA per SM
  const int units = int(std::min<long long>(tiles, resident_pairs(reinterpret_cast<const void*>(kern), smem, pairs)));
  const cudaError_t e = launch_pdl(kern, dim3(unsigned(2 * units)), dim3(kPairThreads), smem, st, 2, mp, mq, msp, msq, p, g);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? DIT_OK : DIT_ECUDA;
}

template <int FMT, typename T>
int launch_split(const dit_fp4_matrix& a, const dit_fp4_matrix& b, Fp4Params p, int bn, int parts, cudaStream_t st) {
  constexpr int G = Scales<FMT>::kGroups;
  p.bn = bn;
  const long long nt = (p.N + 127) / 128, mt = (p.M + bn - 1) / bn;
  if (nt * parts > 0x7fffffffLL || mt > kFp4MaxGridY) return DIT_EUNSUPPORTED;
  const int KB = (p.K + kStageK - 1) / kStageK;
  const uint32_t sb = split_stage_bytes(bn, Scales<FMT>::kBytes);
  // A cluster's CTA asks for more than half of an SM's shared memory, as every kernel here that allocates
  // tensor memory and waits for another CTA: no two of them share an SM, so none waits for tensor memory
  // that another cluster holds. (The half also covers the partial tile, at most 64 KB.) A lone CTA waits
  // for nobody: where there are more than SMs, two share one.
  const uint32_t most = parts == 1 && nt * mt > num_sms() ? 113 * 1024 : 227 * 1024;
  p.stages = std::min((KB + parts - 1) / parts, int((most - kSplitFixed) / sb));
  p.stages = std::max(1, std::min(p.stages, kSplitMaxStages));
  uint32_t smem = kSplitFixed + uint32_t(p.stages) * sb;
  if (parts > 1) smem = std::max(smem, kSplitMinSmem);
  CUtensorMap ma, mb, msa, msb;
  if (!tmap_codes(&ma, a.codes, a.rows, p.K, bn) || !tmap_codes(&mb, b.codes, b.rows, p.K, 128) || !tmap_sf(&msa, a, G, 1) ||
      !tmap_sf(&msb, b, G, 1))
    return DIT_ECUDA;
  auto kern = fp4_split_kernel<FMT, T>;
  static std::atomic<uint64_t> ready{0};
  if (!allow_smem(reinterpret_cast<const void*>(kern), ready)) return DIT_ECUDA;
  const cudaError_t e = launch_pdl(kern, dim3(unsigned(nt * parts), unsigned(mt)), dim3(kSplitThreads), smem, st, parts,
                                   ma, mb, msa, msb, p);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? DIT_OK : DIT_ECUDA;
}

template <int FMT, typename T>
int launch_product(const dit_fp4_matrix& a, const dit_fp4_matrix& b, const Fp4Params& p, cudaStream_t st) {
  const bool rows32 = reinterpret_cast<uintptr_t>(p.out) % 32 == 0 && (p.M == 1 || p.ldo * (long long)sizeof(T) % 32 == 0);
  const Fp4Choice c = fp4_choose(p.M, p.N, p.K, rows32, num_sms());
  if (c.parts > 0) return launch_split<FMT, T>(a, b, p, c.bn, c.parts, st);
  constexpr int kStore = sizeof(T) == 2 ? kEpiStoreBF16 : kEpiStoreF32;
  return c.swap ? launch_pair<FMT, kStore, true>(a, b, p, {}, c.bn, st) : launch_pair<FMT, kStore, false>(a, b, p, {}, c.bn, st);
}

template <int FMT>
int launch_block_linear(const dit_fp4_matrix& a, const dit_fp4_matrix& b, const Fp4Params& p, const GemmParams& g, int epi,
                        cudaStream_t st) {
  switch (epi) {
    case kEpiQKV: return launch_pair<FMT, kEpiQKV, false>(a, b, p, g, 256, st);
    case kEpiGated: return launch_pair<FMT, kEpiGated, false>(a, b, p, g, 256, st);
    case kEpiSwiGLU: return launch_pair<FMT, kEpiSwiGLU, false>(a, b, p, {}, 256, st);
    default: return DIT_EINVAL;
  }
}

Fp4Params product_params(const dit_fp4_matrix& a, const dit_fp4_matrix& b, void* out, long long ldo, int* err, bool b_early) {
  Fp4Params p{};
  p.M = a.rows;
  p.N = b.rows;
  p.K = a.cols;
  p.err = err;
  p.out = out;
  p.ldo = ldo;
  p.a_scale = a.row_scale;
  p.b_scale = b.row_scale;
  p.early = b_early;
  return p;
}

}  // namespace

int fp4_block_linear_launch(const dit_fp4_matrix& a, const dit_fp4_matrix& b, int epi, const GemmParams& g,
                            cudaStream_t st) {
  if (b.rows % 256 != 0 || (epi == kEpiQKV && g.head_dim != 64 && g.head_dim != 128)) return DIT_EUNSUPPORTED;
  const Fp4Params p = product_params(a, b, g.out, g.ldo, g.err, true);
  return a.format == DIT_FP4_NV ? launch_block_linear<DIT_FP4_NV>(a, b, p, g, epi, st)
                                : launch_block_linear<DIT_FP4_MX>(a, b, p, g, epi, st);
}

int fp4_matmul_launch(const dit_fp4_matrix& a, const dit_fp4_matrix& b, void* out, int type, long long ldo, int* err,
                      bool b_early, cudaStream_t st) {
  const Fp4Params p = product_params(a, b, out, ldo, err, b_early);
  if (a.format == DIT_FP4_NV)
    return type == DIT_BF16 ? launch_product<DIT_FP4_NV, __nv_bfloat16>(a, b, p, st)
                            : launch_product<DIT_FP4_NV, float>(a, b, p, st);
  return type == DIT_BF16 ? launch_product<DIT_FP4_MX, __nv_bfloat16>(a, b, p, st)
                          : launch_product<DIT_FP4_MX, float>(a, b, p, st);
}

}  // namespace dit
