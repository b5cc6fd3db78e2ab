// Attention over packed sequences on tcgen05 for sm_103a: many sequences of unlike length in one call, grouped key
// heads, per-row visible keys, capped scores and a distance bias; single rows over long key ranges.
//
// Mathematics. Segment s has the query rows [q_start[s], q_start[s + 1]) and the keys [k_start[s], k_start[s + 1]).
// Row i of a segment (of nq rows, nk keys) sees its keys j < c_i (all without `visible`):
//   x_ij = cap tanh(scale q_i.k_j / cap) - slope_h |i + nk - nq - j|       (either part left out where not given)
//   o_i = sum_j softmax_j(x_ij) v_j,    lse_i = ln sum_j exp(x_ij);    no key seen: o_i = 0, lse_i = -inf
// The softmax runs over key tiles with a running maximum and sum (klein article, section 4.3), in fp32 in log2 units;
// only the weights round to bf16 for the product with V, whose sum is fp32 in tensor memory.
//
// GB300 mapping. The query heads that share a key head stand side by side in one 128-row tile (row r G + g: query row
// r, head g of the G), so K and V are read once for all of them. K and V are rows of any stride: both come by TMA as
// [keys, d] boxes, and V enters its MMA as an MN-major operand, so nothing is transposed in memory. CTAs find their segment
// by a scan over q_start: no lengths on the host, and a captured graph serves other lengths. packed_kernel takes two tiles
// of a segment per CTA: warp 0 loads, warp 1 issues the MMAs, warps 2-9 and 10-17 turn the scores of the two tiles into
// weights, so that one tile's exponentials overlap the other's MMAs; a row's 128 keys of a tile are two threads' work, who
// exchange their maxima through shared memory (4224 rows of 24 heads of 128: 178 us with eight warps of whole rows, 162 so:
// 1350 TFLOP/s, the GPU at its power limit). packed_rows_kernel takes
// segments of few rows or short ones, two CTAs to an SM. Where there are too few tiles for the SMs the key range is split over CTAs
// (blockIdx.z) and a second kernel joins the parts in order.
// Masked places: weights of masked keys are zero, the rows of V behind the last key that any row of the CTA sees are
// zeroed in shared memory (they may be the next segment's, or anything), and a row whose result is not finite while
// its tile held keys that it does not see is summed again over its own keys, unless what it sees makes it so (mend_rows): NaN or
// infinity in a masked place never reaches it.
//
// Tensor memory (512 columns): [0, 128) S0, P0 over it: 32 columns at 0 for keys
// 0-63, 32 at 64 for keys 64-127   [128, 256) S1 / P1   [256, 256 + d) O0   [256 + d, 256 + 2 d) O1
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include "internal.h"
#include "ptx.cuh"
#include "tmap.h"

namespace dit {
namespace {

constexpr float kRescaleStep = 8.0f;  // log2 units: the running maximum moves only past this, so weights stay below 2^8
constexpr int kMaxSplits = 32;
constexpr int kPackedThreads = 64 + 32 * 16;  // loader, MMA issuer, sixteen softmax warps

// What a call's scores go through. kCapped also serves a bias without a cap; its error is a few 2^-24 of the cap, so caps of
// more than kWideLog2 log2 units (where that is 4e-5, what the sums of the products may be off by) go by kWide, whose
// error is relative to the score. (9 sequences of 811 to 1943 rows, 16 heads of 64 over 4: 246 us under a cap of 177, 257 under
// 178 and up; two of 2489 and 2829 rows, 24 heads of 128: 284 and 322; with a score past a quarter of its cap in every
// warp 431 and 506.)
enum Scores : int { kPlain = 0, kCapped = 1, kWide = 2 };
constexpr float kWideLog2 = 256.f, kFixedLog2 = 80.f;

struct PackedParams {
  dit_packed_attention a;
  int G, rpt;  // query heads per key head, query rows of a tile
  int splits, slots;  // CTAs along the keys; ring slots of the few-rows kernel
  float scale_log2;  // scale log2(e)
  float cap_in, cap_out;  // 2 scale log2(e) / cap and cap log2(e); cap_out = 0: no cap
  float cap_arg;  // scale / cap
  float* part_o;   // [split][q_rows][heads][d]
  float2* part_ml;  // [split][q_rows][heads]: running maximum (log2 units) and sum
  int* err;
};

template <int D>
struct PackedCfg {
  static constexpr uint32_t kTile = 128 * D * 2;  // 128 rows of q, k or v
  static constexpr uint32_t kAtom = 128 * 128;    // [128 rows x 64 bf16], 128-byte swizzled
  static constexpr int kKS = D == 128 ? 3 : 4, kVS = D == 128 ? 2 : 4;
  static constexpr int kBars = 2 + 2 * kKS + 2 * kVS + 8;
  // (768: what a base on 256 bytes can be off the tiles' 1024)
  static constexpr uint32_t kSmem = 768 + (2 + kKS + kVS) * kTile + kBars * 8 + 64 + 2 * 2 * 128 * 4;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static_assert(kSmem > 114 * 1024, "one CTA per SM: each takes all of tensor memory");
};

// V as the MN-major operand of O += P V: 64-value rows of a key (128 bytes), swizzled; the next eight keys 1024 bytes on
// (stride byte offset), the next 64 values of d a box of keys on (leading byte offset).
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr, uint32_t box) {
  return uint64_t((saddr & 0x3FFFFu) >> 4) | (uint64_t(box >> 4) << 16) | (uint64_t(1024 >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// cap log2(e) tanh(scale s / cap) as c - 2 c / (1 + 2^(2 scale log2(e) s / cap)): absolute error a few 2^-24 of c
__device__ __forceinline__ float capped(float s, float cap_in, float cap_out) {
  return fmaf(-2.f * cap_out, rcp_approx(1.f + ex2_approx(s * cap_in)), cap_out);
}

// The same for any cap, with an error relative to the score: up to t = scale s / cap = 1/2 the odd series of tanh around 0,
// x (1 - t^2 / 3 + 2 t^4 / 15 - ... + 21844 t^12 / 6081075) with x the uncapped score (the next term is below 2^-23 of it),
// above it c (1 - 2 / (1 + e^2|t|)) with the sign of s, at least 0.46 c. (With c - 2 c / (1 + e^2t) throughout, scores of a few
// units were off by 0.02 under a cap of 1e5 and by 1.7 under 1e7.)
__device__ __forceinline__ float capped_wide(float s, const PackedParams& p) {
  const float t = s * p.cap_arg, z = t * t;
  float f = fmaf(z, 21844.f / 6081075.f, -1382.f / 155925.f);
  f = fmaf(z, f, 62.f / 2835.f);
  f = fmaf(z, f, -17.f / 315.f);
  f = fmaf(z, f, 2.f / 15.f);
  f = fmaf(z, f, -1.f / 3.f);
  f = fmaf(z, f, 1.f);
  const float e = ex2_approx(-fabsf(s * p.cap_in));
  const float far = p.cap_out * fmaf(-2.f * e, rcp_approx(1.f + e), 1.f);
  return fabsf(t) < 0.5f ? s * p.scale_log2 * f : copysignf(far, s);
}

// Two capped scores at once, c tanh t = c - 2 c / (1 + e^2t): one reciprocal serves both (1 / a = b / ab). e^2t is held below
// 2^60, where tanh is 1 to the last place, so that the product stays finite. A NaN takes both with it: masked places are
// cleared before. (9 capped sequences with a quotient for each: 5 % more; with tanh as a polynomial of degree 15 on the FMA pipe, which
// two-value instructions take two cycles of, 12 % more.)
__device__ __forceinline__ void capped2(float& a, float& b, float cap_in, float cap_out) {
  float x = a * cap_in, y = b * cap_in;
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x) : "f"(60.f));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(y) : "f"(60.f));
  const float ea = 1.f + ex2_approx(x), eb = 1.f + ex2_approx(y);
  const float r = -2.f * cap_out * rcp_approx(ea * eb);
  a = fmaf(r, eb, cap_out);
  b = fmaf(r, ea, cap_out);
}

// Raw sums of products into scores in log2 units: cap, then the distance bias (`at`: the row's place less the first
// key's; the row sees the first `seen` of the N, `all`: every row of the warp sees all)
template <int N, int KIND>
__device__ __forceinline__ void general_scores(uint32_t (&x)[N], const PackedParams& p, bool bias, float slope2, float at,
                                               int seen, bool all) {
  auto val = [&](int c) { return __uint_as_float(x[c]); };
  if constexpr (KIND == kWide) {
    // mostly every score of a warp is far below such a cap: up to t = 1/4 five terms of the series do (the sixth is below
    // 2^-26 of the score)
    float top = 0.f;
#pragma unroll
    for (int c = 0; c < N; c += 2) top = fmax3(top, fabsf(val(c)), fabsf(val(c + 1)));
    if (__all_sync(0xffffffffu, top * p.cap_arg <= 0.25f)) {
#pragma unroll
      for (int c = 0; c < N; ++c) {
        const float t = val(c) * p.cap_arg, z = t * t;
        const float f = fmaf(z, fmaf(z, fmaf(z, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f);
        x[c] = __float_as_uint(val(c) * p.scale_log2 * fmaf(z, f, 1.f));
      }
    } else {
#pragma unroll
      for (int c = 0; c < N; ++c) x[c] = __float_as_uint(capped_wide(val(c), p));
    }
  } else if (p.cap_out > 0.f) {
    if (!all) {
#pragma unroll
      for (int c = 0; c < N; ++c)
        if (c >= seen) x[c] = 0u;
    }
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      float u = val(c), v = val(c + 1);
      capped2(u, v, p.cap_in, p.cap_out);
      x[c] = __float_as_uint(u);
      x[c + 1] = __float_as_uint(v);
    }
  }
  const float scale = p.cap_out > 0.f ? 1.f : p.scale_log2;
  if (bias) {
    // keys all behind the row's place, or all before it: the distance is linear in c
    const bool behind = __all_sync(0xffffffffu, at >= float(N - 1)), ahead = __all_sync(0xffffffffu, at <= 0.f);
    if (behind || ahead) {
      const float step = behind ? slope2 : -slope2, base = -step * at;
#pragma unroll
      for (int c = 0; c < N; ++c) x[c] = __float_as_uint(fmaf(val(c), scale, fmaf(float(c), step, base)));
    } else {
#pragma unroll
      for (int c = 0; c < N; ++c) x[c] = __float_as_uint(fmaf(-slope2, fabsf(at - float(c)), val(c) * scale));
    }
  }
}

__device__ __forceinline__ float max64(const uint32_t (&x)[64]) {
  float m4[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) m4[v] = fmax3(__uint_as_float(x[v]), __uint_as_float(x[v + 4]), __uint_as_float(x[v + 8]));
#pragma unroll
  for (int c = 12; c < 60; c += 8)
#pragma unroll
    for (int v = 0; v < 4; ++v) m4[v] = fmax3(m4[v], __uint_as_float(x[c + v]), __uint_as_float(x[c + 4 + v]));
  const float a = fmax3(m4[0], m4[1], m4[2]), b = fmax3(m4[3], __uint_as_float(x[60]), __uint_as_float(x[61]));
  return fmaxf(a, fmax3(b, __uint_as_float(x[62]), __uint_as_float(x[63])));
}

struct Segment {
  int q0, nq, k0, nk;
  int tile;  // of the segment; < 0: none left
};

// The segment and tile of CTA x: tiles of `rows` query rows each, counted segment by segment (warp-collective).
__device__ Segment find_tile(const dit_packed_attention& a, int rows, int x) {
  const int lane = lane_id();
  auto at = [&](const int32_t* p, int s, int top) { return p ? min(max(__ldg(p + s), 0), top) : (s == 0 ? 0 : top); };
  int before = 0;
  for (int base = 0; base < a.segments; base += 128) {
    int n[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = base + 32 * u + lane;
      n[u] = 0;
      if (s < a.segments) n[u] = max(at(a.q_start, s + 1, a.q_rows) - at(a.q_start, s, a.q_rows), 0);
      n[u] = (n[u] + rows - 1) / rows;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      int sum = n[u];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + sum > x);
      if (past) {
        const int l = __ffs(past) - 1, s = base + 32 * u + l;
        const int first = before + __shfl_sync(0xffffffffu, sum - n[u], l);
        Segment g;
        g.q0 = at(a.q_start, s, a.q_rows);
        g.nq = at(a.q_start, s + 1, a.q_rows) - g.q0;
        g.k0 = at(a.k_start, s, a.k_rows);
        g.nk = max(at(a.k_start, s + 1, a.k_rows) - g.k0, 0);
        g.tile = x - first;
        return g;
      }
      before += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  return Segment{0, 0, 0, 0, -1};
}

// Whether resum_row would find anything else than the product did, which left the columns `nan` and `inf` (a bit for each of a
// lane's D / 32) of a row that sees the keys [j0, j1): a column is as it should be where values of V that the row sees make it
// so. (4224 causal rows of 24 heads with an infinite V in the sixth key: 172 ms with every row summed again, 0.5 with this look
// at V first, 0.13 where all is finite; 9 capped sequences 251, 0.7 and 0.24.) A warp per row.
template <int D>
__device__ __forceinline__ bool resum_helps(const PackedParams& p, int k0, int j0, int j1, int kvh, unsigned nan, unsigned inf) {
  constexpr int V = D / 32;
  const uint16_t* v = p.a.v + kvh * p.a.v_head + lane_id() * V;
  unsigned none = 0, up = 0, down = 0;  // of the values seen so far, by column: NaN, an infinity of either sign
  auto wrong = [&] { return (inf & ~(none | up | down)) | (nan & ~(none | (up & down))); };
  for (int base = j0; base < j1; base += 32) {
    if (!__any_sync(0xffffffffu, wrong())) return false;
#pragma unroll 4
    for (int j = base; j < min(base + 32, j1); ++j) {
      uint32_t u[V / 2];
      const uint16_t* at = v + (k0 + (long long)j) * p.a.v_row;
      if constexpr (V == 4) {
        const uint2 x = *reinterpret_cast<const uint2*>(at);
        u[0] = x.x; u[1] = x.y;
      } else {
        u[0] = *reinterpret_cast<const uint32_t*>(at);
      }
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const unsigned h = (u[c >> 1] >> ((c & 1) * 16)) & 0xffffu;
        none |= unsigned((h & 0x7fffu) > 0x7f80u) << c;
        up |= unsigned(h == 0x7f80u) << c;
        down |= unsigned(h == 0xff80u) << c;
      }
    }
  }
  return __any_sync(0xffffffffu, wrong());
}

// Which of 32 columns of this lane's row of O are NaN, and which infinite
__device__ __forceinline__ uint2 odd_columns(uint32_t taddr) {
  uint32_t raw[32];
  tmem_ld32(taddr, raw);
  tmem_ld_wait();
  uint2 b = make_uint2(0, 0);
#pragma unroll
  for (int v = 0; v < 32; ++v) {
    b.x |= unsigned((raw[v] & 0x7fffffffu) > 0x7f800000u) << v;
    b.y |= unsigned((raw[v] & 0x7fffffffu) == 0x7f800000u) << v;
  }
  return b;
}

// f times the weighted sum of V over the keys [j0, j1) that a row does see, on the plain cores: only for rows that the matrix
// product left not finite beside keys they do not see (0 x NaN), or (`own`) under a fixed maximum, where weights above 1 may
// have taken the product past fp32: those are weighed against the row's own maximum, f (1 / sum) taken along.
// A warp per row; lane l ends with values l D / 32 and on.
template <int D, int KIND>
__device__ __forceinline__ void resum_row(const PackedParams& p, int q_at, int k0, int j0, int j1, int head, int kvh, int place,
                                       float m, float f, bool own, float (&acc)[D / 32]) {
  constexpr int V = D / 32;
  const dit_packed_attention& a = p.a;
  const __nv_bfloat16* q = reinterpret_cast<const __nv_bfloat16*>(a.q) + q_at * a.q_row + head * a.q_head + lane_id() * V;
  const __nv_bfloat16* k = reinterpret_cast<const __nv_bfloat16*>(a.k) + kvh * a.k_head + lane_id() * V;
  const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(a.v) + kvh * a.v_head + lane_id() * V;
  float qv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    qv[i] = __bfloat162float(q[i]);
    acc[i] = 0.f;
  }
  auto score = [&](int j) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) s = fmaf(qv[i], __bfloat162float(k[(k0 + (long long)j) * a.k_row + i]), s);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    float x = s * p.scale_log2;
    if constexpr (KIND != kPlain) {
      if constexpr (KIND == kWide) x = capped_wide(s, p);
      else if (p.cap_out > 0.f) x = capped(s, p.cap_in, p.cap_out);
      if (a.slope) x = fmaf(-1.4426950408889634f * __ldg(a.slope + head), fabsf(float(place - j)), x);
    }
    return x;
  };
  if (own) {
    float top = -INFINITY;
    for (int j = j0; j < j1; ++j) top = fmaxf(top, score(j));
    f *= ex2_approx(top - m);
    m = top;
  }
  for (int j = j0; j < j1; ++j) {
    const float w = ex2_approx(score(j) - m) * f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float y = __bfloat162float(v[(k0 + (long long)j) * a.v_row + i]);
      acc[i] = isinf(y) ? acc[i] + y : fmaf(w, y, acc[i]);  // (whose weight may have underflowed, and is above 0 all the same)
    }
  }
}

// The rows `rows` of a warp whose product, in the `cols` columns from `first` on (at tO in tensor memory), is not finite: summed
// again where that helps, and put where a row's result goes: the staged tile (null: the output itself), or the part's sums.
// i, j1 (the end of the keys that it sees), m and f are those of the lane's row. (A function of its own, with few arguments: the
// key loop keeps its registers. 9 capped sequences 229 us with the loop in place, 220 so.)
template <int D, int KIND>
__device__ __noinline__ void mend_rows(const PackedParams& p, unsigned rows, const Segment& seg, int i, int j0, int j1, int kvh, float m, float f, bool own, uint32_t tO, int first, int cols, uint8_t* stage) {
  constexpr int V = D / 32;
  const dit_packed_attention& a = p.a;
  const int lane = lane_id(), col = lane * V;
  const int quad_row = int(threadIdx.x >> 5 & 3) * 32;  // of the tile: the warp's first
  const int q = seg.q0 + i, k0 = seg.k0, place = i + seg.nk - seg.nq, head = kvh * p.G + (quad_row + lane) % p.G;
  const bool mine = col >= first && col < first + cols;
  __syncwarp();  // the rows' own stores come first
  for (; rows; rows &= rows - 1) {
    const int src = __ffs(rows) - 1;
    auto of_row = [&](auto x) { return __shfl_sync(0xffffffffu, x, src); };
    unsigned nan = 0, inf = 0;  // of this lane's columns
    for (int c = 0; c < cols; c += 32) {
      const uint2 b = odd_columns(tO + uint32_t(c));
      const unsigned bn = of_row(b.x), bi = of_row(b.y);
      if (mine && (col - first) / 32 == c / 32) {
        nan = bn >> ((col - first) & 31) & ((1u << V) - 1);
        inf = bi >> ((col - first) & 31) & ((1u << V) - 1);
      }
    }
    const int sq = of_row(q), sh = of_row(head), end = of_row(j1);
    if (!resum_helps<D>(p, k0, j0, end, kvh, nan, inf)) continue;
    float acc[V];
    resum_row<D, KIND>(p, sq, k0, j0, end, sh, kvh, of_row(place), of_row(m == -INFINITY ? 0.f : m), of_row(f), own, acc);
    if (!mine) continue;
    if (p.splits > 1) {
      float* dst = p.part_o + (((long long)blockIdx.z * a.q_rows + sq) * a.heads + sh) * D + col;
#pragma unroll
      for (int v = 0; v < V; ++v) dst[v] = acc[v];
    } else {
      const int row = quad_row + src, at = col * 2;  // byte of the row
      uint32_t* dst = reinterpret_cast<uint32_t*>(stage ? stage + row * (D * 2) + (((at >> 4) ^ (row & 7)) << 4) + (at & 15)
                                                        : reinterpret_cast<uint8_t*>(a.o + sq * a.o_row + sh * a.o_head + col));
#pragma unroll
      for (int v = 0; v < V / 2; ++v) dst[v] = pack_bf16x2(acc[2 * v], acc[2 * v + 1]);
    }
  }
}

// The rest of the key tiles for a warp whose wait gave up at tile `it`, while the other of its row pair may have seen its own
// end: it passes the barriers of the pair as that one does. Both know the maxima of the tiles before and so the same m, and
// both read the same two places here: `own`, which stays as it was, and `theirs`, which the other leaves alone once it has met
// this one, because the scores of tile it + 1 wait for this warp's weights. So both take the same turn at every rescale,
// until the other gives up as well, at the next tile at the latest. (Joining the two verdicts at every tile's barrier instead: 163
// us for two sequences of 24 heads of 128 that take 158 without, and with this.)
__device__ __noinline__ void attend_meetings(const volatile float* s_max, int it, int n, float m) {
  const int warp = int(threadIdx.x >> 5) - 2, pair = 1 + (warp >> 3) * 4 + ((warp + 2) & 3);  // as in packed_kernel
  const volatile float* own = s_max + (warp >> 2) * 128 + ((warp + 2) & 3) * 32 + lane_id();
  const volatile float* theirs = s_max + ((warp >> 2) ^ 1) * 128 + ((warp + 2) & 3) * 32 + lane_id();
  for (; it < n; ++it) {
    asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
    const float mx = fmaxf(*own, *theirs);
    const bool up = mx > m + kRescaleStep;
    if (up) m = mx;
    if (__any_sync(0xffffffffu, up) && it > 0) asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
  }
}

template <int D, int KIND>
__global__ void __launch_bounds__(kPackedThreads, 1)
    packed_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PackedParams p) {
  using Cfg = PackedCfg<D>;
  constexpr bool GEN = KIND != kPlain;
  constexpr int KS = Cfg::kKS, VS = Cfg::kVS;
  extern __shared__ __align__(256) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + 2 * Cfg::kTile;
  uint8_t* sV = sK + KS * Cfg::kTile;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sV + VS * Cfg::kTile);
  uint64_t* drain = q_full + 1;
  uint64_t* k_full = drain + 1;      // [KS]
  uint64_t* k_empty = k_full + KS;   // [KS]
  uint64_t* v_full = k_empty + KS;   // [VS]
  uint64_t* v_empty = v_full + VS;   // [VS]
  uint64_t* s_full = v_empty + VS;   // [2]
  uint64_t* p_half = s_full + 2;     // [2] the first half of each key half's weights stored
  uint64_t* p_full = p_half + 2;     // [2]
  uint64_t* o_done = p_full + 2;     // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_done + 2);
  int* s_lim = reinterpret_cast<int*>(tmem_slot + 1);              // [2] keys that any row of the tile sees
  Segment* s_seg = reinterpret_cast<Segment*>(s_lim + 2);          // 20 bytes
  float* s_max = reinterpret_cast<float*>(tmem_slot + 16);  // [2 tiles][2 key halves][128 rows]

  const dit_packed_attention& a = p.a;
  const int warp = threadIdx.x >> 5, lane = lane_id();
  const int kvh = blockIdx.y, G = p.G, rpt = p.rpt;

  pdl_wait();
  if (warp == 0) {
    // from the last tile: where rows see the keys before them, the long ones start first
    const Segment g = find_tile(a, 2 * rpt, gridDim.x - 1 - blockIdx.x);
    if (lane == 0) *s_seg = g;
  } else if (threadIdx.x == 32) {
    s_lim[0] = s_lim[1] = 0;
    mbar_init(smem_u32(q_full), 1);
    mbar_init(smem_u32(drain), 1);
    for (int s = 0; s < KS; ++s) {
      mbar_init(smem_u32(&k_full[s]), 1);
      mbar_init(smem_u32(&k_empty[s]), 1);
    }
    for (int s = 0; s < VS; ++s) {
      mbar_init(smem_u32(&v_full[s]), 1);
      mbar_init(smem_u32(&v_empty[s]), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(&s_full[t]), 1);
      mbar_init(smem_u32(&p_half[t]), 8);  // one arrival per warp of the tile's group
      mbar_init(smem_u32(&p_full[t]), 8);
      mbar_init(smem_u32(&o_done[t]), 1);
    }
    fence_mbar_init();
  }
  __syncthreads();
  const Segment seg = *s_seg;
  if (seg.tile < 0) return;  // more CTAs than tiles: the bound counts a part-filled tile for every segment

  // a softmax thread's row: query row `i` of the segment, head `head`, seeing `lim` keys
  const int t = (warp - 2) >> 3, half = ((warp - 2) >> 2) & 1, quad = warp & 3, row = quad * 32 + lane;
  const int r = row / G, g = row - r * G;
  const int i = (seg.tile * 2 + t) * rpt + r;
  const int head = kvh * G + g;
  const bool valid = warp >= 2 && r < rpt && i < seg.nq;
  int lim = 0;
  if (warp >= 2) {
    if (valid) lim = a.visible ? min(max(__ldg(a.visible + seg.q0 + i), 0), seg.nk) : seg.nk;
    const int top = __reduce_max_sync(0xffffffffu, lim);
    if (lane == 0 && top > 0) atomicMax(&s_lim[t], top);
  } else if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now: a kernel that starts early on this SM finds this CTA's tensor memory taken, never the other way round
  pdl_trigger();
  const uint32_t tmem_base = *tmem_slot;
  // this CTA's key tiles [ta, tb), and how many of them each tile (or half) takes
  const int lmax = max(s_lim[0], s_lim[1]);
  const int tiles = (lmax + 127) >> 7;
  const int ta = int((long long)tiles * blockIdx.z / p.splits), tb = int((long long)tiles * (blockIdx.z + 1) / p.splits);
  const int n0 = min(max((s_lim[0] + 127) >> 7, ta), tb) - ta, n1 = min(max((s_lim[1] + 127) >> 7, ta), tb) - ta;
  const int loads = max(n0, n1);

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (loads > 0 && elect_one()) {
      const uint32_t qb = smem_u32(q_full);
      const bool first = n0 > 0, second = n1 > 0;
      mbar_arrive_expect_tx(qb, uint32_t(int(first) + int(second)) * (D / 64) * 128u * uint32_t(G * rpt));
      for (int tt = 0; tt < 2; ++tt) {
        if (tt == 0 ? !first : !second) continue;
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(smem_u32(sQ + tt * Cfg::kTile + c * Cfg::kAtom), &tmQ, qb, c * 64, kvh * G,
                      seg.q0 + (seg.tile * 2 + tt) * rpt);
      }
      int nk = 0, nv = 0;
      for (int j = 0; j < loads; ++j) {
        const int key = seg.k0 + (ta + j) * 128;
        const int ks = j % KS, vs = j % VS;
        if (!mbar_wait(smem_u32(&k_empty[ks]), ((j / KS) & 1) ^ 1, p.err, kErrTimeoutProducer)) break;
        const uint32_t kb = smem_u32(&k_full[ks]);
        mbar_arrive_expect_tx(kb, Cfg::kTile);
        for (int c = 0; c < D / 64; ++c) tma_load_3d(smem_u32(sK + ks * Cfg::kTile + c * Cfg::kAtom), &tmK, kb, c * 64, kvh, key);
        ++nk;
        if (!mbar_wait(smem_u32(&v_empty[vs]), ((j / VS) & 1) ^ 1, p.err, kErrTimeoutProducer)) break;
        const uint32_t vb = smem_u32(&v_full[vs]);
        mbar_arrive_expect_tx(vb, Cfg::kTile);
        for (int c = 0; c < D / 64; ++c) tma_load_3d(smem_u32(sV + vs * Cfg::kTile + c * Cfg::kAtom), &tmV, vb, c * 64, kvh, key);
        ++nv;
      }
      // every issued copy lands before the CTA exits, whatever the error word says
      auto landed = [&](uint64_t* bar, uint32_t parity) {
        mbar_wait_cluster(smem_u32(bar), parity, p.err, kErrTimeoutDrain, 4 * kWaitLimitNs, false);
      };
      landed(q_full, 0);
      for (int j = max(0, nk - KS); j < nk; ++j) landed(&k_full[j % KS], (j / KS) & 1);
      for (int j = max(0, nv - VS); j < nv; ++j) landed(&v_full[j % VS], (j / VS) & 1);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (loads > 0 && elect_one()) {
      constexpr uint32_t idesc_s = idesc_bf16(128, 128);
      constexpr uint32_t idesc_o = idesc_bf16(128, D) | (1u << 16);  // B is MN-major
      const uint64_t dq = sw128_desc(smem_u32(sQ)), dv = v_desc(smem_u32(sV), Cfg::kAtom);
      const uint32_t q_lo = uint32_t(dq), hi = uint32_t(dq >> 32);  // the high words agree: 1024-byte strides, same swizzle
      const uint32_t k_lo = uint32_t(sw128_desc(smem_u32(sK))), v_lo = uint32_t(dv);
      bool ok = mbar_wait(smem_u32(q_full), 0, p.err, kErrTimeoutMma);
      auto count = [&](int tt) { return tt == 0 ? n0 : n1; };
      auto issue_s = [&](int tt, int it) {
        const int ks = it % KS;
        const uint32_t d = tmem_base + uint32_t(tt * 128);
        const uint32_t qt = q_lo + uint32_t(tt * (Cfg::kTile >> 4)), kt = k_lo + uint32_t(ks * (Cfg::kTile >> 4));
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t c = uint32_t((kk >> 2) * (Cfg::kAtom >> 4) + 2 * (kk & 3));
          umma_bf16_lo(d, qt + c, kt + c, hi, idesc_s, kk != 0);
        }
        umma_commit(smem_u32(&s_full[tt]));
        if (tt == 1 || it >= n1) umma_commit(smem_u32(&k_empty[ks]));  // the tile's last user
      };
      auto wait_k = [&](int it) { return mbar_wait(smem_u32(&k_full[it % KS]), (it / KS) & 1, p.err, kErrTimeoutMma); };
      for (int tt = 0; tt < 2 && ok; ++tt)
        if (count(tt) > 0) {
          ok = wait_k(0);
          if (!ok) break;
          tc_fence_after();
          issue_s(tt, 0);
        }
      const int most = max(n0, n1);
      for (int it = 0; it < most && ok; ++it) {
#pragma unroll 1
        for (int tt = 0; tt < 2; ++tt) {
          const int n = count(tt);
          if (it >= n) continue;
          const int vs = it % VS;
          // the next K lands long before this tile's weights are ready: waited for first, so that P V and the next S
          // go out back to back
          if (it + 1 < n && !wait_k(it + 1)) { ok = false; break; }
          if (!mbar_wait(smem_u32(&v_full[vs]), (it / VS) & 1, p.err, kErrTimeoutMma)) { ok = false; break; }
          const uint32_t d = tmem_base + 256u + uint32_t(tt * D), pt = tmem_base + uint32_t(tt * 128);
          const uint32_t vt = v_lo + uint32_t(vs * (Cfg::kTile >> 4));
          // in two halves: the 32 keys of each key half whose weights are stored first, then the others
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!mbar_wait(smem_u32(h == 0 ? &p_half[tt] : &p_full[tt]), it & 1, p.err, kErrTimeoutMma)) { ok = false; break; }
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {  // 16 keys a step: 2048 bytes of every box
              if (((kk & 3) >> 1) != h) continue;
              umma_bf16_ts_lo(d, pt + uint32_t((kk >> 2) * 64 + (kk & 3) * 8), vt + uint32_t(kk * 128), hi, idesc_o,
                              it != 0 || kk != 0);
            }
          }
          if (!ok) break;
          if (tt == 1 || it >= n1) umma_commit(smem_u32(&v_empty[vs]));
          if (it + 1 == n) umma_commit(smem_u32(&o_done[tt]));
          else issue_s(tt, it + 1);
        }
      }
      umma_commit(smem_u32(drain));
      mbar_wait_cluster(smem_u32(drain), 0, p.err, kErrTimeoutDrain, 4 * kWaitLimitNs, false);
    }
  } else {
    // ------------------------------------------------------------------ softmax warps: a row's 64 keys per thread
    const uint32_t lane_off = uint32_t(quad * 32) << 16;
    const uint32_t tS = tmem_base + lane_off + uint32_t(t * 128 + half * 64);
    const uint32_t tO = tmem_base + lane_off + 256u + uint32_t(t * D + half * (D / 2));  // this thread's half of O
    const int n = t == 0 ? n0 : n1;
    const int pair = 1 + t * 4 + quad;  // named barrier of the two warps that share 32 rows
    auto meet = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory"); };
    const bool live = __any_sync(0xffffffffu, lim > 0);  // warps without a row that sees a key only keep the barriers
    const int place = i + seg.nk - seg.nq;               // the row's place among the keys
    float slope2 = 0.f;
    if constexpr (GEN)
      if (a.slope && valid) slope2 = 1.4426950408889634f * __ldg(a.slope + head);
    // Capped scores lie within the cap C (log2 units) of 0, or with a bias of what the nearest key that the row sees loses: up to
    // kFixedLog2 the weights are taken against a fixed maximum, C or where that is less 80 - C: they lie within 2^80, and at the
    // row's best key above 2^-80, so that neither keys 2^46 below it nor values of V down to 2^-46 are lost to fp32's least.
    // Values of V so large that a weight takes them past its largest leave the row not finite, and resum_row mends it. (Parts of a
    // split range go without: both halves of a row would have to agree on its maximum again.) Neither the row's own maximum nor the
    // exchange of it is needed (9 sequences, capped: 246 us with, 220 without). The nearest key lies behind the row where the
    // row's place is past what it sees, and ahead of it where there are more rows than keys and the place is negative.
    // (A negative slope grows with the distance: no such bound. And past 2^20 that key's bias, which scores and maximum round
    // apart, would leave their difference too few places.)
    const float near = slope2 * float(max(max(0, place - lim + 1), -place));
    const bool fixed = KIND == kCapped && p.cap_out > 0.f && p.cap_out <= kFixedLog2 && p.splits == 1 &&
                       __all_sync(0xffffffffu, slope2 >= 0.f && near <= 0x1p20f);
    float m = -INFINITY, l = 0.f;
    if (fixed) m = fminf(p.cap_out, 80.f - p.cap_out) - near;
    bool ok = true;
    int it = 0;
    for (; it < n; ++it) {
      const int key0 = (ta + it) * 128;
      // rows of V that no row of the CTA sees, zeroed by the first group that uses the tile
      const int vz = lmax - key0;
      if (vz < 128 && (t == 0 || it >= n0)) {
        if (!mbar_wait_warp(smem_u32(&v_full[it % VS]), (it / VS) & 1, p.err, kErrTimeoutSoftmax)) { ok = false; break; }
        if (row >= vz) {
          uint8_t* at = sV + (it % VS) * Cfg::kTile + row * 128 + (D == 128 ? half * Cfg::kAtom : half * 64);
#pragma unroll
          for (int v = 0; v < (D == 128 ? 8 : 4); ++v) *reinterpret_cast<uint4*>(at + v * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      if (!mbar_wait_warp(smem_u32(&s_full[t]), it & 1, p.err, kErrTimeoutSoftmax)) { ok = false; break; }
      tc_fence_after();
      if (live) {
        uint32_t x[64];
        tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
        tmem_ld32(tS + 32u, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
        tmem_ld_wait();
        const int first = key0 + half * 64;
        const int seen = lim - first;
        const bool all = __all_sync(0xffffffffu, seen >= 64);
        if constexpr (GEN) general_scores<64, KIND>(x, p, a.slope != nullptr, slope2, float(place - first), seen, all);
        if (!all) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c >= seen) x[c] = 0xff800000u;
        }
        float alpha = 1.f;
        if (!fixed) {
          float mx = max64(x);
          if constexpr (!GEN) mx *= p.scale_log2;
          // the row's maximum over both halves of the keys. (One place per row: the other warp has read it before this
          // tile's weights are complete, without which there is no next tile of scores.)
          s_max[(t * 2 + half) * 128 + row] = mx;
          meet();
          mx = fmaxf(mx, s_max[(t * 2 + (half ^ 1)) * 128 + row]);
          if (mx > m + kRescaleStep) {  // also on the first tile with a key (m = -inf)
            alpha = ex2_approx(m - mx);
            m = mx;
          }
          if (it > 0 && __any_sync(0xffffffffu, alpha < 1.0f)) {
            // O holds earlier tiles; this S came after the P V before it, which is done. (Eight columns at a time: the scores
            // keep their registers.)
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[8];
              tmem_ld8(tO + uint32_t(c * 8), o);
              tmem_ld_wait();
#pragma unroll
              for (int v = 0; v < 8; ++v) o[v] = __float_as_uint(__uint_as_float(o[v]) * alpha);
              tmem_st8(tO + uint32_t(c * 8), o);
            }
            // both warps' halves of O before the first product adds to them
            tmem_st_wait();
            tc_fence_before();
            meet();
          }
        }
        const float base = m == -INFINITY ? 0.f : m;  // nothing seen yet: weights 2^-inf = 0
        const float scale = GEN ? 1.f : p.scale_log2;
        const uint64_t scale2 = f2_pack(scale, scale), neg2 = f2_pack(-base, -base);
        uint64_t sum2[4] = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int k0 = c * 32 + 2 * v;
            const uint64_t s2 = f2_pack(__uint_as_float(x[k0]), __uint_as_float(x[k0 + 1]));
            const uint64_t e2 = GEN ? f2_add(s2, neg2) : f2_fma(s2, scale2, neg2);
            const float w0 = ex2_approx(f2_lo(e2)), w1 = ex2_approx(f2_hi(e2));
            sum2[v & 3] = f2_add(sum2[v & 3], f2_pack(w0, w1));
            pk[v] = pack_bf16x2(w0, w1);
          }
          tmem_st16(tS + uint32_t(c * 16), pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(c == 0 ? &p_half[t] : &p_full[t]));
        }
        const uint64_t s4 = f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3]));
        l = fmaf(l, alpha, f2_lo(s4) + f2_hi(s4));
      } else {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&p_half[t]));
          mbar_arrive(smem_u32(&p_full[t]));
        }
      }
    }

    // ---- the end of the key range
    if (!ok && live && !fixed)
      attend_meetings(s_max, it, n, m);
    if (n > 0 && ok) ok = mbar_wait_warp(smem_u32(&o_done[t]), 0, p.err, kErrTimeoutSoftmax);
    // (what follows has the same barriers whatever happened, as the tiles had: attend_meetings)
    uint8_t* stage = sQ + t * Cfg::kTile;  // Q has been read; [row][D] bf16, chunks swizzled by the row
    if (n > 0) {
      // the row's sum over both halves, through the places of the maxima (the staged rows of other warps lie over everything
      // else that is free)
      meet();  // a last tile's maximum has been read
      s_max[(t * 2 + half) * 128 + row] = l;
      meet();
      l += s_max[(t * 2 + (half ^ 1)) * 128 + row];
    }
    if (ok) {
      tc_fence_after();
      const bool whole = p.splits == 1;
      const int covered = (ta + n) * 128;  // keys behind the last tile of this row's sums
      const int last = min(lmax, covered);
      const float inv = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
      const long long at = ((long long)blockIdx.z * a.q_rows + seg.q0 + i) * a.heads + head;  // of the partial sums
      float4* po = reinterpret_cast<float4*>(p.part_o + at * D + half * (D / 2));
      float bad = 0.f;
      unsigned again = 0;
      if (live && n > 0) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t raw[32];
          tmem_ld32(tO + uint32_t(c * 32), raw);
          tmem_ld_wait();
          float o[32];
#pragma unroll
          for (int v = 0; v < 32; ++v) {
            o[v] = lim > 0 ? __uint_as_float(raw[v]) : 0.f;
            bad = fmaf(o[v], 0.f, bad);
            o[v] *= inv;
          }
          if (whole) {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              *reinterpret_cast<uint4*>(stage + row * (D * 2) + (((half * (D / 16) + c * 4 + v) ^ (row & 7)) << 4)) =
                  make_uint4(pack_bf16x2(o[8 * v], o[8 * v + 1]), pack_bf16x2(o[8 * v + 2], o[8 * v + 3]),
                             pack_bf16x2(o[8 * v + 4], o[8 * v + 5]), pack_bf16x2(o[8 * v + 6], o[8 * v + 7]));
          } else if (valid) {
#pragma unroll
            for (int v = 0; v < 8; ++v) po[c * 8 + v] = make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
          }
        }
        // rows with something that is not finite (in this half of O) beside keys they do not see, or by their weights; where
        // the weights' sum is NaN already, it is for scores that the row sees
        again = __ballot_sync(0xffffffffu, valid && bad != 0.f && l == l && (lim < last || fixed));
      } else if (whole) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          *reinterpret_cast<uint4*>(stage + row * (D * 2) + (((half * (D / 16) + c) ^ (row & 7)) << 4)) = make_uint4(0, 0, 0, 0);
      }
      if (valid && half == 0) {
        if (!whole) p.part_ml[at] = make_float2(l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m), l);  // (no key; scores all NaN: seen)
        else if (a.lse)
          a.lse[(long long)head * a.q_rows + seg.q0 + i] =
              l > 0.f || l != l ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
      }
      // (here, behind the stores of lse: right behind the vote, two sequences of 24 heads of 128 take 161 us, so 157)
      if (again)
        mend_rows<D, KIND>(p, again, *s_seg, i, ta * 128, min(lim, covered), kvh, m, inv, fixed, tO, half * (D / 2), D / 2, stage);
    }
    if (p.splits == 1) {
      // whole rows out of the staged tile: D / 8 lanes of 16 bytes to a row; each warp every other row of the pair's 32
      meet();
      constexpr int per = 32 / (D / 8);
      if (ok)
        for (int rr = lane / (D / 8) + half * per; rr < 32; rr += 2 * per) {
          const int srow = quad * 32 + rr, sr = srow / G, sg = srow - sr * G, c = lane % (D / 8);
          const int si = (seg.tile * 2 + t) * rpt + sr;
          if (sr >= rpt || si >= seg.nq) continue;
          const uint4 v = *reinterpret_cast<const uint4*>(stage + srow * (D * 2) + ((c ^ (srow & 7)) << 4));
          *reinterpret_cast<uint4*>(a.o + (seg.q0 + si) * a.o_row + (kvh * G + sg) * a.o_head + c * 8) = v;
        }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, 512);
}

// ------------------------------------------------------------------------------------------
// Few rows over many keys, HBM-bound, and short segments, bound by a CTA's start and end. One tile of up to 128 (row, head) pairs per CTA, key tiles of 64, two CTAs to an SM
// (256 columns of tensor memory and at most 113 KB of shared memory each), so that one CTA's start and end run under the
// other's loads. K and V tiles come through one ring in the order in which the MMAs use them: K0 K1 V0 K2 V1 ... The
// scores of tile j + 1 are computed while the softmax works on tile j. Q takes only the rows it has: the MMA's other
// rows read what follows in shared memory, and nothing reads their results.
// Tensor memory (256 columns): [0, 64) and [64, 128) S of even and odd tiles, P over them   [128, 128 + d) O
// ------------------------------------------------------------------------------------------
constexpr int kRowKeys = 64, kRowSlotsMost = 12, kRowThreads = 192;
constexpr uint32_t kRowSmem = 113 * 1024, kRowBars = 8 * (2 * kRowSlotsMost + 8) + 64;

// Place of a key tile's K and V in the ring's order, for n tiles
__device__ __forceinline__ int place_k(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int place_v(int j, int n) { return j + 1 < n ? 2 * j + 2 : 2 * j + 1; }

template <int D, int KIND>
__global__ void __launch_bounds__(kRowThreads, 2)
    packed_rows_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ PackedParams p) {
  constexpr bool GEN = KIND != kPlain;
  constexpr uint32_t kSlot = kRowKeys * D * 2, kBox = kRowKeys * 128;  // a tile of K or V; its boxes of 64 values
  extern __shared__ __align__(256) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t q_box = uint32_t((p.G * p.rpt + 7) & ~7) * 128u;
  const int T = p.slots;
  uint8_t* sQ = smem;
  uint8_t* ring = sQ + q_box * (D / 64);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + T * kSlot);  // [T]
  uint64_t* empty = full + kRowSlotsMost;                          // [T]
  uint64_t* q_full = empty + kRowSlotsMost;
  uint64_t* s_full = q_full + 1;   // [2]
  uint64_t* p_full = s_full + 2;   // [2]
  uint64_t* pv_done = p_full + 2;  // a phase per key tile
  uint64_t* o_done = pv_done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_done + 1);
  int* s_lim = reinterpret_cast<int*>(tmem_slot + 1);
  Segment* s_seg = reinterpret_cast<Segment*>(s_lim + 1);

  const dit_packed_attention& a = p.a;
  const int warp = threadIdx.x >> 5, lane = lane_id();
  const int kvh = blockIdx.y, G = p.G, rpt = p.rpt;

  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 256);
    tmem_relinquish();
  } else if (threadIdx.x == 64) {
    *s_lim = 0;
    for (int i = 0; i < T; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), 1);
    }
    mbar_init(smem_u32(q_full), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), 4);
    }
    mbar_init(smem_u32(pv_done), 1);
    mbar_init(smem_u32(o_done), 1);
    fence_mbar_init();
  }
  pdl_wait();
  if (warp == 0) {
    const Segment g = find_tile(a, rpt, blockIdx.x);
    if (lane == 0) *s_seg = g;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // only now: a kernel that starts early on this SM finds this CTA's tensor memory taken, never the other way round
  pdl_trigger();
  const uint32_t tmem_base = *tmem_slot;
  const Segment seg = *s_seg;

  // a softmax thread's row: query row `i` of the segment, head `head`, seeing `lim` keys
  const int quad = warp & 3, row = quad * 32 + lane;
  const int r = row / G, g = row - r * G;
  const int i = seg.tile * rpt + r, head = kvh * G + g;
  const bool valid = warp >= 2 && seg.tile >= 0 && r < rpt && i < seg.nq;
  int lim = 0;
  if (warp >= 2) {
    if (valid) lim = a.visible ? min(max(__ldg(a.visible + seg.q0 + i), 0), seg.nk) : seg.nk;
    const int top = __reduce_max_sync(0xffffffffu, lim);
    if (lane == 0 && top > 0) atomicMax(s_lim, top);
  }
  __syncthreads();
  const int lmax = *s_lim, tiles = (lmax + kRowKeys - 1) / kRowKeys;
  const int ta = int((long long)tiles * blockIdx.z / p.splits), tb = int((long long)tiles * (blockIdx.z + 1) / p.splits);
  const int n = tb - ta;

  if (warp == 0) {
    // ------------------------------------------------------------------ TMA producer
    if (n > 0 && elect_one()) {
      const uint32_t qb = smem_u32(q_full);
      mbar_arrive_expect_tx(qb, (D / 64) * 128u * uint32_t(G * rpt));
      for (int c = 0; c < D / 64; ++c)
        tma_load_3d(smem_u32(sQ + c * q_box), &tmQ, qb, c * 64, kvh * G, seg.q0 + seg.tile * rpt);
      int x = 0;
      bool ok = true;
      auto load = [&](const CUtensorMap* m, int j) {
        const int slot = x % T;
        if (!mbar_wait(smem_u32(&empty[slot]), ((x / T) & 1) ^ 1, p.err, kErrTimeoutProducer)) { ok = false; return; }
        const uint32_t fb = smem_u32(&full[slot]);
        mbar_arrive_expect_tx(fb, kSlot);
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(smem_u32(ring + slot * kSlot + c * kBox), m, fb, c * 64, kvh, seg.k0 + (ta + j) * kRowKeys);
        ++x;
      };
      load(&tmK, 0);
      for (int j = 0; j < n && ok; ++j) {
        if (j + 1 < n) load(&tmK, j + 1);
        if (ok) load(&tmV, j);
      }
      // every issued copy lands before the CTA exits, whatever the error word says
      mbar_wait_cluster(qb, 0, p.err, kErrTimeoutDrain, 4 * kWaitLimitNs, false);
      for (int y = max(0, x - T); y < x; ++y)
        mbar_wait_cluster(smem_u32(&full[y % T]), (y / T) & 1, p.err, kErrTimeoutDrain, 4 * kWaitLimitNs, false);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    if (n > 0 && elect_one()) {
      constexpr uint32_t idesc_s = idesc_bf16(128, kRowKeys);
      constexpr uint32_t idesc_o = idesc_bf16(128, D) | (1u << 16);  // B is MN-major
      const uint64_t dq = sw128_desc(smem_u32(sQ));
      const uint32_t q_lo = uint32_t(dq), hi = uint32_t(dq >> 32);
      const uint32_t k_lo = uint32_t(sw128_desc(smem_u32(ring))), v_lo = uint32_t(v_desc(smem_u32(ring), kBox));
      auto landed = [&](int x) { return mbar_wait(smem_u32(&full[x % T]), (x / T) & 1, p.err, kErrTimeoutMma); };
      auto issue_s = [&](int j) {
        const int x = place_k(j);
        const uint32_t kt = k_lo + uint32_t((x % T) * (kSlot >> 4)), d = tmem_base + uint32_t((j & 1) * kRowKeys);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          umma_bf16_lo(d, q_lo + uint32_t((kk >> 2) * (q_box >> 4) + 2 * (kk & 3)),
                       kt + uint32_t((kk >> 2) * (kBox >> 4) + 2 * (kk & 3)), hi, idesc_s, kk != 0);
        umma_commit(smem_u32(&s_full[j & 1]));
        umma_commit(smem_u32(&empty[x % T]));
      };
      bool ok = mbar_wait(smem_u32(q_full), 0, p.err, kErrTimeoutMma);
      for (int j = 0; j < 2 && j < n && ok; ++j) {
        ok = landed(place_k(j));
        if (!ok) break;
        tc_fence_after();
        issue_s(j);
      }
      for (int j = 0; j < n && ok; ++j) {
        const int x = place_v(j, n);
        if (!landed(x) || !mbar_wait(smem_u32(&p_full[j & 1]), (j >> 1) & 1, p.err, kErrTimeoutMma)) break;
        tc_fence_after();
        const uint32_t vt = v_lo + uint32_t((x % T) * (kSlot >> 4)), pt = tmem_base + uint32_t((j & 1) * kRowKeys);
#pragma unroll
        for (int kk = 0; kk < kRowKeys / 16; ++kk)
          umma_bf16_ts_lo(tmem_base + 128u, pt + uint32_t(kk * 8), vt + uint32_t(kk * 128), hi, idesc_o, j != 0 || kk != 0);
        umma_commit(smem_u32(&empty[x % T]));
        umma_commit(smem_u32(pv_done));
        if (j + 2 < n) {
          if (!landed(place_k(j + 2))) break;
          tc_fence_after();
          issue_s(j + 2);
        }
      }
      // every MMA has completed before tensor memory is given back (also where a wait gave up)
      umma_commit(smem_u32(o_done));
      mbar_wait_cluster(smem_u32(o_done), 0, p.err, kErrTimeoutDrain, 4 * kWaitLimitNs, false);
    }
  } else {
    // ------------------------------------------------------------------ softmax warps, one row per thread
    const uint32_t lane_off = uint32_t(quad * 32) << 16;
    const uint32_t tO = tmem_base + lane_off + 128u;
    const bool live = __any_sync(0xffffffffu, lim > 0);  // warps without a row that sees a key only keep the barriers
    const int place = i + seg.nk - seg.nq;               // the row's place among the keys
    float slope2 = 0.f;
    if constexpr (GEN)
      if (a.slope && valid) slope2 = 1.4426950408889634f * __ldg(a.slope + head);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      const int key0 = (ta + j) * kRowKeys;
      const uint32_t tS = tmem_base + lane_off + uint32_t((j & 1) * kRowKeys);
      if (!mbar_wait_warp(smem_u32(&s_full[j & 1]), (j >> 1) & 1, p.err, kErrTimeoutSoftmax)) { ok = false; break; }
      tc_fence_after();
      if (live) {
        uint32_t x[64];
        tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&x[0]));
        tmem_ld32(tS + 32u, *reinterpret_cast<uint32_t(*)[32]>(&x[32]));
        tmem_ld_wait();
        const int seen = lim - key0;
        const bool all = __all_sync(0xffffffffu, seen >= kRowKeys);
        if constexpr (GEN) general_scores<64, KIND>(x, p, a.slope != nullptr, slope2, float(place - key0), seen, all);
        if (!all) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c >= seen) x[c] = 0xff800000u;
        }
        float mx = max64(x);
        if constexpr (!GEN) mx *= p.scale_log2;
        float alpha = 1.f;
        if (mx > m + kRescaleStep) {  // also on the first tile with a key (m = -inf)
          alpha = ex2_approx(m - mx);
          m = mx;
        }
        const float base = m == -INFINITY ? 0.f : m;  // nothing seen yet: weights 2^-inf = 0
        const float scale = GEN ? 1.f : p.scale_log2;
        const uint64_t scale2 = f2_pack(scale, scale), neg2 = f2_pack(-base, -base);
        uint64_t sum2[4] = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int k0 = c * 32 + 2 * v;
            const uint64_t s2 = f2_pack(__uint_as_float(x[k0]), __uint_as_float(x[k0 + 1]));
            const uint64_t e2 = GEN ? f2_add(s2, neg2) : f2_fma(s2, scale2, neg2);
            const float w0 = ex2_approx(f2_lo(e2)), w1 = ex2_approx(f2_hi(e2));
            sum2[v & 3] = f2_add(sum2[v & 3], f2_pack(w0, w1));
            pk[v] = pack_bf16x2(w0, w1);
          }
          tmem_st16(tS + uint32_t(c * 16), pk);
        }
        const uint64_t s4 = f2_add(f2_add(sum2[0], sum2[1]), f2_add(sum2[2], sum2[3]));
        l = fmaf(l, alpha, f2_lo(s4) + f2_hi(s4));
        if (j > 0 && __any_sync(0xffffffffu, alpha < 1.0f)) {
          // O holds earlier tiles: the last P V must be done. (This S came after the P V before that one, so its phase is the
          // barrier's current one or has just completed, and the parity tells the two apart.)
          if (!mbar_wait_warp(smem_u32(pv_done), (j - 1) & 1, p.err, kErrTimeoutSoftmax)) {
            tmem_st_wait();  // the weights' stores land before tensor memory is given back
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + uint32_t(c * 32), o);
            tmem_ld_wait();
#pragma unroll
            for (int v = 0; v < 32; ++v) o[v] = __float_as_uint(__uint_as_float(o[v]) * alpha);
            tmem_st32(tO + uint32_t(c * 32), o);
          }
        }
        tmem_st_wait();
      }
      // rows of V that no row of the CTA sees
      const int vz = lmax - key0;
      if (vz < kRowKeys) {
        const int x = place_v(j, n);
        if (!mbar_wait_warp(smem_u32(&full[x % T]), (x / T) & 1, p.err, kErrTimeoutSoftmax)) { ok = false; break; }
        if ((row >> 1) >= vz) {  // two threads to a key's row
          uint8_t* at = ring + (x % T) * kSlot + (row >> 1) * 128 + (row & 1) * 64;
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
#pragma unroll
            for (int v = 0; v < 4; ++v) *reinterpret_cast<uint4*>(at + c * kBox + v * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&p_full[j & 1]));
    }

    if (n > 0 && ok) ok = mbar_wait_warp(smem_u32(o_done), 0, p.err, kErrTimeoutSoftmax);
    const bool any = __any_sync(0xffffffffu, valid);
    if (ok && any) {
      tc_fence_after();
      const bool whole = p.splits == 1;
      const int covered = tb * kRowKeys, last = min(lmax, covered);
      const float inv = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
      const long long at = ((long long)blockIdx.z * a.q_rows + seg.q0 + i) * a.heads + head;  // of the partial sums
      uint16_t* po = a.o + (seg.q0 + i) * a.o_row + head * a.o_head;
      float bad = 0.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t raw[32];
        if (n > 0) {
          tmem_ld32(tO + uint32_t(c * 32), raw);
          tmem_ld_wait();
        }
        float o[32];
#pragma unroll
        for (int v = 0; v < 32; ++v) {
          o[v] = n > 0 && lim > 0 ? __uint_as_float(raw[v]) : 0.f;
          bad = fmaf(o[v], 0.f, bad);
          o[v] *= inv;
        }
        if (!valid) continue;
        if (whole) {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            *reinterpret_cast<uint4*>(po + c * 32 + v * 8) =
                make_uint4(pack_bf16x2(o[8 * v], o[8 * v + 1]), pack_bf16x2(o[8 * v + 2], o[8 * v + 3]),
                           pack_bf16x2(o[8 * v + 4], o[8 * v + 5]), pack_bf16x2(o[8 * v + 6], o[8 * v + 7]));
        } else if (n > 0) {
#pragma unroll
          for (int v = 0; v < 8; ++v)
            reinterpret_cast<float4*>(p.part_o + at * D)[c * 8 + v] = make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
        }
      }
      if (valid) {
        if (!whole) p.part_ml[at] = make_float2(m == -INFINITY && l != l ? 0.f : m, l);  // scores all NaN: seen
        else if (a.lse)
          a.lse[(long long)head * a.q_rows + seg.q0 + i] =
              l > 0.f || l != l ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
      }
      // rows with something that is not finite beside keys they do not see
      unsigned again = __ballot_sync(0xffffffffu, valid && bad != 0.f && l == l && lim < last);
      if (again)
        mend_rows<D, KIND>(p, again, *s_seg, i, ta * kRowKeys, min(lim, covered), kvh, m, inv, false, tO, 0,
                           D, nullptr);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, 256);
}

// The parts of a split key range joined, a warp per (row, head): weights 2^(m_z - max m), parts without a key skipped
// (their sums were never written).
template <int D>
__global__ void __launch_bounds__(256) packed_join_kernel(const __grid_constant__ PackedParams p) {
  constexpr int V = D / 32;
  const dit_packed_attention& a = p.a;
  pdl_wait();
  pdl_trigger();
  const long long unit = (long long)blockIdx.x * 8 + (threadIdx.x >> 5), units = (long long)a.q_rows * a.heads;
  if (unit >= units) return;
  const int q = int(unit / a.heads), head = int(unit - (long long)q * a.heads), lane = lane_id();
  if (a.q_start) {  // rows of no segment stay as they are
    const int first = max(__ldg(a.q_start), 0), end = min(__ldg(a.q_start + a.segments), a.q_rows);
    if (q < first || q >= end) return;
  }
  float2 ml = make_float2(-INFINITY, 0.f);
  if (lane < p.splits) ml = p.part_ml[((long long)lane * a.q_rows + q) * a.heads + head];
  float top = ml.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float w = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - top);
  float l = w * ml.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  const unsigned some = __ballot_sync(0xffffffffu, ml.x != -INFINITY);
  float acc[V] = {};
#pragma unroll 4
  for (int z = 0; z < p.splits; ++z) {
    const float wz = __shfl_sync(0xffffffffu, w, z);
    if (!((some >> z) & 1u)) continue;
    const float* src = p.part_o + (((long long)z * a.q_rows + q) * a.heads + head) * D + lane * V;
    if constexpr (V == 4) {
      const float4 v = *reinterpret_cast<const float4*>(src);
      acc[0] = fmaf(v.x, wz, acc[0]); acc[1] = fmaf(v.y, wz, acc[1]);
      acc[2] = fmaf(v.z, wz, acc[2]); acc[3] = fmaf(v.w, wz, acc[3]);
    } else {
      const float2 v = *reinterpret_cast<const float2*>(src);
      acc[0] = fmaf(v.x, wz, acc[0]); acc[1] = fmaf(v.y, wz, acc[1]);
    }
  }
  uint32_t* dst = reinterpret_cast<uint32_t*>(a.o + q * a.o_row + head * a.o_head + lane * V);
#pragma unroll
  for (int v = 0; v < V / 2; ++v) dst[v] = pack_bf16x2(acc[2 * v] * inv, acc[2 * v + 1] * inv);
  if (a.lse && lane == 0)
    a.lse[(long long)head * a.q_rows + q] = l > 0.f || l != l ? (top + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// Tiles, CTAs and key splits of a call. Segments whose rows fit one tile, on average, go to the few-rows kernel, in tiles of
// the average's rows (32 (row, head) pairs at least: a tile's rows are shared memory); so do segments of 1024 keys at most on
// average, where the start and the end of a CTA cost more than K and V read once for two tiles saves (whole tiles against few
// rows: 300 rows and keys 12.5 and 8.5 us, 600 in 24 heads 15.2 and 12.9, 7 x 800 91 and 78, 64 x 583 114 and 104; 1088 in 24
// heads 21.6 and 22.9, 4224 163 and 182). The key range is split where the
// tiles leave SMs idle.
struct PackedPlan {
  int G, rpt, slots, splits;
  bool few;
  long long tiles;
  size_t part_bytes;
};
PackedPlan packed_plan(int q_rows, int k_rows, int segments, int heads, int kv_heads, int d) {
  PackedPlan r{};
  r.G = heads / kv_heads;
  r.rpt = 128 / r.G;
  const bool tall = (long long)q_rows > (long long)segments * r.rpt;
  r.few = !tall || k_rows <= 1024LL * segments;
  if (r.few) r.rpt = std::min(r.rpt, std::max(32 / r.G, std::max(1, int(((long long)q_rows + segments - 1) / segments))));
  const long long rows = (r.few ? 1LL : 2LL) * r.rpt;
  r.tiles = std::min<long long>((q_rows + segments * (rows - 1)) / rows, q_rows);
  const uint32_t q_bytes = uint32_t((r.G * r.rpt + 7) / 8 * 8) * d * 2;
  r.slots = std::min<int>(kRowSlotsMost, int((kRowSmem - 1024 - kRowBars - q_bytes) / (kRowKeys * d * 2)));
  const long long units = r.tiles * kv_heads, sms = std::max(num_sms(), 1);
  const long long keys = k_rows / segments;
  // Few rows, two CTAs to an SM: with fewer tiles than those, one wave of parts of 256 keys at least (1 row, 24 heads, 1088 keys:
  // 16.0 us whole, 10.9 in four; 32 tiles over 4000 keys: 45.2 whole, 15.9 in eight, 22.0 in twelve, which is more than a
  // wave); with more, six waves of parts of 1024 keys at least, which evens out unlike lengths (512 tiles over 2048 to 8192
  // keys: 257 us whole, 229 in four, 253 in eight). Short segments of several tiles:
  // only where there are an eighth of the SMs' tiles at most (600 rows and keys, 24 heads: 12.9 us whole, 22.4 in two; 1000 in
  // one head: 15.6 whole, 13.3 in three). Whole tiles: only where a wave of them would fit twice.
  long long want, least;
  if (!r.few) {
    want = sms / units;
    least = 512;
  } else if (tall && 8 * units > sms) {
    want = least = 1;
  } else if (units <= 2 * sms) {
    want = 2 * sms / units;
    least = 256;
  } else {
    want = (12 * sms + units - 1) / units;
    least = 1024;
  }
  r.splits = int(std::max<long long>(1, std::min<long long>({want, keys / least, (long long)kMaxSplits})));
  r.part_bytes = r.splits > 1 ? (size_t(r.splits) * q_rows * heads * (size_t(d) * 4 + 8) + 255) / 256 * 256 : 0;
  return r;
}

bool packed_map(CUtensorMap* m, const void* base, int d, int heads, int rows, long long head, long long row, int box_heads,
                int box_rows) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(rows)};
  cuuint64_t strides[2] = {cuuint64_t(heads > 1 ? head : d) * 2, cuuint64_t(rows > 1 ? row : d) * 2};
  cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_rows)}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool FEW, int KIND>
int packed_go(const PackedParams& p, const PackedPlan& pl, cudaStream_t st) {
  const dit_packed_attention& a = p.a;
  constexpr int kKeys = FEW ? kRowKeys : 128;
  CUtensorMap tq, tk, tv;
  const bool keys = a.k_rows > 0;  // none: the maps are not read
  if (!packed_map(&tq, a.q, D, a.heads, a.q_rows, a.q_head, a.q_row, pl.G, pl.rpt) ||
      !packed_map(&tk, keys ? a.k : a.q, D, a.kv_heads, keys ? a.k_rows : 1, keys ? a.k_head : a.q_head, a.k_row, 1, kKeys) ||
      !packed_map(&tv, keys ? a.v : a.q, D, a.kv_heads, keys ? a.k_rows : 1, keys ? a.v_head : a.q_head, a.v_row, 1, kKeys))
    return DIT_ECUDA;
  const dim3 grid(unsigned(pl.tiles), unsigned(a.kv_heads), unsigned(p.splits));
  cudaError_t e;
  if constexpr (FEW) {
    auto kern = packed_rows_kernel<D, KIND>;
    if (!smem_attr_once(reinterpret_cast<const void*>(kern), kRowSmem)) return DIT_ECUDA;
    e = launch_pdl(kern, grid, dim3(kRowThreads), kRowSmem, st, 1, tq, tk, tv, p);
  } else {
    using Cfg = PackedCfg<D>;
    auto kern = packed_kernel<D, KIND>;
    if (!smem_attr_once(reinterpret_cast<const void*>(kern), Cfg::kSmem)) return DIT_ECUDA;
    e = launch_pdl(kern, grid, dim3(kPackedThreads), Cfg::kSmem, st, 1, tq, tk, tv, p);
  }
  if (e != cudaSuccess) return DIT_ECUDA;
  if (p.splits > 1) {
    const long long units = (long long)a.q_rows * a.heads;
    if (launch_pdl(packed_join_kernel<D>, dim3(unsigned((units + 7) / 8)), dim3(256), 0, st, 1, p) != cudaSuccess) return DIT_ECUDA;
  }
  return cudaGetLastError() == cudaSuccess ? DIT_OK : DIT_ECUDA;
}

template <int D, bool FEW>
int packed_kind(const PackedParams& p, const PackedPlan& pl, cudaStream_t st) {
  if (p.cap_out > kWideLog2) return packed_go<D, FEW, kWide>(p, pl, st);
  return p.cap_out > 0.f || p.a.slope ? packed_go<D, FEW, kCapped>(p, pl, st) : packed_go<D, FEW, kPlain>(p, pl, st);
}
template <int D>
int packed_rows(const PackedParams& p, const PackedPlan& pl, cudaStream_t st) {
  return pl.few ? packed_kind<D, true>(p, pl, st) : packed_kind<D, false>(p, pl, st);
}

bool packed_al16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool packed_al4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

int packed_sizes(int q_rows, int k_rows, int segments, int heads, int kv_heads, int d) {
  if (q_rows < 0 || k_rows < 0 || segments < 0 || heads < 1 || kv_heads < 1 || d < 1) return DIT_EINVAL;
  if ((d != 64 && d != 128) || heads % kv_heads != 0 || heads / kv_heads > 128 || kv_heads > 65535) return DIT_EUNSUPPORTED;
  // coordinates of a tile's rows stay within 32 bits; a join has a warp per row and head
  if (q_rows > INT_MAX - 256 || k_rows > INT_MAX - 256 || (long long)q_rows * heads > (1LL << 33)) return DIT_EUNSUPPORTED;
  return DIT_OK;
}

}  // namespace
}  // namespace dit

using namespace dit;

extern "C" {

size_t dit_attention_packed_workspace_bytes(int q_rows, int k_rows, int segments, int heads, int kv_heads, int head_dim) {
  if (packed_sizes(q_rows, k_rows, segments, heads, kv_heads, head_dim) != DIT_OK || q_rows == 0 || segments == 0) return 0;
  return packed_plan(q_rows, k_rows, segments, heads, kv_heads, head_dim).part_bytes;
}

}  // extern "C"

namespace dit {

int packed_attention_launch(const dit_packed_attention& a, void* ws, size_t ws_bytes, int* err, cudaStream_t st) {
  PackedPlan pl = packed_plan(a.q_rows, a.k_rows, a.segments, a.heads, a.kv_heads, a.head_dim);
  PackedParams p;
  std::memset(&p, 0, sizeof(p));
  p.a = a;
  p.G = pl.G;
  p.rpt = pl.rpt;
  p.slots = pl.slots;
  p.splits = pl.splits > 1 && ws && ws_bytes >= pl.part_bytes ? pl.splits : 1;
  p.part_o = static_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + size_t(p.splits) * a.q_rows * a.heads * a.head_dim);
  const double log2e = 1.4426950408889634;
  p.scale_log2 = float(a.scale * log2e);
  if (a.cap > 0.f) {
    p.cap_in = float(2.0 * a.scale * log2e / a.cap);
    p.cap_out = float(a.cap * log2e);
    p.cap_arg = float(double(a.scale) / a.cap);
  }
  p.err = err;
  return a.head_dim == 64 ? packed_rows<64>(p, pl, st) : packed_rows<128>(p, pl, st);
}

int packed_attention_check(const dit_packed_attention* a, const void* ws) {
  if (!a) return DIT_EINVAL;
  const int rc = packed_sizes(a->q_rows, a->k_rows, a->segments, a->heads, a->kv_heads, a->head_dim);
  if (rc != DIT_OK) return rc;
  if (!(a->scale > 0.f) || !std::isfinite(a->scale) || !(a->cap >= 0.f) || !std::isfinite(a->cap)) return DIT_EINVAL;
  // what the kernels are handed in log2 units
  if (a->scale > 2e38f || (a->cap > 0.f && (a->cap > 2e38f || !std::isfinite(float(3.0 * a->scale / a->cap))))) return DIT_EINVAL;
  if (a->q_rows == 0 || a->segments == 0) return DIT_OK;
  if (a->segments > 1 && (!a->q_start || !a->k_start)) return DIT_EINVAL;
  if ((a->q_start == nullptr) != (a->k_start == nullptr)) return DIT_EINVAL;
  if (!packed_al4(a->q_start) || !packed_al4(a->k_start) || !packed_al4(a->visible) || !packed_al4(a->slope) ||
      !packed_al4(a->lse) || !packed_al16(ws))
    return DIT_EINVAL;
  struct Side {
    const void* p;
    long long row, head;
    int rows, heads;
  } side[4] = {{a->q, a->q_row, a->q_head, a->q_rows, a->heads},
               {a->k, a->k_row, a->k_head, a->k_rows, a->kv_heads},
               {a->v, a->v_row, a->v_head, a->k_rows, a->kv_heads},
               {a->o, a->o_row, a->o_head, a->q_rows, a->heads}};
  for (const Side& s : side) {
    if (s.rows == 0) continue;
    if (!s.p || !packed_al16(s.p)) return DIT_EINVAL;
    // tensor maps take strides of whole 16 bytes, above zero and below 2^40 bytes
    if (s.rows > 1 && (s.row < 8 || s.row % 8 || s.row >= 1LL << 39)) return DIT_EINVAL;
    if (s.heads > 1 && (s.head < 8 || s.head % 8 || s.head >= 1LL << 39)) return DIT_EINVAL;
  }
  if (a->o == a->q || a->o == a->k || a->o == a->v) return DIT_EINVAL;
  return DIT_OK;
}

}  // namespace dit
