// Microscaled 4-bit floating point (e2m1 codes with a scale per block): quantisation and its inverse
// (the product is in fp4_gemm.cu).
//
// A code stands for 0, 0.5, 1, 1.5, 2, 3, 4 or 6 with a sign. Two formats:
//   DIT_FP4_NV  blocks of 16 values, e4m3 block scale s, fp32 scale g per row: value = code * s * g
//   DIT_FP4_MX  blocks of 32 values, block scale 2^e (e8m0): value = code * 2^e
// Every decision of the quantiser is a single IEEE fp32 operation, so a plain fp32 program gives the
// same codes and scales bit for bit.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "fp4.cuh"
#include "fp4.h"
#include "internal.h"
#include "ptx.cuh"

namespace dit {
namespace {

constexpr int kUnit = 16;  // values per thread step: one NV block, half an MX block

// ---------------------------------------------------------------------------------------------
// quantisation
// ---------------------------------------------------------------------------------------------
// 16 consecutive values as they are stored
template <typename T>
struct Unit {
  uint32_t w[kUnit * sizeof(T) / 4];
};
template <typename T>
__device__ __forceinline__ void unit_values(const Unit<T>& u, float (&v)[kUnit]) {
#pragma unroll
  for (int j = 0; j < kUnit; ++j) {
    if constexpr (sizeof(T) == 2)
      v[j] = __uint_as_float(j & 1 ? u.w[j >> 1] & 0xffff0000u : u.w[j >> 1] << 16);
    else
      v[j] = __uint_as_float(u.w[j]);
  }
}
// The bits of the largest magnitude; their order is finite < infinity < NaN.
template <typename T>
__device__ __forceinline__ uint32_t unit_max(const Unit<T>& u) {
  if constexpr (sizeof(T) == 2) {
    uint32_t m[4];  // max.xorsign.abs: the larger magnitude of each half (with a sign that is masked below)
#pragma unroll
    for (int j = 0; j < 4; ++j) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m[j]) : "r"(u.w[2 * j]), "r"(u.w[2 * j + 1]));
    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m[0]) : "r"(m[1]));
    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m[2]) : "r"(m[3]));
    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m[0]) : "r"(m[2]));
    return max(m[0] & 0x7fff0000u, (m[0] << 16) & 0x7fff0000u);
  } else {
    uint32_t m = u.w[0] & 0x7fffffffu;
#pragma unroll
    for (int j = 1; j < kUnit; ++j) m = max(m, u.w[j] & 0x7fffffffu);
    return m;
  }
}
// words[i] <- words[i + bytes / 4] (a byte offset below 16, even), as if the words were one string of bytes
template <int N>
__device__ __forceinline__ void shift_down(uint32_t (&w)[N], int bytes) {
#pragma unroll
  for (int i = 0; i + 2 < N; ++i) w[i] = bytes & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i + 1 < N; ++i) w[i] = bytes & 4 ? w[i + 1] : w[i];
#pragma unroll
  for (int i = 0; i + 1 < N; ++i) w[i] = bytes & 2 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
}

// 16 values from column c of a row, zero past cols. Rows on 16 bytes (VEC) are read as they lie. Others are
// read through the aligned 16-byte words around the values and shifted into place, but for the units whose
// words would reach over either end of the row, which are read value by value.
template <typename T, bool VEC>
__device__ __forceinline__ Unit<T> unit_load(const T* x, int c, int cols) {
  Unit<T> u;
  constexpr int kWords = kUnit * sizeof(T) / 4, kSpill = VEC ? 0 : 16 / int(sizeof(T));
  if ((VEC || c > 0) && c + kUnit + kSpill <= cols) {
    const int off = VEC ? 0 : int(reinterpret_cast<uintptr_t>(x + c) & 15u);
    const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(x + c) - off);
    uint32_t w[kWords + (VEC ? 0 : 4)];
#pragma unroll
    for (int h = 0; h < kWords / 4 + (VEC ? 0 : 1); ++h) {
      const uint4 q = p[h];
      w[4 * h] = q.x;
      w[4 * h + 1] = q.y;
      w[4 * h + 2] = q.z;
      w[4 * h + 3] = q.w;
    }
    if constexpr (!VEC) shift_down(w, off);
#pragma unroll
    for (int j = 0; j < kWords; ++j) u.w[j] = w[j];
  } else {
    using Bits = typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type;
    const Bits* b = reinterpret_cast<const Bits*>(x);
#pragma unroll
    for (int j = 0; j < kUnit; ++j) {
      const uint32_t e = c + j < cols ? b[c + j] : 0u;
      if constexpr (sizeof(T) == 4) u.w[j] = e;
      else u.w[j >> 1] = j & 1 ? u.w[j >> 1] | e << 16 : e;
    }
  }
  return u;
}

// Codes and scale byte of the unit i in v. A group's four scale bytes are gathered in one thread, so every
// lane of the warp takes part.
template <typename T, int FMT>
__device__ __forceinline__ void unit_quantize(const Unit<T>& v, int i, float fu, float ft, int units, int code_units,
                                              uint8_t* crow, uint8_t* srow) {
  uint32_t m = unit_max(v);
  float inv;
  if constexpr (FMT == DIT_FP4_NV) {
    const Fp4Block b = fp4_block_nv(m, fu, ft);
    inv = b.inv;
    uint32_t w = b.byte << (8 * (i & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 1);
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    if (i < units && (i & 3) == 0) *reinterpret_cast<uint32_t*>(srow + fp4_scale_block(i)) = w;
  } else {
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const Fp4Block b = fp4_block_mx(m);
    inv = b.inv;
    uint32_t w = b.byte << (8 * ((i >> 1) & 3));
    w |= __shfl_xor_sync(0xffffffffu, w, 2);
    w |= __shfl_xor_sync(0xffffffffu, w, 4);
    if (i < units && (i & 7) == 0) *reinterpret_cast<uint32_t*>(srow + fp4_scale_block(i >> 1)) = w;
  }
  if (i < code_units) {
    float f[kUnit];
    unit_values(v, f);
    *reinterpret_cast<uint2*>(crow + 8 * i) = fp4_codes16(f, inv);
  }
}

// Sizes of a row's parts. Units run to whole groups of four blocks, so that every scale byte a K = 64
// step of the product may read is written; codes run to whole 32 values.
template <int FMT>
struct RowShape {
  int units, code_units;
  __device__ explicit RowShape(int cols)
      : units(fp4_groups(FMT, cols) * (FMT == DIT_FP4_NV ? 4 : 8)), code_units(int(fp4_code_row_bytes(cols) / 8)) {}
};

// Many rows of up to LANES x NU units: LANES (8, 16 or 32) lanes of a warp per row. A lane holds NU units of 16
// values (one NV block, half an MX block) in registers, so the row is read once, all its loads in flight
// together, for its largest magnitude and for its codes, and no barrier joins the warps. Bound by HBM: the
// values in, 9/16 byte per value out. 4224 x 3072 bf16: 6.7 us, 5.0 TB/s (one CTA of 192 threads per row: 9.5
// us; eight units per lane where six cover the row: 7.9 us, their registers leaving fewer rows on an SM).
// Several short rows share a warp: 100000 x 64 and x 128 bf16 take 12 us between events, 33 with a warp each.
constexpr int kRowWarps = 4;
template <typename T, int FMT, bool VEC, int NU, int LANES>
__global__ void __launch_bounds__(32 * kRowWarps) fp4_quantize_warp_kernel(const T* x, long long ldx, int rows, int cols,
                                                                           uint8_t* codes, uint8_t* scales,
                                                                           float* row_scale) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & (LANES - 1), first = blockIdx.x * (32 * kRowWarps / LANES);
  if (first + int(threadIdx.x & ~31u) / LANES >= rows) return;
  int r = first + int(threadIdx.x) / LANES;
  const bool live = r < rows;  // a warp stays whole: its lanes past the last row hold an empty row
  if (!live) r = 0, cols = 0;
  x += r * ldx;
  const RowShape<FMT> sh(cols);
  Unit<T> v[NU];
#pragma unroll
  for (int k = 0; k < NU; ++k)
    if (LANES < 32 || k * 32 < sh.units) v[k] = unit_load<T, VEC>(x, (k * LANES + lane) * kUnit, cols);
  float fu = 0.f, ft = 0.f;
  if constexpr (FMT == DIT_FP4_NV) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < NU; ++k)
      if (LANES < 32 || k * 32 < sh.units) m = max(m, unit_max(v[k]));
    if constexpr (LANES == 32) {
      m = __reduce_max_sync(0xffffffffu, m);
    } else {
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    }
    const Fp4Row fr = LANES == 32 ? fp4_row(m) : fp4_row_of_lane(m);
    fu = fr.u;
    ft = fr.t;
    if (lane == 0 && live) row_scale[r] = fr.g;
  }
  uint8_t* crow = codes + (long long)r * fp4_code_row_bytes(cols);
  uint8_t* srow = scales + fp4_scale_row(FMT, r, cols);
#pragma unroll
  for (int k = 0; k < NU; ++k)
    if (LANES < 32 || k * 32 < sh.units)
      unit_quantize<T, FMT>(v[k], k * LANES + lane, fu, ft, sh.units, sh.code_units, crow, srow);
}

// Few or long rows: one CTA per row, NU units per thread and chunk. Rows longer than NU units per thread
// repeat the passes over chunks (NV: the second pass rereads the row, which L2 holds).
// 4224 x 12288 bf16: 25.5 us, 5.2 TB/s (eight units per thread: 29.5 us); 9216 x 3072 fp32: 20.5 us in 32-value blocks,
// 21.2 in 16-value ones, 6.2 TB/s. Rows off 16 bytes, one call between events: 4224 x 12288 bf16 at a
// stride of 12289 39 us (MX) and 47 (NV), 4000 x 5001 fp32 25 and 29; through shared memory with single loads
// they took 151, 180, 39 and 37.
template <typename T, int FMT, bool VEC, int NU>
__global__ void __launch_bounds__(256) fp4_quantize_kernel(const T* x, long long ldx, int cols, uint8_t* codes,
                                                           uint8_t* scales, float* row_scale) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x, nt = blockDim.x;
  x += r * ldx;
  const RowShape<FMT> sh(cols);
  uint8_t* crow = codes + (long long)r * fp4_code_row_bytes(cols);
  uint8_t* srow = scales + fp4_scale_row(FMT, r, cols);
  const int span = nt * NU;  // units per chunk
  const int chunks = (sh.units + span - 1) / span;
  Unit<T> v[NU];
  auto load = [&](int c) {
#pragma unroll
    for (int k = 0; k < NU; ++k) v[k] = unit_load<T, VEC>(x, (c * span + k * nt + int(threadIdx.x)) * kUnit, cols);
  };
  float fu = 0.f, ft = 0.f;
  if constexpr (FMT == DIT_FP4_NV) {
    __shared__ uint32_t part[8];
    uint32_t m = 0;
    for (int c = chunks - 1; c >= 0; --c) {  // the first chunk last: it stays in the registers
      load(c);
#pragma unroll
      for (int k = 0; k < NU; ++k) m = max(m, unit_max(v[k]));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = part[0];
    for (int w = 1; w < (nt >> 5); ++w) m = max(m, part[w]);
    const Fp4Row fr = fp4_row(m);
    fu = fr.u;
    ft = fr.t;
    if (threadIdx.x == 0) row_scale[r] = fr.g;
  }
  for (int c = 0; c < chunks; ++c) {
    if (c > 0 || FMT == DIT_FP4_MX) load(c);
#pragma unroll
    for (int k = 0; k < NU; ++k)
      unit_quantize<T, FMT>(v[k], c * span + k * nt + threadIdx.x, fu, ft, sh.units, sh.code_units, crow, srow);
  }
}

// `lanes` threads to a row, units of 16 values: 8 code bytes and a scale byte in, 32 or 64 bytes out. Rows on 32
// bytes (VEC) are stored as they come. Elsewhere a unit straddles aligned 16-byte words: a lane takes the
// end of its neighbour's unit before its own and stores whole words, shifted into place; only the ends of a
// row and of a warp are stored value by value. Bound by HBM, the values out above all. 4224 x 12288 to bf16: 23
// us, 5.7 TB/s; 9216 x 3072 to fp32: 20 us, 6.4 TB/s. Rows off 32 bytes, one call between events: 4224 x 12288
// to bf16 at a stride of 12289 35 us, 4000 x 5001 to fp32 29-31; through shared memory in single values 49-53 and 27-29.
template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(256, VEC ? 6 : 4) fp4_dequantize_kernel(const uint8_t* codes, const uint8_t* scales,
                                                                          const float* row_scale, int rows, int cols,
                                                                          int lanes, T* out, long long ldo) {
  pdl_wait();
  pdl_trigger();
  const int in_cta = int(threadIdx.x) / lanes, lane = int(threadIdx.x) - in_cta * lanes;
  const long long r = (long long)blockIdx.x * (int(blockDim.x) / lanes) + in_cta;
  const int units = r < rows ? (cols + kUnit - 1) / kUnit : 0;
  const uint8_t* crow = codes + r * fp4_code_row_bytes(cols);
  const uint8_t* srow = scales + fp4_scale_row(FMT, int(r), cols);
  const float g = FMT == DIT_FP4_NV && r < rows ? __ldg(row_scale + r) : 1.f;
  T* orow = out + r * ldo;
  constexpr int kWords = kUnit * sizeof(T) / 4;
  const int in_warp = threadIdx.x & 31, in_last = int(blockDim.x) - int(threadIdx.x & ~31u);
  const uint32_t warp = in_last >= 32 ? 0xffffffffu : (1u << in_last) - 1;  // the last warp may be a part of one
#pragma unroll 1
  for (int u0 = 0; u0 * kUnit < cols; u0 += lanes) {  // the same turns for every lane: they exchange values
    const int u = u0 + lane, c = u * kUnit;
    uint32_t q[kWords] = {};
    if (u < units) {
      const uint2 w = *reinterpret_cast<const uint2*>(crow + 8 * u);
      const int byte = srow[fp4_scale_block(FMT == DIT_FP4_NV ? u : u >> 1)];
      float v[kUnit];
      fp4_values16(w, v);
      const float s = FMT == DIT_FP4_NV ? fp4_e4m3(byte) : fp4_e8m0(byte);
#pragma unroll
      for (int j = 0; j < kUnit; ++j) v[j] = FMT == DIT_FP4_NV ? v[j] * s * g : v[j] * s;
#pragma unroll
      for (int j = 0; j < kWords; ++j)
        q[j] = sizeof(T) == 2 ? pack_bf16x2(v[(2 * j) % kUnit], v[(2 * j + 1) % kUnit]) : __float_as_uint(v[j]);
    }
    using Bits = typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type;
    Bits* o = reinterpret_cast<Bits*>(orow + c);
    auto one = [&](int j) { o[j] = Bits(sizeof(T) == 2 && j & 1 ? q[j >> 1] >> 16 : q[j * kWords / kUnit]); };
    const bool whole = u < units && c + kUnit <= cols;
    if constexpr (VEC) {
      if (whole) {
#pragma unroll
        for (int h = 0; h < kWords; h += 8) {
          const uint32_t t[8] = {q[h], q[h + 1], q[h + 2], q[h + 3], q[h + 4], q[h + 5], q[h + 6], q[h + 7]};
          st_global_256(reinterpret_cast<uint32_t*>(o) + h, t);
        }
      }
    } else {
      uint32_t w[4 + kWords];  // the neighbour's last 16 bytes, then this unit
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __shfl_up_sync(warp, q[kWords - 4 + j], 1);
#pragma unroll
      for (int j = 0; j < kWords; ++j) w[4 + j] = q[j];
      if (whole) {
        const int off = int(reinterpret_cast<uintptr_t>(o) & 15u);  // bytes of the first word before this unit
        const bool before = in_warp > 0 && lane > 0;  // the lane below holds the unit before, whole too
        const bool after = in_warp < 31 && lane + 1 < lanes && c + 2 * kUnit <= cols;  // the lane above stores the end
        shift_down(w, (16 - off) & 15);
        uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(o) - off);
        const int skip = off == 0 ? 4 : 0;  // on 16 bytes nothing was shifted: the words start with the unit
#pragma unroll
        for (int h = 0; h < kWords; h += 4)
          if (off == 0 || h > 0 || before)
            p[h / 4] = make_uint4(skip ? w[h + 4] : w[h], skip ? w[h + 5] : w[h + 1], skip ? w[h + 6] : w[h + 2],
                                  skip ? w[h + 7] : w[h + 3]);
        if (off > 0 && !before) {
#pragma unroll
          for (int j = 0; j < 16 / int(sizeof(T)); ++j)
            if (j * int(sizeof(T)) < 16 - off) one(j);
        }
        if (off > 0 && !after) {
#pragma unroll
          for (int j = kUnit - 16 / int(sizeof(T)); j < kUnit; ++j)
            if ((kUnit - j) * int(sizeof(T)) <= off) one(j);
        }
      }
    }
    if (u < units && !whole) {
#pragma unroll
      for (int j = 0; j < kUnit; ++j)
        if (c + j < cols) one(j);
    }
  }
}

template <typename T, int FMT, bool VEC>
cudaError_t quantize_nu(const T* x, long long ldx, const dit_fp4_matrix& m, cudaStream_t st) {
  const int units = fp4_groups(FMT, m.cols) * (FMT == DIT_FP4_NV ? 4 : 8);
  auto go = [&](auto kern, int nu) {
    const int threads = std::min(256, (units + 32 * nu - 1) / (32 * nu) * 32);
    return launch_pdl(kern, dim3(m.rows), dim3(threads), 0, st, 1, x, ldx, m.cols, m.codes, m.scales, m.row_scale);
  };
  // a warp per row: 8 units of bf16, 4 of fp32 per lane at most (64 registers of values)
  constexpr int kMost = sizeof(T) == 2 ? 8 : 4;
  if (units <= 32 * kMost && m.rows >= 4 * num_sms()) {
    auto rows = [&](auto kern, int lanes) {
      const int per_cta = 32 * kRowWarps / lanes;
      return launch_pdl(kern, dim3((m.rows + per_cta - 1) / per_cta), dim3(32 * kRowWarps), 0, st, 1, x, ldx, m.rows,
                        m.cols, m.codes, m.scales, m.row_scale);
    };
    if (units <= 8) return rows(fp4_quantize_warp_kernel<T, FMT, VEC, 1, 8>, 8);
    if (units <= 16) return rows(fp4_quantize_warp_kernel<T, FMT, VEC, 1, 16>, 16);
    if (units <= 64) return rows(fp4_quantize_warp_kernel<T, FMT, VEC, 2, 32>, 32);
    if (units <= 128) return rows(fp4_quantize_warp_kernel<T, FMT, VEC, 4, 32>, 32);
    if constexpr (kMost > 6)
      if (units <= 192) return rows(fp4_quantize_warp_kernel<T, FMT, VEC, 6, 32>, 32);
    return rows(fp4_quantize_warp_kernel<T, FMT, VEC, kMost, 32>, 32);
  }
  // units per thread: few for short rows, whose threads are few already
  if (units <= (sizeof(T) == 4 && m.rows >= 4 * num_sms() ? 128 : 256)) return go(fp4_quantize_kernel<T, FMT, VEC, 1>, 1);
  if constexpr (sizeof(T) == 2)
    if (units > 512) {
      constexpr int kLong = 4;  // (8: 29.5 against 27.4 us on 4224 rows of 12288)
      return go(fp4_quantize_kernel<T, FMT, VEC, kLong>, kLong);
    }
  return go(fp4_quantize_kernel<T, FMT, VEC, 2>, 2);
}
template <typename T, int FMT>
cudaError_t quantize_go(const T* x, long long ldx, const dit_fp4_matrix& m, cudaStream_t st) {
  const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (m.rows == 1 || ldx * (long long)sizeof(T) % 16 == 0);
  return vec ? quantize_nu<T, FMT, true>(x, ldx, m, st) : quantize_nu<T, FMT, false>(x, ldx, m, st);
}
template <typename T, int FMT>
cudaError_t dequantize_go(const dit_fp4_matrix& m, T* out, long long ldo, cudaStream_t st) {
  const int units = (m.cols + kUnit - 1) / kUnit;
  // threads along a row; short rows share a CTA
  const int lanes = std::min(256, units > 128 ? (units + 31) / 32 * 32 : units), rows = units > 128 ? 1 : 256 / lanes;
  const bool vec = reinterpret_cast<uintptr_t>(out) % 32 == 0 && (m.rows == 1 || ldo * (long long)sizeof(T) % 32 == 0);
  auto kern = vec ? fp4_dequantize_kernel<T, FMT, true> : fp4_dequantize_kernel<T, FMT, false>;
  return launch_pdl(kern, dim3(unsigned((m.rows + (long long)rows - 1) / rows)), dim3(lanes * rows), 0, st, 1, m.codes,
                    m.scales, m.row_scale, m.rows, m.cols, lanes, out, ldo);
}

}  // namespace

int fp4_quantize_launch(const void* x, int type, long long ldx, const dit_fp4_matrix& m, cudaStream_t st) {
  cudaError_t e;
  if (type == DIT_BF16) {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(x);
    e = m.format == DIT_FP4_NV ? quantize_go<__nv_bfloat16, DIT_FP4_NV>(p, ldx, m, st)
                               : quantize_go<__nv_bfloat16, DIT_FP4_MX>(p, ldx, m, st);
  } else {
    const float* p = static_cast<const float*>(x);
    e = m.format == DIT_FP4_NV ? quantize_go<float, DIT_FP4_NV>(p, ldx, m, st)
                               : quantize_go<float, DIT_FP4_MX>(p, ldx, m, st);
  }
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? DIT_OK : DIT_ECUDA;
}

int fp4_dequantize_launch(const dit_fp4_matrix& m, void* out, int type, long long ldo, cudaStream_t st) {
  cudaError_t e;
  if (type == DIT_BF16) {
    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(out);
    e = m.format == DIT_FP4_NV ? dequantize_go<__nv_bfloat16, DIT_FP4_NV>(m, p, ldo, st)
                               : dequantize_go<__nv_bfloat16, DIT_FP4_MX>(m, p, ldo, st);
  } else {
    float* p = static_cast<float*>(out);
    e = m.format == DIT_FP4_NV ? dequantize_go<float, DIT_FP4_NV>(m, p, ldo, st)
                               : dequantize_go<float, DIT_FP4_MX>(m, p, ldo, st);
  }
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? DIT_OK : DIT_ECUDA;
}

}  // namespace dit
