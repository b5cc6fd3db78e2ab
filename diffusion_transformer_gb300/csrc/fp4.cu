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
// 16 values from column c of a row that starts on 16 bytes, zero past cols
template <typename T>
__device__ __forceinline__ Unit<T> unit_load(const T* x, int c, int cols) {
  Unit<T> u;
  if (c + kUnit <= cols) {
#pragma unroll
    for (int h = 0; h < int(sizeof(T)); ++h) {
      const uint4 q = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint8_t*>(x + c) + 16 * h);
      u.w[4 * h] = q.x;
      u.w[4 * h + 1] = q.y;
      u.w[4 * h + 2] = q.z;
      u.w[4 * h + 3] = q.w;
    }
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
// Rows staged in shared memory: a word of padding behind every unit, so that the units of a warp lie on
// different banks. The place of value i, in values:
template <typename T>
__device__ __forceinline__ int staged_at(int i) {
  return i + i / kUnit * int(4 / sizeof(T));
}
template <typename T>
constexpr size_t kStagedUnit = kUnit * sizeof(T) + 4;

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

// Many rows of up to 32 NU units: one warp per row. A lane holds NU units of 16 values (one NV block, half
// an MX block) in registers, so the row is read once, all its loads in flight together, for its largest
// magnitude and for its codes, and no barrier joins the warps. Bound by HBM: the values in, 9/16 byte
// per value out. 4224 x 3072 bf16: 6.7 us, 5.0 TB/s (one CTA of 192 threads per row: 9.5 us; eight units
// per lane where six cover the row: 7.9 us, their registers leaving fewer rows on an SM).
constexpr int kRowWarps = 4;
template <typename T, int FMT, int NU>
__global__ void __launch_bounds__(32 * kRowWarps) fp4_quantize_warp_kernel(const T* x, long long ldx, int rows, int cols,
                                                                           uint8_t* codes, uint8_t* scales,
                                                                           float* row_scale) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x * kRowWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= rows) return;
  x += r * ldx;
  const RowShape<FMT> sh(cols);
  Unit<T> v[NU];
#pragma unroll
  for (int k = 0; k < NU; ++k)
    if (k * 32 < sh.units) v[k] = unit_load(x, (k * 32 + lane) * kUnit, cols);
  float fu = 0.f, ft = 0.f;
  if constexpr (FMT == DIT_FP4_NV) {
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < NU; ++k)
      if (k * 32 < sh.units) m = max(m, unit_max(v[k]));
    const Fp4Row fr = fp4_row(__reduce_max_sync(0xffffffffu, m));
    fu = fr.u;
    ft = fr.t;
    if (lane == 0) row_scale[r] = fr.g;
  }
  uint8_t* crow = codes + (long long)r * fp4_code_row_bytes(cols);
  uint8_t* srow = scales + fp4_scale_row(FMT, r, cols);
#pragma unroll
  for (int k = 0; k < NU; ++k)
    if (k * 32 < sh.units) unit_quantize<T, FMT>(v[k], k * 32 + lane, fu, ft, sh.units, sh.code_units, crow, srow);
}

// Few rows, long rows, or rows off 16 bytes: one CTA per row, NU units per thread and chunk. Rows longer
// than NU units per thread repeat the passes over chunks (NV: the second pass rereads the row, which L2
// holds). A row that starts off 16 bytes (VEC = false) is staged through shared memory with coalesced
// single loads. 4224 x 12288 bf16: 25.5 us, 5.2 TB/s (eight units per thread: 29.5 us); 9216 x 3072 fp32: 20.5 us
// in 32-value blocks, 21.2 in 16-value ones, 6.2 TB/s; 4000 x 5001 fp32, staged: 31 us, 3.0 TB/s (114 us with
// the units read off one bank).
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
  extern __shared__ uint32_t staged[];
  T* sx = reinterpret_cast<T*>(staged);
  const int span = nt * NU;  // units per chunk
  const int chunks = (sh.units + span - 1) / span;
  Unit<T> v[NU];
  auto load = [&](int c) {
    const int c0 = c * span * kUnit;
    if constexpr (!VEC) {
      __syncthreads();
      T t[NU * kUnit];
#pragma unroll
      for (int k = 0; k < NU * kUnit; ++k) {  // all loads in flight before the first is stored
        const int i = int(threadIdx.x) + k * nt;
        t[k] = c0 + i < cols ? x[c0 + i] : T(0.f);
      }
#pragma unroll
      for (int k = 0; k < NU * kUnit; ++k) sx[staged_at<T>(int(threadIdx.x) + k * nt)] = t[k];
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int u = threadIdx.x + k * nt;
      if constexpr (VEC) {
        v[k] = unit_load(x, c0 + u * kUnit, cols);
      } else {
        const uint32_t* w = staged + u * (kStagedUnit<T> / 4);
#pragma unroll
        for (int j = 0; j < int(kUnit * sizeof(T) / 4); ++j) v[k].w[j] = w[j];
      }
    }
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

// `lanes` threads to a row, units of 16 values: 8 code bytes and a scale byte in, 32 or 64
// bytes out, or (VEC = false: rows off 32 bytes) through shared memory in whole lines. Bound by HBM, the
// values out above all. 4224 x 12288 to bf16: 23 us, 5.7 TB/s; 9216 x 3072 to fp32: 20 us, 6.4 TB/s.
template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(256, 6) fp4_dequantize_kernel(const uint8_t* codes, const uint8_t* scales,
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
  __shared__ uint8_t staging[VEC ? 1 : 256 * kStagedUnit<T>];
  T* staged = reinterpret_cast<T*>(staging + (VEC ? 0 : (threadIdx.x - lane) * kStagedUnit<T>));
#pragma unroll 1
  for (int u0 = 0; u0 * kUnit < cols; u0 += lanes) {
    const int u = u0 + lane, c = u * kUnit;
    if (u < units) {
      const uint2 w = *reinterpret_cast<const uint2*>(crow + 8 * u);
      const int byte = srow[fp4_scale_block(FMT == DIT_FP4_NV ? u : u >> 1)];
      float v[kUnit];
      fp4_values16(w, v);
      const float s = FMT == DIT_FP4_NV ? fp4_e4m3(byte) : fp4_e8m0(byte);
#pragma unroll
      for (int j = 0; j < kUnit; ++j) v[j] = FMT == DIT_FP4_NV ? v[j] * s * g : v[j] * s;
      if (VEC && c + kUnit <= cols) {
        uint32_t q[8];
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int j = 0; j < 8; ++j) q[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
          st_global_256(orow + c, q);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = __float_as_uint(v[8 * h + j]);
            st_global_256(orow + c + 8 * h, q);
          }
        }
      } else if (VEC) {
#pragma unroll
        for (int j = 0; j < kUnit; ++j)
          if (c + j < cols) orow[c + j] = T(v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < kUnit; ++j) staged[staged_at<T>(lane * kUnit) + j] = T(v[j]);
      }
    }
    if constexpr (!VEC) {
      __syncthreads();
      const int n = units > 0 ? min(lanes * kUnit, cols - u0 * kUnit) : 0;
      for (int i = lane; i < n; i += lanes) orow[u0 * kUnit + i] = staged[staged_at<T>(i)];
      __syncthreads();
    }
  }
}

template <typename T, int FMT, bool VEC>
cudaError_t quantize_nu(const T* x, long long ldx, const dit_fp4_matrix& m, cudaStream_t st) {
  const int units = fp4_groups(FMT, m.cols) * (FMT == DIT_FP4_NV ? 4 : 8);
  auto go = [&](auto kern, int nu) {
    const int threads = std::min(256, (units + 32 * nu - 1) / (32 * nu) * 32);
    const size_t smem = VEC ? 0 : size_t(threads) * nu * kStagedUnit<T>;
    return launch_pdl(kern, dim3(m.rows), dim3(threads), smem, st, 1, x, ldx, m.cols, m.codes, m.scales, m.row_scale);
  };
  if constexpr (VEC) {
    // a warp per row: 8 units of bf16, 4 of fp32 per lane at most (64 registers of values)
    constexpr int kMost = sizeof(T) == 2 ? 8 : 4;
    if (units <= 32 * kMost && m.rows >= 4 * num_sms()) {
      auto rows = [&](auto kern) {
        return launch_pdl(kern, dim3((m.rows + kRowWarps - 1) / kRowWarps), dim3(32 * kRowWarps), 0, st, 1, x, ldx, m.rows,
                          m.cols, m.codes, m.scales, m.row_scale);
      };
      if (units <= 64) return rows(fp4_quantize_warp_kernel<T, FMT, 2>);
      if (units <= 128) return rows(fp4_quantize_warp_kernel<T, FMT, 4>);
      if constexpr (kMost > 6)
        if (units <= 192) return rows(fp4_quantize_warp_kernel<T, FMT, 6>);
      return rows(fp4_quantize_warp_kernel<T, FMT, kMost>);
    }
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
