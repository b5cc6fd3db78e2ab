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

#include "fp4.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace dit {
namespace {

constexpr int kUnit = 16;  // values per thread step: one NV block, half an MX block

// ---------------------------------------------------------------------------------------------
// quantisation
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// 16 values of row x from column c on (zero past cols) as fp32
template <typename T, bool VEC>
__device__ __forceinline__ void load16(float (&v)[kUnit], const T* x, int c, int cols) {
  if (VEC && c + kUnit <= cols) {
    if constexpr (sizeof(T) == 2) {
      uint32_t w[8];
      ld_global_256(w, x + c);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    } else {
      uint32_t w[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ld_global_256(w, x + c + 8 * h);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[8 * h + j] = __uint_as_float(w[j]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kUnit; ++j) v[j] = c + j < cols ? float(x[c + j]) : 0.f;
  }
}

__device__ __forceinline__ uint32_t unit_max(const float (&v)[kUnit]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kUnit; ++j) m = max(m, abs_bits(v[j]));  // bit order: finite < inf < NaN
  return m;
}

// One row per CTA. A thread takes units of 16 values; the row is read once for its largest magnitude
// (NV) and again, out of L1/L2, for the codes. Units run to whole groups of four blocks, so that
// every scale byte a K = 64 step of the product may read is written; codes run to whole 32 values.
template <typename T, int FMT, bool VEC>
__global__ void __launch_bounds__(256) fp4_quantize_kernel(const T* x, long long ldx, int cols, uint8_t* codes,
                                                           uint8_t* scales, float* row_scale) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x;
  x += r * ldx;
  const int code_units = fp4_code_row_bytes(cols) / 8;              // 8 code bytes per unit
  const int units = fp4_groups(FMT, cols) * (FMT == DIT_FP4_NV ? 4 : 8);
  uint8_t* crow = codes + (long long)r * fp4_code_row_bytes(cols);
  uint8_t* srow = scales + fp4_scale_row(FMT, r, cols);
  float u = 0.f, t = 0.f, g = 0.f;
  __shared__ uint32_t part[8];
  if constexpr (FMT == DIT_FP4_NV) {
    uint32_t m = 0;
    for (int i = threadIdx.x; i * kUnit < cols; i += blockDim.x) {
      float v[kUnit];
      load16<T, VEC>(v, x, i * kUnit, cols);
      m = max(m, unit_max(v));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
    __syncthreads();
    m = 0;
    for (int w = 0; w < int(blockDim.x >> 5); ++w) m = max(m, part[w]);
    const Fp4Row fr = fp4_row(m);
    u = fr.u;
    t = fr.t;
    g = fr.g;
    if (threadIdx.x == 0) row_scale[r] = g;
  }
  const int rounds = (units + blockDim.x - 1) / blockDim.x;  // whole warps stay together for the shuffle
  for (int k = 0; k < rounds; ++k) {
    const int i = threadIdx.x + k * blockDim.x;
    float v[kUnit];
#pragma unroll
    for (int j = 0; j < kUnit; ++j) v[j] = 0.f;
    if (i * kUnit < cols) load16<T, VEC>(v, x, i * kUnit, cols);
    uint32_t m = unit_max(v);
    float inv;
    if constexpr (FMT == DIT_FP4_NV) {
      const Fp4Block b = fp4_block_nv(m, u, t);
      inv = b.inv;
      if (i < units) srow[fp4_scale_block(i)] = uint8_t(b.byte);
    } else {
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      const Fp4Block b = fp4_block_mx(m);
      inv = b.inv;
      if (i < units && (i & 1) == 0) srow[fp4_scale_block(i >> 1)] = uint8_t(b.byte);
    }
    if (i < code_units) {
      uint32_t w[2];
      fp4_codes16(v, inv, w);
      *reinterpret_cast<uint2*>(crow + 8 * i) = make_uint2(w[0], w[1]);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) fp4_dequantize_kernel(int fmt, const uint8_t* codes, const uint8_t* scales,
                                                             const float* row_scale, long long n_units, int row_units,
                                                             int cols, T* out, long long ldo, bool vec) {
  pdl_wait();
  pdl_trigger();
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= n_units) return;
  const long long r = i / row_units;
  const int u = int(i - r * row_units), c = u * kUnit;
  const uint2 w = *reinterpret_cast<const uint2*>(codes + r * fp4_code_row_bytes(cols) + 8 * u);
  const int byte = scales[fp4_scale_row(fmt, int(r), cols) + fp4_scale_block(fmt == DIT_FP4_NV ? u : u >> 1)];
  float v[kUnit];
  fp4_values16(w, v);
  if (fmt == DIT_FP4_NV) {
    const float s = fp4_e4m3(byte), g = row_scale[r];
#pragma unroll
    for (int j = 0; j < kUnit; ++j) v[j] = v[j] * s * g;
  } else {
    const float s = fp4_e8m0(byte);
#pragma unroll
    for (int j = 0; j < kUnit; ++j) v[j] *= s;
  }
  T* o = out + r * ldo + c;
  if (vec && c + kUnit <= cols) {
    if constexpr (sizeof(T) == 2) {
      uint4* d = reinterpret_cast<uint4*>(o);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        d[h] = make_uint4(pack_bf16x2(v[8 * h], v[8 * h + 1]), pack_bf16x2(v[8 * h + 2], v[8 * h + 3]),
                          pack_bf16x2(v[8 * h + 4], v[8 * h + 5]), pack_bf16x2(v[8 * h + 6], v[8 * h + 7]));
    } else {
      float4* d = reinterpret_cast<float4*>(o);
#pragma unroll
      for (int h = 0; h < 4; ++h) d[h] = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
    }
  } else {
    for (int j = 0; j < kUnit && c + j < cols; ++j) o[j] = T(v[j]);
  }
}

template <typename T, int FMT>
cudaError_t quantize_go(const T* x, long long ldx, const dit_fp4_matrix& m, cudaStream_t st) {
  const int units = fp4_groups(FMT, m.cols) * (FMT == DIT_FP4_NV ? 4 : 8);
  const int threads = units >= 256 ? 256 : (units + 31) / 32 * 32;
  const bool vec = reinterpret_cast<uintptr_t>(x) % 32 == 0 && ldx * (long long)sizeof(T) % 32 == 0;
  return vec ? launch_pdl(fp4_quantize_kernel<T, FMT, true>, dim3(m.rows), dim3(threads), 0, st, 1, x, ldx, m.cols,
                          m.codes, m.scales, m.row_scale)
             : launch_pdl(fp4_quantize_kernel<T, FMT, false>, dim3(m.rows), dim3(threads), 0, st, 1, x, ldx, m.cols,
                          m.codes, m.scales, m.row_scale);
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
  const int row_units = (m.cols + kUnit - 1) / kUnit;
  const long long n = (long long)m.rows * row_units;
  const long long ctas = (n + 255) / 256;
  if (ctas > 0x7fffffffLL) return DIT_EUNSUPPORTED;
  const int size = type == DIT_BF16 ? 2 : 4;
  const bool vec = reinterpret_cast<uintptr_t>(out) % 16 == 0 && ldo * size % 16 == 0;
  const cudaError_t e =
      type == DIT_BF16
          ? launch_pdl(fp4_dequantize_kernel<__nv_bfloat16>, dim3(unsigned(ctas)), dim3(256), 0, st, 1, m.format, m.codes,
                       m.scales, m.row_scale, n, row_units, m.cols, static_cast<__nv_bfloat16*>(out), ldo, vec)
          : launch_pdl(fp4_dequantize_kernel<float>, dim3(unsigned(ctas)), dim3(256), 0, st, 1, m.format, m.codes,
                       m.scales, m.row_scale, n, row_units, m.cols, static_cast<float*>(out), ldo, vec);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? DIT_OK : DIT_ECUDA;
}

}  // namespace dit
