// The arithmetic of microscaled 4-bit matrices, shared by the kernels that write, read and multiply
// them (fp4_layout.h: where their bytes stand). (The conversions are PTX cvt instructions: one rounding each, to
// nearest with ties to even.)
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/dit.h"
#include "fp4_layout.h"
#include "fp4_ptx.cuh"

namespace dit {

// A row's derived factors (NV) from the bits of its largest magnitude A: u = 448 / A maps a block's
// magnitude to its e4m3 scale, t = 2688 / A = 1 / g, g = A / 2688 (448 * 6: the largest scale times the
// largest code). Below 2^-100 the quotients would overflow: such a row counts as zero. An infinity or
// NaN makes g NaN: the row's values, and its products, come out as NaN.
struct Fp4Row {
  float u, t, g;
};
// Called by a whole warp with one value of `bits`: lanes 0 to 2 make one of the three quotients each.
__device__ __forceinline__ Fp4Row fp4_row(uint32_t bits) {
  if (bits < 0x0d800000u) return Fp4Row{0.f, 0.f, 0.f};  // 2^-100
  if (bits >= 0x7f800000u) return Fp4Row{0.f, 0.f, __uint_as_float(0x7fc00000u)};
  const float a = __uint_as_float(bits);
  const int lane = threadIdx.x & 31;
  const float q = __fdiv_rn(lane == 2 ? a : (lane == 1 ? 2688.f : 448.f), lane == 2 ? 2688.f : a);
  return Fp4Row{__shfl_sync(0xffffffffu, q, 0), __shfl_sync(0xffffffffu, q, 1), __shfl_sync(0xffffffffu, q, 2)};
}
// The same by each lane for itself, where the rows of a warp's lanes differ: no lane waits for another.
__device__ __forceinline__ Fp4Row fp4_row_of_lane(uint32_t bits) {
  if (bits < 0x0d800000u) return Fp4Row{0.f, 0.f, 0.f};
  if (bits >= 0x7f800000u) return Fp4Row{0.f, 0.f, __uint_as_float(0x7fc00000u)};
  const float a = __uint_as_float(bits);
  return Fp4Row{__fdiv_rn(448.f, a), __fdiv_rn(2688.f, a), __fdiv_rn(a, 2688.f)};
}

struct Fp4Block {
  uint32_t byte;  // the block scale
  float inv;      // what a value is multiplied with before it is rounded to a code
};

__device__ __forceinline__ float fp4_e4m3(uint32_t byte) {
  uint32_t h;
  asm("{\n.reg .b16 p;\ncvt.u16.u32 p, %1;\ncvt.rn.f16x2.e4m3x2 %0, p;\n}" : "=r"(h) : "r"(byte));
  float f;
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.f32.f16 %0, lo;\n}" : "=f"(f) : "r"(h));
  return f;
}
__device__ __forceinline__ float fp4_e8m0(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte == 0 ? 1u << 22 : byte << 23);
}

__device__ __forceinline__ Fp4Block fp4_block_nv(uint32_t bits, float u, float t) {
  // a row with an infinity or NaN has u = t = 0; only finite products may reach the conversion
  const float v = u > 0.f ? fminf(__fmul_rn(__uint_as_float(bits), u), 448.f) : 0.f;
  uint32_t byte;
  asm("{\n.reg .b16 p;\ncvt.rn.satfinite.e4m3x2.f32 p, %2, %1;\ncvt.u32.u16 %0, p;\n}" : "=r"(byte) : "f"(v), "f"(0.f));
  const float s = fp4_e4m3(byte);
  return Fp4Block{byte, s > 0.f ? __fdiv_rn(t, s) : 0.f};
}
__device__ __forceinline__ Fp4Block fp4_block_mx(uint32_t bits) {
  if (bits >= 0x7f800000u) return Fp4Block{255u, 0.f};
  if (bits == 0u) return Fp4Block{0u, 0.f};
  // floor(log2) of a magnitude below 2^-126 clamps to the same lowest scale
  const int e = max(int(bits >> 23) - 127 - 2, -127);
  return Fp4Block{uint32_t(e + 127), __uint_as_float(uint32_t(127 - e) << 23)};
}

// Eight codes of (pairs of) products, the lower columns first; conversions saturate at 6.
__device__ __forceinline__ uint32_t fp4_codes8(const uint64_t (&y)[4]) {
  uint32_t w;
  asm("{\n.reg .b8 a, b, c, d;\n.reg .f32 l, h;\n"
      "mov.b64 {l, h}, %1;\ncvt.rn.satfinite.e2m1x2.f32 a, h, l;\n"
      "mov.b64 {l, h}, %2;\ncvt.rn.satfinite.e2m1x2.f32 b, h, l;\n"
      "mov.b64 {l, h}, %3;\ncvt.rn.satfinite.e2m1x2.f32 c, h, l;\n"
      "mov.b64 {l, h}, %4;\ncvt.rn.satfinite.e2m1x2.f32 d, h, l;\n"
      "mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(w)
      : "l"(y[0]), "l"(y[1]), "l"(y[2]), "l"(y[3]));
  return w;
}
// 16 values times inv (two products per instruction, each rounded as a single one), rounded to codes: 8
// bytes. inv = 0 gives zero codes whatever the values (a row or block with an infinity or NaN keeps none).
__device__ __forceinline__ uint2 fp4_codes16(const float* v, float inv) {
  const uint64_t i2 = f2_pack(inv, inv);
  uint64_t y[2][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j >> 2][j & 3] = f2_mul(f2_pack(v[2 * j], v[2 * j + 1]), i2);
  const uint2 w = make_uint2(fp4_codes8(y[0]), fp4_codes8(y[1]));
  return inv != 0.f ? w : make_uint2(0u, 0u);
}

__device__ __forceinline__ void fp4_values16(uint2 w, float* v) {
  const uint32_t u[2] = {w.x, w.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p[4];
    asm("{\n.reg .b8 a, b, c, d;\n"
        "mov.b32 {a, b, c, d}, %4;\n"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n}"
        : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
        : "r"(u[h]));
#pragma unroll
    for (int j = 0; j < 4; ++j)
      asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\ncvt.f32.f16 %0, lo;\ncvt.f32.f16 %1, hi;\n}"
          : "=f"(v[8 * h + 2 * j]), "=f"(v[8 * h + 2 * j + 1])
          : "r"(p[j]));
  }
}

// Eight fp32 values of global memory, as one 32-byte access where `whole` (32-byte aligned), else two of 16.
__device__ __forceinline__ void ld_global_8(float (&v)[8], const float* p, bool whole) {
  if (whole) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(p));
  } else {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}
__device__ __forceinline__ bool on_32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
// 32 bytes of global memory (32-byte aligned) in one store
__device__ __forceinline__ void st_global_256(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

}  // namespace dit
