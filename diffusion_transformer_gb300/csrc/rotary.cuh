// What the rotary operators share: an angle's cosine and sine, rows in 16-byte or single accesses, a plan's checks.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "../../include/dit.h"
#include "ptx.cuh"

namespace dit {

// cos and sin of p U / 2^64 turns, times the amplitude
__device__ __forceinline__ float2 rot_cos_sin(long long p, unsigned long long U, float amp) {
  const unsigned long long t = (unsigned long long)p * U;  // modulo one turn
  const unsigned q = unsigned((t + (1ull << 61)) >> 62);   // nearest quarter turn
  const long long r = (long long)(t - ((unsigned long long)q << 62));
  float s, c;
  sincospif(float(r) * 0x1p-63f, &s, &c);  // 2 r / 2^64 half turns
  const float cc = (q & 1) ? s : c, ss = (q & 1) ? c : s;
  // quarter turns: (c, s), (-s, c), (-c, -s), (s, -c)
  return make_float2((q == 1 || q == 2) ? -cc * amp : cc * amp, (q == 2 || q == 3) ? -ss * amp : ss * amp);
}

// VE consecutive values as they are stored: one 16-byte access, or one value
template <typename T, int VE>
struct Raw {
  uint4 u;
};
template <typename T>
struct Raw<T, 1> {
  T u;
};
template <typename T, int VE>
__device__ __forceinline__ Raw<T, VE> rot_load(const T* p) {
  Raw<T, VE> r;
  if constexpr (VE == 1) r.u = *p;
  else r.u = *reinterpret_cast<const uint4*>(p);
  return r;
}
template <typename T, int VE>
__device__ __forceinline__ void rot_store(T* p, const Raw<T, VE>& r) {
  if constexpr (VE == 1) *p = r.u;
  else *reinterpret_cast<uint4*>(p) = r.u;
}
template <typename T, int VE>
__device__ __forceinline__ void rot_values(const Raw<T, VE>& r, float (&v)[VE]) {
  if constexpr (VE == 1) {
    v[0] = float(r.u);
  } else {
    const uint32_t w[4] = {r.u.x, r.u.y, r.u.z, r.u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (VE == 8) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      } else {
        v[j] = __uint_as_float(w[j]);
      }
    }
  }
}
template <typename T, int VE>
__device__ __forceinline__ Raw<T, VE> rot_raw(const float (&v)[VE]) {
  Raw<T, VE> r;
  if constexpr (VE == 1) r.u = T(v[0]);
  else if constexpr (VE == 8)
    r.u = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  else
    r.u = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  return r;
}

inline bool al4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

inline bool plan_ok(const dit_rotary_plan* p) {
  if (!p || p->pairs < 1 || p->pairs > DIT_ROTARY_MAX_PAIRS || p->axes < 1 || p->axes > DIT_ROTARY_MAX_AXES) return false;
  if (p->layout != DIT_ROTARY_PAIRS && p->layout != DIT_ROTARY_HALVES) return false;
  for (int i = 0; i < p->pairs; ++i)
    if (p->axis[i] >= p->axes) return false;
  return true;
}

}  // namespace dit
