// Rotary positions: the values of a head turned pair by pair through angles that grow with the row's
// positions (the gizai:dit reference's prepOf; host contract, section 4), for any head width, a
// rotated part of the head, several position axes, adjacent-pair and split-halves layouts, and
// frequencies rescaled for sequences longer than the trained ones.
//
// Mathematics. Pair i of a head belongs to position axis a(i) and turns by p_a f_i radians; with
// u_i = f_i / 2 pi (turns per position, below 1) as a 64-bit binary fraction U_i = rint(2^64 u_i), the
// angle modulo one turn is the low 64 bits of p U_i: one integer product, exact for every 32-bit
// position of either sign, so far positions lose nothing (|error| <= |p| 2^-65 turns: 2^-34 at the
// last 32-bit position). The nearest quarter turn is taken off in integers before the conversion to
// fp32, so the residual, at most an eighth of a turn, carries 24 bits (2^-28 turns) into sincospif.
//
// What bounds it: HBM. Each value is read once and written once; a row's cosines and sines are
// computed once into shared memory and serve all of its heads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "internal.h"
#include "ptx.cuh"

namespace dit {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotUnroll = 4;  // units in flight per thread

struct RotArgs {
  const void* x[2];
  void* out[2];
  long long xb[2], xr[2], xh[2], ob[2], orow[2], oh[2];  // strides in values
  int heads[2];
  int copy[2];       // values behind the rotated part are copied (not in place)
  int rows;          // rows per batch entry
  long long total;   // batch * rows
  int rows_per_cta;
  int head_dim;
  int lanes_log2;    // threads along one head (a power of two, at least the units of a head)
  int inverse;
  const int32_t* pos;
  dit_rotary_plan plan;
};

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

template <int N>
__device__ __forceinline__ void rot_load(float (&v)[N], const __nv_bfloat16* p) {
  if constexpr (N == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = __bfloat162float(p[j]);
  }
}
template <int N>
__device__ __forceinline__ void rot_load(float (&v)[N], const float* p) {
  if constexpr (N == 4) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = p[j];
  }
}
template <int N>
__device__ __forceinline__ void rot_store(__nv_bfloat16* p, const float (&v)[N]) {
  if constexpr (N == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) p[j] = __float2bfloat16_rn(v[j]);
  }
}
template <int N>
__device__ __forceinline__ void rot_store(float* p, const float (&v)[N]) {
  if constexpr (N == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) p[j] = v[j];
  }
}

// A unit is what one thread turns: VE consecutive values (adjacent pairs; two values when VE = 1), or
// VE values of the first half and their VE partners in the second, or VE values that pass unturned.
// VE = 16 bytes' worth of values where every row and head starts on 16 bytes and the rotated part ends
// on such a boundary, else 1. blockIdx.x: rows, blockIdx.y: which of q and k.
template <typename T, int VE, bool HALVES>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotArgs a) {
  constexpr int kTurn = HALVES ? VE : (VE == 1 ? 1 : VE / 2);  // pairs per turned unit
  constexpr int kA = HALVES ? VE : (VE == 1 ? 2 : VE);         // values of a turned unit's first load
  constexpr int kAll = HALVES ? 2 * VE : kA;
  extern __shared__ float2 cs[];  // [rows_per_cta][pairs]
  const int pairs = a.plan.pairs;
  const long long row0 = (long long)blockIdx.x * a.rows_per_cta;
  const int nrows = int(a.total - row0 < a.rows_per_cta ? a.total - row0 : a.rows_per_cta);
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < nrows * pairs; i += kRotThreads) {
    const int rr = i / pairs, k = i - rr * pairs;
    const int32_t p = __ldg(a.pos + (row0 + rr) * a.plan.axes + a.plan.axis[k]);
    float2 v = rot_cos_sin(p, a.plan.turns[k], a.plan.amplitude);
    if (a.inverse) v.y = -v.y;
    cs[i] = v;
  }
  __syncthreads();
  const int z = blockIdx.y;
  const int unit = threadIdx.x & ((1 << a.lanes_log2) - 1);
  const int group = threadIdx.x >> a.lanes_log2, groups = kRotThreads >> a.lanes_log2;
  const int turned = pairs / kTurn;
  const int tail = a.copy[z] ? (a.head_dim - 2 * pairs) / VE : 0;
  if (unit >= turned + tail) return;
  const bool turn = unit < turned;
  const int off = turn ? (HALVES ? unit * VE : unit * kA) : 2 * pairs + (unit - turned) * VE;
  const T* x = static_cast<const T*>(a.x[z]);
  T* out = static_cast<T*>(a.out[z]);
  const int H = a.heads[z];
  // one (row, head) after another, kRotUnroll of them loaded before the first is turned
  for (int g0 = group; g0 < nrows * H; g0 += groups * kRotUnroll) {
    float v[kRotUnroll][kAll];
    long long dst[kRotUnroll];
    int rr_[kRotUnroll];
#pragma unroll
    for (int u = 0; u < kRotUnroll; ++u) {
      const int g = g0 + u * groups;
      if (g < nrows * H) {
        const int rr = g / H, h = g - rr * H;
        const long long r = row0 + rr;
        const long long b = r / a.rows, t = r - b * a.rows;
        const long long src = b * a.xb[z] + t * a.xr[z] + h * a.xh[z] + off;
        dst[u] = b * a.ob[z] + t * a.orow[z] + h * a.oh[z] + off;
        rr_[u] = rr;
        if (turn) {
          float p0[kA];
          rot_load<kA>(p0, x + src);
#pragma unroll
          for (int j = 0; j < kA; ++j) v[u][j] = p0[j];
          if constexpr (HALVES) {
            rot_load<kA>(p0, x + src + pairs);
#pragma unroll
            for (int j = 0; j < kA; ++j) v[u][kA + j] = p0[j];
          }
        } else {
          float p0[VE];
          rot_load<VE>(p0, x + src);
#pragma unroll
          for (int j = 0; j < VE; ++j) v[u][j] = p0[j];
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kRotUnroll; ++u) {
      const int g = g0 + u * groups;
      if (g < nrows * H) {
        if (turn) {
          const float2* c = cs + rr_[u] * pairs + unit * kTurn;
          float w0[kA], w1[kA];
#pragma unroll
          for (int j = 0; j < kTurn; ++j) {
            const float2 t = c[j];
            if constexpr (HALVES) {
              w0[j] = v[u][j] * t.x - v[u][kA + j] * t.y;
              w1[j] = v[u][j] * t.y + v[u][kA + j] * t.x;
            } else {
              w0[2 * j] = v[u][2 * j] * t.x - v[u][2 * j + 1] * t.y;
              w0[2 * j + 1] = v[u][2 * j] * t.y + v[u][2 * j + 1] * t.x;
            }
          }
          rot_store<kA>(out + dst[u], w0);
          if constexpr (HALVES) rot_store<kA>(out + dst[u] + pairs, w1);
        } else {
          float p0[VE];
#pragma unroll
          for (int j = 0; j < VE; ++j) p0[j] = v[u][j];
          rot_store<VE>(out + dst[u], p0);
        }
      }
    }
  }
}

__global__ void __launch_bounds__(kRotThreads) rotary_tables_kernel(const __grid_constant__ dit_rotary_plan plan,
                                                                    const int32_t* pos, long long n, float* cos,
                                                                    float* sin) {
  pdl_wait();
  pdl_trigger();
  const long long i = (long long)blockIdx.x * kRotThreads + threadIdx.x;
  if (i >= n) return;
  const long long r = i / plan.pairs;
  const int k = int(i - r * plan.pairs);
  const float2 v = rot_cos_sin(__ldg(pos + r * plan.axes + plan.axis[k]), plan.turns[k], plan.amplitude);
  cos[i] = v.x;
  sin[i] = v.y;
}

template <typename T, int VE>
cudaError_t rotary_go(const RotArgs& a, dim3 grid, size_t smem, cudaStream_t st) {
  return a.plan.layout == DIT_ROTARY_HALVES
             ? launch_pdl(rotary_kernel<T, VE, true>, grid, dim3(kRotThreads), smem, st, 1, a)
             : launch_pdl(rotary_kernel<T, VE, false>, grid, dim3(kRotThreads), smem, st, 1, a);
}

bool plan_ok(const dit_rotary_plan* p) {
  if (!p || p->pairs < 1 || p->pairs > DIT_ROTARY_MAX_PAIRS || p->axes < 1 || p->axes > DIT_ROTARY_MAX_AXES) return false;
  if (p->layout != DIT_ROTARY_PAIRS && p->layout != DIT_ROTARY_HALVES) return false;
  for (int i = 0; i < p->pairs; ++i)
    if (p->axis[i] >= p->axes) return false;
  return true;
}

}  // namespace
}  // namespace dit

using namespace dit;

extern "C" {

int dit_rotary_plan_init(const dit_rotary_spec* s, dit_rotary_plan* plan) {
  if (!s || !plan) return DIT_EINVAL;
  if (s->axes < 1 || s->axes > DIT_ROTARY_MAX_AXES || !(s->theta > 1.0) || !std::isfinite(s->theta)) return DIT_EINVAL;
  if (s->layout != DIT_ROTARY_PAIRS && s->layout != DIT_ROTARY_HALVES) return DIT_EINVAL;
  if (s->scaling < DIT_ROTARY_UNSCALED || s->scaling > DIT_ROTARY_YARN) return DIT_EINVAL;
  if (s->scaling != DIT_ROTARY_UNSCALED && !(s->factor >= 1.0 && std::isfinite(s->factor))) return DIT_EINVAL;
  if (s->scaling == DIT_ROTARY_YARN &&
      (s->original < 1 || !(s->beta_slow > 0.0) || !(s->beta_fast >= s->beta_slow) || !std::isfinite(s->beta_fast)))
    return DIT_EINVAL;
  int pairs = 0;
  for (int a = 0; a < s->axes; ++a) {
    if (s->width[a] < 2 || s->width[a] % 2 != 0 || s->width[a] > 2 * DIT_ROTARY_MAX_PAIRS) return DIT_EINVAL;
    pairs += s->width[a] / 2;
  }
  if (pairs > DIT_ROTARY_MAX_PAIRS) return DIT_EUNSUPPORTED;
  dit_rotary_plan p;
  std::memset(&p, 0, sizeof(p));
  p.pairs = pairs;
  p.axes = s->axes;
  p.layout = s->layout;
  p.amplitude = 1.f;
  const double two_pi = 6.283185307179586476925286766559;
  int i = 0;
  for (int a = 0; a < s->axes; ++a) {
    const int w = s->width[a];
    double theta = s->theta;
    if (s->scaling == DIT_ROTARY_NTK && w > 2) theta *= std::pow(s->factor, double(w) / (w - 2));
    double lo = 0, span = 1;
    if (s->scaling == DIT_ROTARY_YARN) {
      auto at = [&](double turns) { return w * std::log(s->original / (turns * two_pi)) / (2 * std::log(theta)); };
      lo = std::fmax(0.0, std::floor(at(s->beta_fast)));
      const double hi = std::fmin(double(w / 2 - 1), std::ceil(at(s->beta_slow)));
      span = std::fmax(hi - lo, 1e-3);
      p.amplitude = float(0.1 * std::log(s->factor) + 1.0);
    }
    for (int k = 0; k < w / 2; ++k, ++i) {
      double f = std::pow(theta, -2.0 * k / w);
      if (s->scaling == DIT_ROTARY_LINEAR) f /= s->factor;
      if (s->scaling == DIT_ROTARY_YARN) {
        const double ramp = std::fmin(1.0, std::fmax(0.0, (k - lo) / span));
        f = f * (1.0 - ramp) + f / s->factor * ramp;
      }
      p.turns[i] = (uint64_t)std::llrint(std::ldexp(f / two_pi, 62)) << 2;  // below 2^62 turns: no overflow
      p.axis[i] = uint8_t(a);
    }
  }
  *plan = p;
  return DIT_OK;
}

int dit_rotary_tables(const dit_rotary_plan* plan, const int32_t* pos, int rows, float* cos, float* sin,
                      dit_stream_t stream) {
  if (!plan_ok(plan) || rows < 0) return DIT_EINVAL;
  if (rows == 0) return DIT_OK;
  if (!pos || !cos || !sin) return DIT_EINVAL;
  const long long n = (long long)rows * plan->pairs;
  if (launch_pdl(rotary_tables_kernel, dim3(unsigned((n + kRotThreads - 1) / kRotThreads)), dim3(kRotThreads), 0,
                 reinterpret_cast<cudaStream_t>(stream), 1, *plan, pos, n, cos, sin) != cudaSuccess)
    return DIT_ECUDA;
  return cudaGetLastError() == cudaSuccess ? DIT_OK : DIT_ECUDA;
}

int dit_rotary(const dit_rotary_plan* plan, const dit_rotary_rows* q, const dit_rotary_rows* k, int type, int batch,
               int rows, int head_dim, const int32_t* pos, int inverse, dit_stream_t stream) {
  if (!plan_ok(plan) || !q || batch < 0 || rows < 0 || (type != DIT_BF16 && type != DIT_F32)) return DIT_EINVAL;
  if (head_dim < 2 * plan->pairs) return DIT_EINVAL;
  if (head_dim > 2 * DIT_ROTARY_MAX_PAIRS) return DIT_EUNSUPPORTED;
  const dit_rotary_rows* part[2] = {q, k};
  const int size = type == DIT_BF16 ? 2 : 4, ve = 16 / size;
  for (const dit_rotary_rows* r : part)
    if (r && r->heads < 0) return DIT_EINVAL;
    else if (r && r->heads > 1 << 20) return DIT_EUNSUPPORTED;
  if (batch == 0 || rows == 0) return DIT_OK;
  if (!pos) return DIT_EINVAL;
  RotArgs a;
  std::memset(&a, 0, sizeof(a));
  int n = 0;
  bool vec = head_dim % ve == 0 && (plan->layout == DIT_ROTARY_HALVES ? plan->pairs : 2 * plan->pairs) % ve == 0;
  for (const dit_rotary_rows* r : part) {
    if (!r || r->heads == 0) continue;
    if (!r->x || !r->out || reinterpret_cast<uintptr_t>(r->x) % size || reinterpret_cast<uintptr_t>(r->out) % size)
      return DIT_EINVAL;
    // rows that share their place in the output would race
    if ((batch > 1 && r->out_batch == 0) || (rows > 1 && r->out_row == 0) || (r->heads > 1 && r->out_head == 0))
      return DIT_EINVAL;
    a.x[n] = r->x;
    a.out[n] = r->out;
    a.xb[n] = r->x_batch;
    a.xr[n] = r->x_row;
    a.xh[n] = r->x_head;
    a.ob[n] = r->out_batch;
    a.orow[n] = r->out_row;
    a.oh[n] = r->out_head;
    a.heads[n] = r->heads;
    const bool same = r->x == r->out && (rows == 1 || r->x_row == r->out_row) &&
                      (r->heads == 1 || r->x_head == r->out_head) && (batch == 1 || r->x_batch == r->out_batch);
    a.copy[n] = !same;
    auto on16 = [&](const void* p, long long s0, long long s1, long long s2) {
      return reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 % ve == 0 && s1 % ve == 0 && s2 % ve == 0;
    };
    vec = vec && on16(r->x, batch > 1 ? r->x_batch : 0, rows > 1 ? r->x_row : 0, r->heads > 1 ? r->x_head : 0) &&
          on16(r->out, batch > 1 ? r->out_batch : 0, rows > 1 ? r->out_row : 0, r->heads > 1 ? r->out_head : 0);
    ++n;
  }
  if (n == 0) return DIT_OK;
  a.rows = rows;
  a.total = (long long)batch * rows;
  a.head_dim = head_dim;
  a.inverse = inverse != 0;
  a.pos = pos;
  a.plan = *plan;
  const int v = vec ? ve : 1;
  const int turned = plan->pairs / (plan->layout == DIT_ROTARY_HALVES ? v : (v == 1 ? 1 : v / 2));
  const int units = turned + (head_dim - 2 * plan->pairs) / v;
  while ((1 << a.lanes_log2) < units) ++a.lanes_log2;
  a.rows_per_cta = 2;
  const long long ctas = (a.total + a.rows_per_cta - 1) / a.rows_per_cta;
  if (ctas > 0x7fffffffLL) return DIT_EUNSUPPORTED;
  const dim3 grid{unsigned(ctas), unsigned(n), 1u};
  const size_t smem = size_t(a.rows_per_cta) * plan->pairs * sizeof(float2);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (type == DIT_BF16)
    e = vec ? rotary_go<__nv_bfloat16, 8>(a, grid, smem, st) : rotary_go<__nv_bfloat16, 1>(a, grid, smem, st);
  else
    e = vec ? rotary_go<float, 4>(a, grid, smem, st) : rotary_go<float, 1>(a, grid, smem, st);
  if (e != cudaSuccess) return DIT_ECUDA;
  return cudaGetLastError() == cudaSuccess ? DIT_OK : DIT_ECUDA;
}

}  // extern "C"
