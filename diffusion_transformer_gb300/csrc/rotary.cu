// Rotary positions: the values of a head turned pair by pair through angles that grow with the row's
// positions (the gizai:dit reference's prepOf; host contract, section 4), for any head width, a
// rotated part of the head, several position axes, adjacent-pair and split-halves layouts, and
// frequencies rescaled for sequences longer than the trained ones.
//
// Mathematics. Pair i of a head belongs to position axis a(i) and turns by p_a f_i radians; with
// u_i = f_i / 2 pi (turns per position, below 1) as a 64-bit binary fraction U_i, the angle modulo one turn is
// the low 64 bits of p U_i: one integer product, exact for every 32-bit position of either sign. U_i itself comes of
// 64-bit floating point (a power and a quotient, then rounded at 2^-62): off by less than 2^-54 turns, most by
// 2^-56, so an angle is off by |p| 2^-54 turns: 2^-30 at 2^24 positions, below what fp32 keeps of it, and 2^-23 at the
// last 32-bit position. The nearest quarter turn is taken off in integers before the conversion to
// fp32, so the residual, at most an eighth of a turn, carries 24 bits (2^-28 turns) into sincospif.
//
// What bounds it: HBM. Each value is read once and written once; a row's cosines and sines are
// computed once into shared memory and serve all of its heads. 131072 rows of 10 heads (96 of 128 values
// turned, bf16, written head-major): 109 us, 6.2 TB/s; 4224 rows of 48 heads out of packed QKV rows: 18.5 us,
// 5.6 TB/s; one row: 3.8 us, the launch and one chain of loads.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "internal.h"
#include "ptx.cuh"
#include "rotary.cuh"

namespace dit {
namespace {

constexpr int kRotThreads = 256;
// rows in flight per thread: two where a row is four 16-byte accesses, which leaves room for five CTAs
// (two against four: 131 against 146 us on 131072 rows of 10 heads)
__host__ __device__ constexpr int rot_unroll(bool wide) { return wide ? 2 : 4; }
constexpr int kRotMaxRows = 32;  // rows per CTA at most

constexpr int kRotPad = 2;

struct RotArgs {
  const void* x[2];
  void* out[2];
  long long xb[2], xr[2], xh[2], ob[2], orow[2], oh[2];  // strides in values
  int q_heads, heads;  // q's, q's and k's together
  int copy[2];         // values behind the rotated part are copied (not in place)
  int rows;            // rows per batch entry
  int rows_per_cta, row_ctas;           // row_ctas CTAs per batch entry
  int units, turned_units, row_units;  // units of a head, turned units of a row, units of a row
  int groups;            // rows taken at a time (1 where a row has more units than the CTA threads)
  int inverse;
  const int32_t* pos;
  dit_rotary_plan plan;
};

// A unit is what one thread turns: VE consecutive values in the adjacent-pair layout (two values when
// VE = 1), VE values of the first half and their VE partners in the second, or VE values that pass
// unturned. VE = 16 bytes' worth of values where every row and head starts on 16 bytes and the rotated
// part ends on such a boundary, else 1.
// A CTA takes rows_per_cta rows of one batch entry. A thread keeps one unit of one head (of q or k) through
// the rows, so its addresses are worked out once; it then goes on to its next unit. The turned units of
// all heads come first and the passing ones after them, so a warp rarely holds both kinds. Rows with fewer
// units than threads are taken several at a time. A few rows are loaded before the first is turned, and
// the first of them before the CTA works out its cosines and sines. Those stand in shared memory as
// [row][angle of a unit][unit], so neighbouring threads read neighbouring 16 bytes. (On 131072 rows of 10
// heads: 168 us with a unit's angles side by side and turned and passing units mixed, 146 with both mended, 120
// with neighbouring threads on neighbouring rows of one pair where the angles are made, 109 with two rows in
// flight and five CTAs per SM.)
template <typename T, int VE, bool HALVES>
__global__ void __launch_bounds__(kRotThreads, HALVES && VE > 1 ? 5 : 4) rotary_kernel(const __grid_constant__ RotArgs a) {
  constexpr bool kTwo = HALVES || VE == 1;                     // a turned unit is two accesses
  constexpr int kTurn = HALVES ? VE : (VE == 1 ? 1 : VE / 2);  // pairs per turned unit
  constexpr int kU = rot_unroll(HALVES && VE > 1);
  constexpr int kPack = kTurn > 1 ? 2 : 1;                     // angles per shared-memory access
  using R = Raw<T, VE>;
  extern __shared__ float2 cs[];
  const int pairs = a.plan.pairs, turned = pairs / kTurn;
  const int stride = pairs + kRotPad;  // off the multiples of the banks, where the rows' angles are written
  const int b = int(blockIdx.x / a.row_ctas), t0 = int(blockIdx.x - b * a.row_ctas) * a.rows_per_cta;
  const int nrows = min(a.rows_per_cta, a.rows - t0);
  pdl_wait();
  pdl_trigger();
  bool first = true;
  const int group = int(threadIdx.x) / a.row_units;  // rows taken at a time when a row has few units
  int i = int(threadIdx.x) - group * a.row_units;    // the unit among the row's
  if (group >= a.groups) i = a.row_units;            // threads left over
  do {  // every thread makes the first turn, for the barrier in it
    const bool turn = i < a.turned_units;
    const int per = turn ? turned : a.units - turned, i0 = turn ? i : i - a.turned_units;
    const int hh = per > 0 ? i0 / per : 0, unit = i0 - hh * per;
    const int z = hh >= a.q_heads, h = z ? hh - a.q_heads : hh;
    const bool live = i < a.row_units && (turn || a.copy[z]);
    const int off = turn ? (HALVES ? unit * VE : unit * 2 * kTurn) : 2 * pairs + unit * VE;
    const T* x = static_cast<const T*>(a.x[z]) + b * a.xb[z] + (t0 + group) * a.xr[z] + h * a.xh[z] + off;
    T* out = static_cast<T*>(a.out[z]) + b * a.ob[z] + (t0 + group) * a.orow[z] + h * a.oh[z] + off;
    const long long dx = a.groups * a.xr[z], dy = a.groups * a.orow[z];
    const float2* c = cs + (group * stride + unit * kPack);
    int left = live ? (nrows - group + a.groups - 1) / a.groups : 0;  // rows of this thread
    do {
      R v[kU][kTwo ? 2 : 1];
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (u < left) {
          v[u][0] = rot_load<T, VE>(x + u * dx);
          if constexpr (kTwo)
            if (turn) v[u][1] = rot_load<T, VE>(x + u * dx + (HALVES ? pairs : 1));
        }
      if (first) {
        for (int k = threadIdx.x; k < nrows * pairs; k += kRotThreads) {
          const int f = k / nrows, r = k - f * nrows;  // neighbours share a pair: its plan entry is one constant
          const int32_t p = __ldg(a.pos + ((long long)b * a.rows + t0 + r) * a.plan.axes + a.plan.axis[f]);
          float2 t = rot_cos_sin(p, a.plan.turns[f], a.plan.amplitude);
          if (a.inverse) t.y = -t.y;
          const int j = f % kTurn;
          cs[r * stride + (j / kPack * turned + f / kTurn) * kPack + j % kPack] = t;
        }
        __syncthreads();
        first = false;
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (u >= left) continue;
        T* dst = out + u * dy;
        if (!turn) {
          rot_store<T, VE>(dst, v[u][0]);
          continue;
        }
        float2 t[kTurn];
        const float2* cu = c + u * a.groups * stride;
        if constexpr (kPack == 2) {  // pairs even, so 16-byte steps stay on 16 bytes
#pragma unroll
          for (int j = 0; j < kTurn / 2; ++j) {
            const float4 q = *reinterpret_cast<const float4*>(cu + j * 2 * turned);
            t[2 * j] = make_float2(q.x, q.y);
            t[2 * j + 1] = make_float2(q.z, q.w);
          }
        } else {
          t[0] = *cu;
        }
        float x0[VE];
        rot_values<T, VE>(v[u][0], x0);
        if constexpr (kTwo) {
          float x1[VE], y0[VE], y1[VE];
          rot_values<T, VE>(v[u][1], x1);
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            y0[j] = x0[j] * t[j].x - x1[j] * t[j].y;
            y1[j] = x0[j] * t[j].y + x1[j] * t[j].x;
          }
          rot_store<T, VE>(dst, rot_raw<T, VE>(y0));
          rot_store<T, VE>(dst + (HALVES ? pairs : 1), rot_raw<T, VE>(y1));
        } else {
          float y[VE];
#pragma unroll
          for (int j = 0; j < kTurn; ++j) {
            y[2 * j] = x0[2 * j] * t[j].x - x0[2 * j + 1] * t[j].y;
            y[2 * j + 1] = x0[2 * j] * t[j].y + x0[2 * j + 1] * t[j].x;
          }
          rot_store<T, VE>(dst, rot_raw<T, VE>(y));
        }
      }
      left -= kU;
      x += kU * dx;
      out += kU * dy;
      c += kU * a.groups * stride;
    } while (left > 0);
    i += kRotThreads;
  } while (i < a.row_units);
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
      const double hi = std::fmin(double(w - 1), std::ceil(at(s->beta_slow)));  // may lie past the last pair
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
  if (!pos || !cos || !sin || !al4(pos) || !al4(cos) || !al4(sin)) return DIT_EINVAL;
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
  if (batch == 0 || rows == 0 || (q->heads == 0 && (!k || k->heads == 0))) return DIT_OK;
  if (!pos || !al4(pos)) return DIT_EINVAL;
  // one tensor as q and k, written by one of them at least: which of the two is read first would be chance
  if (k && q->heads > 0 && k->heads > 0 && (q->out == k->out || q->out == k->x || k->out == q->x)) return DIT_EINVAL;
  RotArgs a;
  std::memset(&a, 0, sizeof(a));
  bool vec = head_dim % ve == 0 && (plan->layout == DIT_ROTARY_HALVES ? plan->pairs : 2 * plan->pairs) % ve == 0;
  for (int z = 0; z < 2; ++z) {
    const dit_rotary_rows* r = part[z];
    if (!r || r->heads == 0) continue;
    if (!r->x || !r->out || reinterpret_cast<uintptr_t>(r->x) % size || reinterpret_cast<uintptr_t>(r->out) % size)
      return DIT_EINVAL;
    // rows that share their place in the output would race
    if ((batch > 1 && r->out_batch == 0) || (rows > 1 && r->out_row == 0) || (r->heads > 1 && r->out_head == 0))
      return DIT_EINVAL;
    a.x[z] = r->x;
    a.out[z] = r->out;
    a.xb[z] = r->x_batch;
    a.xr[z] = r->x_row;
    a.xh[z] = r->x_head;
    a.ob[z] = r->out_batch;
    a.orow[z] = r->out_row;
    a.oh[z] = r->out_head;
    a.heads += r->heads;
    if (z == 0) a.q_heads = r->heads;
    const bool same = r->x == r->out && (rows == 1 || r->x_row == r->out_row) &&
                      (r->heads == 1 || r->x_head == r->out_head) && (batch == 1 || r->x_batch == r->out_batch);
    if (r->x == r->out && !same) return DIT_EINVAL;  // in place under other strides: rows over one another
    a.copy[z] = !same;
    auto on16 = [&](const void* p, long long s0, long long s1, long long s2) {
      return reinterpret_cast<uintptr_t>(p) % 16 == 0 && s0 % ve == 0 && s1 % ve == 0 && s2 % ve == 0;
    };
    vec = vec && on16(r->x, batch > 1 ? r->x_batch : 0, rows > 1 ? r->x_row : 0, r->heads > 1 ? r->x_head : 0) &&
          on16(r->out, batch > 1 ? r->out_batch : 0, rows > 1 ? r->out_row : 0, r->heads > 1 ? r->out_head : 0);
  }
  // batch entries that follow one another in every tensor are rows of one entry
  auto joined = [&](const dit_rotary_rows* r) {
    return !r || r->heads == 0 || (r->x_batch == rows * r->x_row && r->out_batch == rows * r->out_row);
  };
  if (batch > 1 && joined(q) && joined(k) && (long long)batch * rows <= 0x7fffffffLL) {
    rows *= batch;
    batch = 1;
  }
  a.rows = rows;
  a.inverse = inverse != 0;
  a.pos = pos;
  a.plan = *plan;
  const int v = vec ? ve : 1;
  const int turned = plan->pairs / (plan->layout == DIT_ROTARY_HALVES ? v : (v == 1 ? 1 : v / 2));
  a.units = turned + (head_dim - 2 * plan->pairs) / v;
  const long long row_units = (long long)a.units * a.heads;
  if (row_units > 0x7fffffffLL - kRotThreads) return DIT_EUNSUPPORTED;
  a.row_units = int(row_units);
  a.turned_units = turned * a.heads;
  a.groups = std::max(1, kRotThreads / a.row_units);
  // Two rounds per thread and two units, while there are CTAs for every SM several times over.
  const int round = rot_unroll(plan->layout == DIT_ROTARY_HALVES && vec);
  long long per = std::max<long long>(2 * round * a.groups, 8LL * kRotThreads / row_units);
  per = std::min<long long>(per, kRotMaxRows);
  per = std::max(1LL, std::min(per, (long long)batch * rows / (3LL * num_sms())));
  if (per > round * a.groups) per -= per % (round * a.groups);  // whole rounds: 6 rows 22.5, 8 rows 18.5 us at 4224 rows
  per = std::min<long long>(per, rows);
  a.rows_per_cta = int(per);
  a.row_ctas = int((rows + per - 1) / per);
  const long long ctas = (long long)batch * a.row_ctas;
  if (ctas > 0x7fffffffLL) return DIT_EUNSUPPORTED;
  const dim3 grid{unsigned(ctas), 1u, 1u};
  const size_t smem = size_t(per) * (plan->pairs + kRotPad) * sizeof(float2);
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
