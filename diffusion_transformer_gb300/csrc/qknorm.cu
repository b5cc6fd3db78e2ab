// Per-head RMS norm of q and k with their rotary turn in one pass, and its gradient (the QK norm and turn of the
// gizai:dit reference's prepOf and of the klein article's section 4.4, there an epilogue of the bf16 QKV product).
//
// Mathematics. For a head x of d values with weights w, r = rsqrt(mean(x^2) + eps) and R the row's turn (times the
// plan's amplitude):   y = R (x r w).   With the gradient dy of y:   g = R^T dy,  u = g w,
//   dx = r (u - x r mean(u x r)),      dw = sum over rows and heads of g x r.
// All in fp32 with one rounding to the tensor's type; the angles are those of rotary.cuh.
//
// What bounds it: HBM. Forward: each value read once and written once. Backward: x and dy read once, dx written
// once; dw is summed in registers along the rows a thread meets, over the CTA's groups in shared memory, and over
// the CTAs by a second small kernel, each in a fixed order, so a call's result does not depend on timing. 4224 rows of
// 24 + 24 heads of 128 in bf16: 20.7 us forward (5.0 TB/s, instruction issue at 0.69 of a cycle), 35 backward (4.4 TB/s); one row
// 3.3 us.
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

constexpr int kQkThreads = 256;
constexpr int kQkMaxCtas = 320;  // CTAs of the backward pass at most: each leaves one row of partial sums

struct QkArgs {
  const void* x[2];
  const void* dy[2];
  void* out[2];
  long long xb[2], xr[2], xh[2], yb[2], yr[2], yh[2], ob[2], orow[2], oh[2];  // strides in values
  const float* w[2];  // null: ones
  int heads[2];
  int d, rows, rows_per_chunk, row_chunks;  // rows of a batch entry, of a chunk; chunks of a batch entry
  int chunks;
  int row_groups;  // groups of lanes that share a row's heads
  int lanes, units, turned;  // lanes of a head (a power of two), its units, those of them that turn
  float eps;
  float* partial;  // backward: [CTA][q, k][d]
  const int32_t* pos;
  dit_rotary_plan plan;
};

// A unit is what one lane holds of a head, as in the rotary kernel: VE consecutive values, with their VE partners
// in the split-halves layout (VE = 1: one pair, or one value that does not turn). A head stands on `lanes`
// neighbouring lanes, NU units on each, so its sum of squares is a butterfly within a warp and the values stay in
// registers between the sum and the turn. A CTA takes a chunk of rows, whose cosines and sines it works out once into shared
// memory; a group of lanes takes one of them (or shares it with others) and keeps its units' angles in registers through
// the row's heads. (4224 rows of 24 + 24 heads in bf16: 26.8 us with groups that stepped through heads of several rows,
// 24.0 with the next heads loaded ahead, 20.7 with a row to a group.)
// Heads in a lane's registers at a time (and as many on their way): two of eight values, one of sixteen
__host__ __device__ constexpr int qk_flight(int nu, int vals) { return nu == 1 && vals <= 8 ? 2 : 1; }
template <typename T, int VE, bool HALVES, int NU, bool GRAD>
struct QkCfg {
  static constexpr bool kTwo = HALVES || VE == 1;
  static constexpr int kTurn = HALVES ? VE : (VE == 1 ? 1 : VE / 2);  // pairs of a turned unit
  static constexpr int kVals = kTwo ? 2 * VE : VE;
  static constexpr int kPiece = kTurn < 4 ? kTurn : 4;  // angles per shared-memory access
  static constexpr int kU = qk_flight(NU, kVals);
};

// n = kPiece floats at 4 n bytes alignment
template <int N>
__device__ __forceinline__ void ld_piece(const float* p, float* v) {
  if constexpr (N == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else if constexpr (N == 2) {
    const float2 q = *reinterpret_cast<const float2*>(p);
    v[0] = q.x; v[1] = q.y;
  } else {
    v[0] = *p;
  }
}

template <typename T, int VE, bool HALVES, int NU, bool GRAD>
__global__ void __launch_bounds__(kQkThreads, VE > 1 && NU == 1 ? (GRAD ? 2 : 4) : 1) qknorm_kernel(const __grid_constant__ QkArgs a) {
  using C = QkCfg<T, VE, HALVES, NU, GRAD>;
  using R = Raw<T, VE>;
  constexpr int kU = C::kU, kVals = C::kVals, kTurn = C::kTurn, kPiece = C::kPiece;
  constexpr bool kTwo = C::kTwo;
  extern __shared__ float qk_smem[];
  const int pairs = a.plan.pairs, turned = a.turned;
  float* sc = qk_smem;                             // [row][angle piece of a unit][unit]
  float* ss = qk_smem + a.rows_per_chunk * pairs;  // (neighbouring lanes read neighbouring pieces)
  const int groups = kQkThreads / a.lanes, group = int(threadIdx.x) / a.lanes, u0 = int(threadIdx.x) % a.lanes;
  int off[NU];
  bool live[NU], turn[NU];
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    const int u = u0 + n * a.lanes;
    live[n] = u < a.units;
    turn[n] = u < turned;
    off[n] = turn[n] ? (HALVES ? u * VE : u * 2 * kTurn) : 2 * pairs + (u - turned) * VE;
  }
  const float inv_d = 1.f / float(a.d);
  const int far = HALVES ? pairs : 1;  // from a unit's first values to their partners
  float acc[GRAD ? 2 : 1][NU][kVals];
#pragma unroll
  for (int z = 0; z < (GRAD ? 2 : 1); ++z)
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
      for (int j = 0; j < kVals; ++j) acc[z][n][j] = 0.f;
  pdl_wait();
  pdl_trigger();

  for (int chunk = blockIdx.x; chunk < a.chunks; chunk += gridDim.x) {
    const int b = chunk / a.row_chunks, t0 = (chunk - b * a.row_chunks) * a.rows_per_chunk;
    const int nrows = min(a.rows_per_chunk, a.rows - t0);
    const int row = group / a.row_groups, phase = group - row * a.row_groups;  // this group's row of the chunk, its first head
    const bool here = row < nrows;
    bool angles = false;
    float c[NU][kTurn], sn[NU][kTurn];  // the row's cosines and sines of this lane's pairs
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int heads = a.heads[z];
      if (heads == 0) continue;  // the same for the CTA
      const long long first = here ? (long long)row : 0;
      const T* x = static_cast<const T*>(a.x[z]) + b * a.xb[z] + (t0 + first) * a.xr[z] + phase * a.xh[z];
      const T* dy = GRAD ? static_cast<const T*>(a.dy[z]) + b * a.yb[z] + (t0 + first) * a.yr[z] + phase * a.yh[z] : nullptr;
      T* out = static_cast<T*>(a.out[z]) + b * a.ob[z] + (t0 + first) * a.orow[z] + phase * a.oh[z];
      const long long xd = a.row_groups * a.xh[z], yd = a.row_groups * a.yh[z], od = a.row_groups * a.oh[z];
      int left_in = here ? heads - phase : 0, left_out = left_in;  // heads of the row from the next one on
      // heads loaded, and the ones before them turned while they come
      struct Batch {
        R v[kU][NU][kTwo ? 2 : 1], e[GRAD ? kU : 1][NU][kTwo ? 2 : 1];
      };
      auto fetch = [&](Batch& q) {
#pragma unroll
        for (int k = 0; k < kU; ++k) {
          const T *px = x + k * xd, *py = GRAD ? dy + k * yd : nullptr;
#pragma unroll
          for (int n = 0; n < NU; ++n) {
#pragma unroll
            for (int i = 0; i < (kTwo ? 2 : 1); ++i) {
              q.v[k][n][i] = R{};
              if constexpr (GRAD) q.e[k][n][i] = R{};
            }
            if (left_in <= k * a.row_groups || !live[n]) continue;
            q.v[k][n][0] = rot_load<T, VE>(px + off[n]);
            if constexpr (kTwo)
              if (turn[n]) q.v[k][n][1] = rot_load<T, VE>(px + off[n] + far);
            if constexpr (GRAD) {
              q.e[k][n][0] = rot_load<T, VE>(py + off[n]);
              if constexpr (kTwo)
                if (turn[n]) q.e[k][n][1] = rot_load<T, VE>(py + off[n] + far);
            }
          }
        }
        left_in -= kU * a.row_groups;
        x += kU * xd;
        if constexpr (GRAD) dy += kU * yd;
      };
      const int rounds = (heads + a.row_groups * kU - 1) / (a.row_groups * kU);
      Batch next;
      fetch(next);
      float w[NU][kVals];
#pragma unroll
      for (int n = 0; n < NU; ++n)
#pragma unroll
        for (int j = 0; j < kVals; ++j)
          w[n][j] = a.w[z] && live[n] && (j < VE || turn[n]) ? __ldg(a.w[z] + off[n] + (j < VE ? j : far + j - VE)) : 1.f;
      if (!angles) {  // once per chunk, behind the first loads
        if (chunk != int(blockIdx.x)) __syncthreads();  // the last chunk's angles have been read
        for (int k = threadIdx.x; k < nrows * pairs; k += kQkThreads) {
          const int f = k / nrows, r = k - f * nrows;  // neighbours share a pair: its plan entry is one constant
          const int32_t p = __ldg(a.pos + ((long long)b * a.rows + t0 + r) * a.plan.axes + a.plan.axis[f]);
          const float2 t = rot_cos_sin(p, a.plan.turns[f], a.plan.amplitude);
          const int u = f / kTurn, j = f - u * kTurn;
          const int place = r * pairs + (j / kPiece) * (kPiece * turned) + u * kPiece + j % kPiece;
          sc[place] = t.x;
          ss[place] = GRAD ? -t.y : t.y;
        }
        __syncthreads();
        angles = true;
#pragma unroll
        for (int n = 0; n < NU; ++n) {
#pragma unroll
          for (int i = 0; i < kTurn / kPiece; ++i) {
#pragma unroll
            for (int j = 0; j < kPiece; ++j) {
              c[n][i * kPiece + j] = 1.f;
              sn[n][i * kPiece + j] = 0.f;
            }
            if (turn[n]) {
              const int at = int(first) * pairs + (u0 + n * a.lanes) * kPiece + i * kPiece * turned;
              ld_piece<kPiece>(sc + at, c[n] + i * kPiece);
              ld_piece<kPiece>(ss + at, sn[n] + i * kPiece);
            }
          }
        }
      }
      // the turn of one unit: (p, q) -> (p c - q s, p s + q c)
      auto spin = [&](float* m, int n) {
#pragma unroll
        for (int f = 0; f < kTurn; ++f) {
          const int p0 = kTwo ? f : 2 * f, p1 = kTwo ? VE + f : 2 * f + 1;
          const float u = m[p0], v = m[p1];
          m[p0] = u * c[n][f] - v * sn[n][f];
          m[p1] = u * sn[n][f] + v * c[n][f];
        }
      };
      for (int round = 0; round < rounds; ++round) {
        Batch q = next;
        if (round + 1 < rounds) fetch(next);
#pragma unroll
        for (int k = 0; k < kU; ++k) {
          const bool ok = left_out > k * a.row_groups;
          float y[NU][kVals];
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < NU; ++n) {
            float h[VE];
            rot_values<T, VE>(q.v[k][n][0], h);
#pragma unroll
            for (int j = 0; j < VE; ++j) y[n][j] = h[j];
            if constexpr (kTwo) {
              rot_values<T, VE>(q.v[k][n][1], h);
#pragma unroll
              for (int j = 0; j < VE; ++j) y[n][VE + j] = h[j];
            }
#pragma unroll
            for (int j = 0; j < kVals; ++j) sum = fmaf(y[n][j], y[n][j], sum);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1)
            if (o < a.lanes) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          const float r = rsqrtf(fmaf(sum, inv_d, a.eps));
          if constexpr (!GRAD) {
#pragma unroll
            for (int n = 0; n < NU; ++n) {
#pragma unroll
              for (int j = 0; j < kVals; ++j) y[n][j] = y[n][j] * r * w[n][j];
              spin(y[n], n);  // (a unit that passes: by the cosine 1)
            }
          } else {
            float g[NU][kVals];
            float dot = 0.f;
#pragma unroll
            for (int n = 0; n < NU; ++n) {
              float h[VE];
              rot_values<T, VE>(q.e[k][n][0], h);
#pragma unroll
              for (int j = 0; j < VE; ++j) g[n][j] = h[j];
              if constexpr (kTwo) {
                rot_values<T, VE>(q.e[k][n][1], h);
#pragma unroll
                for (int j = 0; j < VE; ++j) g[n][VE + j] = h[j];
              }
              spin(g[n], n);
#pragma unroll
              for (int j = 0; j < kVals; ++j) {
                y[n][j] *= r;
                if (ok) acc[GRAD ? z : 0][n][j] = fmaf(g[n][j], y[n][j], acc[GRAD ? z : 0][n][j]);
                g[n][j] *= w[n][j];
                dot = fmaf(g[n][j], y[n][j], dot);
              }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
              if (o < a.lanes) dot += __shfl_xor_sync(0xffffffffu, dot, o);
            dot *= inv_d;
#pragma unroll
            for (int n = 0; n < NU; ++n)
#pragma unroll
              for (int j = 0; j < kVals; ++j) y[n][j] = r * (g[n][j] - y[n][j] * dot);
          }
          if (!ok) continue;
          T* po = out + k * od;
#pragma unroll
          for (int n = 0; n < NU; ++n) {
            if (!live[n]) continue;
            float h[VE];
#pragma unroll
            for (int j = 0; j < VE; ++j) h[j] = y[n][j];
            rot_store<T, VE>(po + off[n], rot_raw<T, VE>(h));
            if constexpr (kTwo)
              if (turn[n]) {
#pragma unroll
                for (int j = 0; j < VE; ++j) h[j] = y[n][VE + j];
                rot_store<T, VE>(po + off[n] + far, rot_raw<T, VE>(h));
              }
          }
        }
        left_out -= kU * a.row_groups;
        out += kU * od;
      }
    }
  }

  if constexpr (GRAD) {
    // this CTA's sums for the weights' gradients, over its groups in order
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NU; ++n) {
        if (!live[n]) continue;
#pragma unroll
        for (int j = 0; j < kVals; ++j)
          if (j < VE || turn[n]) qk_smem[group * a.d + off[n] + (j < VE ? j : far + j - VE)] = acc[z][n][j];
      }
      __syncthreads();
      for (int j = threadIdx.x; j < a.d; j += kQkThreads) {
        float s = 0.f;
        for (int g = 0; g < groups; ++g) s += qk_smem[g * a.d + j];
        a.partial[((long long)blockIdx.x * 2 + z) * a.d + j] = s;
      }
    }
  }
}

// The weights' gradients from the CTAs' sums: a block per 32 values of one norm, 32 slices of the CTAs, each with all
// of its loads in flight, then a butterfly over the slices.
constexpr int kSumSlices = 32, kSumLoads = kQkMaxCtas / kSumSlices;
__global__ void __launch_bounds__(1024) qknorm_sum_kernel(const float* partial, int ctas, int d, float* dq, float* dk) {
  __shared__ float part[kSumSlices][33];
  pdl_wait();
  pdl_trigger();
  const int z = blockIdx.y, lane = threadIdx.x & 31, j = blockIdx.x * 32 + lane, slice = threadIdx.x >> 5;
  float* out = z ? dk : dq;
  if (!out) return;
  float v[kSumLoads];
#pragma unroll
  for (int i = 0; i < kSumLoads; ++i) {
    const int c = slice + i * kSumSlices;
    v[i] = c < ctas && j < d ? partial[((long long)c * 2 + z) * d + j] : 0.f;
  }
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kSumLoads; ++i) s += v[i];
  part[slice][lane] = s;
  __syncthreads();
  s = part[lane][slice];  // a warp per value now
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int col = blockIdx.x * 32 + slice;
  if (lane == 0 && col < d) out[col] = s;
}

template <typename T, int VE, bool HALVES, bool GRAD>
cudaError_t qk_units(const QkArgs& a, unsigned ctas, size_t smem, cudaStream_t st) {
  const dim3 grid(ctas), block(kQkThreads);
  if (a.units <= 32) return launch_pdl(qknorm_kernel<T, VE, HALVES, 1, GRAD>, grid, block, smem, st, 1, a);
  if constexpr (VE != 8)
    if (a.units <= 64) return launch_pdl(qknorm_kernel<T, VE, HALVES, 2, GRAD>, grid, block, smem, st, 1, a);
  if constexpr (VE == 1) return launch_pdl(qknorm_kernel<T, VE, HALVES, 8, GRAD>, grid, block, smem, st, 1, a);
  return cudaErrorInvalidValue;
}
template <typename T, int VE>
cudaError_t qk_go(const QkArgs& a, bool grad, unsigned ctas, size_t smem, cudaStream_t st) {
  const bool halves = a.plan.layout == DIT_ROTARY_HALVES;
  if (grad) return halves ? qk_units<T, VE, true, true>(a, ctas, smem, st) : qk_units<T, VE, false, true>(a, ctas, smem, st);
  return halves ? qk_units<T, VE, true, false>(a, ctas, smem, st) : qk_units<T, VE, false, false>(a, ctas, smem, st);
}

// One of the tensors a call reads or writes: `p` with its strides, for `heads` heads.
struct Tensor {
  const void* p;
  long long s[3];  // batch, row, head
};

struct Extents {
  int batch, rows, heads;
};

bool same_strides(const Tensor& a, const Tensor& b, const Extents& n) {
  return (n.batch == 1 || a.s[0] == b.s[0]) && (n.rows == 1 || a.s[1] == b.s[1]) && (n.heads == 1 || a.s[2] == b.s[2]);
}

// Both passes: checks, geometry, launch. `rows_of` z: x, dy (backward), out of q (0) and k (1).
int qk_launch(const dit_rotary_plan* plan, const int heads[2], const Tensor x[2], const Tensor dy[2], const Tensor out[2],
              const float* q_norm, const float* k_norm, float eps, int type, int batch, int rows, int head_dim,
              const int32_t* pos, bool grad, float* partial, unsigned* ctas_out, cudaStream_t st) {
  const int size = type == DIT_BF16 ? 2 : 4, ve = 16 / size;
  if (!pos || !al4(pos)) return DIT_EINVAL;
  QkArgs a;
  std::memset(&a, 0, sizeof(a));
  bool vec = head_dim % ve == 0 && (plan->layout == DIT_ROTARY_HALVES ? plan->pairs : 2 * plan->pairs) % ve == 0;
  bool joined = true;
  const float* norm[2] = {q_norm, k_norm};
  for (int z = 0; z < 2; ++z) {
    if (heads[z] == 0) continue;
    if (norm[z] && !al4(norm[z])) return DIT_EINVAL;
    const Extents n{batch, rows, heads[z]};
    const Tensor* t[3] = {&x[z], &out[z], grad ? &dy[z] : &x[z]};
    for (const Tensor* p : t) {
      if (!p->p || reinterpret_cast<uintptr_t>(p->p) % size) return DIT_EINVAL;
      vec = vec && reinterpret_cast<uintptr_t>(p->p) % 16 == 0 && (batch == 1 || p->s[0] % ve == 0) &&
            (rows == 1 || p->s[1] % ve == 0) && (heads[z] == 1 || p->s[2] % ve == 0);
      joined = joined && p->s[0] == rows * p->s[1];
    }
    // values of an output that share a place would race
    if ((batch > 1 && out[z].s[0] == 0) || (rows > 1 && out[z].s[1] == 0) || (heads[z] > 1 && out[z].s[2] == 0)) return DIT_EINVAL;
    // in place: over an input of the same strides, which each head's lanes have read before they write
    if (out[z].p == x[z].p && !same_strides(out[z], x[z], n)) return DIT_EINVAL;
    if (grad && out[z].p == dy[z].p && !same_strides(out[z], dy[z], n)) return DIT_EINVAL;
    a.x[z] = x[z].p;
    a.out[z] = const_cast<void*>(out[z].p);
    a.xb[z] = x[z].s[0]; a.xr[z] = x[z].s[1]; a.xh[z] = x[z].s[2];
    a.ob[z] = out[z].s[0]; a.orow[z] = out[z].s[1]; a.oh[z] = out[z].s[2];
    if (grad) {
      a.dy[z] = dy[z].p;
      a.yb[z] = dy[z].s[0]; a.yr[z] = dy[z].s[1]; a.yh[z] = dy[z].s[2];
    }
    a.w[z] = norm[z];
    a.heads[z] = heads[z];
  }
  // one tensor as q and k, written by one of them at least: which of the two is read first would be chance
  if (heads[0] > 0 && heads[1] > 0) {
    if (out[0].p == out[1].p || out[0].p == x[1].p || out[1].p == x[0].p) return DIT_EINVAL;
    if (grad && (out[0].p == dy[1].p || out[1].p == dy[0].p)) return DIT_EINVAL;
  }
  // batch entries that follow one another in every tensor are rows of one entry
  if (batch > 1 && joined && (long long)batch * rows <= 0x7fffffffLL) {
    rows *= batch;
    batch = 1;
  }
  const int v = vec ? ve : 1;
  a.d = head_dim;
  a.rows = rows;
  a.eps = eps;
  a.partial = partial;
  a.pos = pos;
  a.plan = *plan;
  a.turned = plan->pairs / (plan->layout == DIT_ROTARY_HALVES ? v : (v == 1 ? 1 : v / 2));
  a.units = a.turned + (head_dim - 2 * plan->pairs) / v;
  a.lanes = 1;
  const int per_lane = a.units <= 32 ? 1 : (a.units <= 64 ? 2 : 8);
  while (a.lanes * per_lane < a.units) a.lanes *= 2;
  const int groups = kQkThreads / a.lanes, all = heads[0] + heads[1];
  // Groups of a row, and so rows of a chunk: one where there are rows enough, more while there are fewer chunks than the SMs
  // hold half of (forward: two to an SM, backward: one) and the row has heads for them
  const int most = std::max(heads[0], heads[1]);
  a.row_groups = 1;
  while (2 * a.row_groups <= std::min(groups, most) && (long long)batch * rows * a.row_groups < (grad ? 1LL : 2LL) * num_sms() * groups)
    a.row_groups *= 2;
  const long long per = std::min<long long>(groups / a.row_groups, rows);
  if (per * all > 0x7fffffffLL / 4) return DIT_EUNSUPPORTED;
  a.rows_per_chunk = int(per);
  a.row_chunks = int((rows + per - 1) / per);
  const long long chunks = (long long)batch * a.row_chunks;
  if (chunks > 0x7fffffffLL) return DIT_EUNSUPPORTED;
  a.chunks = int(chunks);
  const unsigned ctas = grad ? unsigned(std::min<long long>(chunks, std::min(2 * num_sms(), kQkMaxCtas))) : unsigned(chunks);
  size_t smem = size_t(per) * plan->pairs * 2 * sizeof(float);
  if (grad) smem = std::max(smem, size_t(groups) * head_dim * sizeof(float));
  cudaError_t e;
  if (type == DIT_BF16)
    e = vec ? qk_go<__nv_bfloat16, 8>(a, grad, ctas, smem, st) : qk_go<__nv_bfloat16, 1>(a, grad, ctas, smem, st);
  else
    e = vec ? qk_go<float, 4>(a, grad, ctas, smem, st) : qk_go<float, 1>(a, grad, ctas, smem, st);
  if (e != cudaSuccess || cudaGetLastError() != cudaSuccess) return DIT_ECUDA;
  if (ctas_out) *ctas_out = ctas;
  return DIT_OK;
}

int qk_check(const dit_rotary_plan* plan, int type, int batch, int rows, int head_dim, float eps, int q_heads, int k_heads) {
  if (!plan_ok(plan) || batch < 0 || rows < 0 || (type != DIT_BF16 && type != DIT_F32)) return DIT_EINVAL;
  if (head_dim < 2 * plan->pairs || !(eps >= 0.f) || !std::isfinite(eps) || q_heads < 0 || k_heads < 0) return DIT_EINVAL;
  if (head_dim > 2 * DIT_ROTARY_MAX_PAIRS || q_heads > 1 << 20 || k_heads > 1 << 20) return DIT_EUNSUPPORTED;
  return DIT_OK;
}

}  // namespace
}  // namespace dit

using namespace dit;

extern "C" {

int dit_qknorm_rotary(const dit_rotary_plan* plan, const dit_rotary_rows* q, const dit_rotary_rows* k, const float* q_norm,
                      const float* k_norm, float eps, int type, int batch, int rows, int head_dim, const int32_t* pos,
                      dit_stream_t stream) {
  if (!q) return DIT_EINVAL;
  const int heads[2] = {q->heads, k ? k->heads : 0};
  const int rc = qk_check(plan, type, batch, rows, head_dim, eps, heads[0], heads[1]);
  if (rc != DIT_OK) return rc;
  if (batch == 0 || rows == 0 || heads[0] + heads[1] == 0) return DIT_OK;
  Tensor x[2] = {}, out[2] = {};
  const dit_rotary_rows* part[2] = {q, k};
  for (int z = 0; z < 2; ++z)
    if (heads[z] > 0) {
      x[z] = Tensor{part[z]->x, {part[z]->x_batch, part[z]->x_row, part[z]->x_head}};
      out[z] = Tensor{part[z]->out, {part[z]->out_batch, part[z]->out_row, part[z]->out_head}};
    }
  return qk_launch(plan, heads, x, x, out, q_norm, k_norm, eps, type, batch, rows, head_dim, pos, false, nullptr, nullptr,
                   reinterpret_cast<cudaStream_t>(stream));
}

size_t dit_qknorm_rotary_backward_workspace_bytes(int head_dim) {
  return head_dim < 1 || head_dim > 2 * DIT_ROTARY_MAX_PAIRS ? 0 : size_t(kQkMaxCtas) * 2 * head_dim * sizeof(float);
}

int dit_qknorm_rotary_backward(const dit_rotary_plan* plan, const dit_rotary_grad* q, const dit_rotary_grad* k,
                               const float* q_norm, const float* k_norm, float eps, int type, int batch, int rows,
                               int head_dim, const int32_t* pos, float* q_norm_grad, float* k_norm_grad, void* ws,
                               size_t ws_bytes, dit_stream_t stream) {
  if (!q) return DIT_EINVAL;
  const int heads[2] = {q->heads, k ? k->heads : 0};
  int rc = qk_check(plan, type, batch, rows, head_dim, eps, heads[0], heads[1]);
  if (rc != DIT_OK) return rc;
  if ((q_norm_grad && !al4(q_norm_grad)) || (k_norm_grad && !al4(k_norm_grad))) return DIT_EINVAL;
  if (q_norm_grad && q_norm_grad == k_norm_grad) return DIT_EINVAL;
  if (ws && reinterpret_cast<uintptr_t>(ws) % 256) return DIT_EINVAL;
  if (!ws || ws_bytes < dit_qknorm_rotary_backward_workspace_bytes(head_dim)) return DIT_EWORKSPACE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  unsigned ctas = 0;
  if (batch > 0 && rows > 0 && heads[0] + heads[1] > 0) {
    Tensor x[2] = {}, dy[2] = {}, out[2] = {};
    const dit_rotary_grad* part[2] = {q, k};
    for (int z = 0; z < 2; ++z)
      if (heads[z] > 0) {
        const dit_rotary_grad& g = *part[z];
        x[z] = Tensor{g.x, {g.x_batch, g.x_row, g.x_head}};
        dy[z] = Tensor{g.dy, {g.dy_batch, g.dy_row, g.dy_head}};
        out[z] = Tensor{g.dx, {g.dx_batch, g.dx_row, g.dx_head}};
      }
    rc = qk_launch(plan, heads, x, dy, out, q_norm, k_norm, eps, type, batch, rows, head_dim, pos, true,
                   static_cast<float*>(ws), &ctas, st);
    if (rc != DIT_OK) return rc;
  }
  if (!q_norm_grad && !k_norm_grad) return DIT_OK;
  // no rows: sums of nothing, which are written too
  if (launch_pdl(qknorm_sum_kernel, dim3(unsigned((head_dim + 31) / 32), 2), dim3(1024), 0, st, 1,
                 static_cast<const float*>(ws), int(ctas), head_dim, q_norm_grad, k_norm_grad) != cudaSuccess)
    return DIT_ECUDA;
  return cudaGetLastError() == cudaSuccess ? DIT_OK : DIT_ECUDA;
}

}  // extern "C"
