// Epilogues that drain an accumulator tile from tensor memory: shared by the bf16 / int8 GEMMs and the
// 4-bit product (the gizai:dit reference's linearInto / gatedInto / gluRows / prepOf; see gemm.cu for the
// list).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace dit {
namespace {

__device__ __forceinline__ float silu_f(float z) { return z / (1.0f + __expf(-z)); }

__device__ __forceinline__ void store_bf16x32(uint16_t* dst, const float* v) {
  uint4* d = reinterpret_cast<uint4*>(dst);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint4 u;
    u.x = pack_bf16x2(v[8 * c + 0], v[8 * c + 1]);
    u.y = pack_bf16x2(v[8 * c + 2], v[8 * c + 3]);
    u.z = pack_bf16x2(v[8 * c + 4], v[8 * c + 5]);
    u.w = pack_bf16x2(v[8 * c + 6], v[8 * c + 7]);
    d[c] = u;
  }
}

// ----------------------------------------------------------------------------------------------
// epilogues: thread `lane` of epilogue warp `quad` owns TMEM lane quad * 32 + lane, i.e. output row
// row0 + lane of the warp's 32-row slab; taddr points at (its lane, column n0). tcgen05.ld is
// warp-collective, so every lane loads even when its row is out of range. `stage` is this warp's
// 4 KB shared-memory scratch (the transposed v store, the gated residual's transpose). BN here is
// the warp's column count.
// ----------------------------------------------------------------------------------------------
template <int BN, int EPI, bool kRowPerThread>
__device__ __forceinline__ void epilogue_tile(const GemmParams& p, uint32_t taddr, int row0, int row_end, int lane,
                                              int n0, uint8_t* stage) {
  const int row = row0 + lane;
  const bool row_ok = row < row_end;
  if constexpr (EPI == kEpiQKV) {
    const int d = p.head_dim;
    const int H = p.H;
    const int R = p.R_total > 0 ? p.R_total : p.M;  // rows of the q, k and vt layouts
    const int srow = row + p.row_off;                // sequence row of this thread's GEMM row
    const int tw = p.rope_split ? 3 * d / 8 : d / 2;  // rotary table columns per row
    for (int hh = 0; hh < BN / d; ++hh) {
      const int col0 = n0 + hh * d;
      const int which = col0 / H;              // 0 = q, 1 = k, 2 = v
      const int head = (col0 - which * H) / d;
      const uint32_t ta = taddr + hh * d;
      if (which == 2) {
        // v, transposed: vt[head*d + j][row]. Stage the warp's 32 rows x 32 values as bf16 (64 B
        // per row, 16-byte chunks XOR-swizzled by (row >> 1) & 3), then lane j writes value j of
        // all 32 rows as 64 contiguous bytes.
        uint32_t* st32 = reinterpret_cast<uint32_t*>(stage);
        for (int c = 0; c < d / 32; ++c) {
          uint32_t v[32];
          tmem_ld32(ta + c * 32, v);
          tmem_ld_wait();
          __syncwarp();
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int slot = q ^ ((lane >> 1) & 3);
            *reinterpret_cast<uint4*>(stage + lane * 64 + slot * 16) =
                make_uint4(pack_bf16x2(__uint_as_float(v[8 * q + 0]), __uint_as_float(v[8 * q + 1])),
                           pack_bf16x2(__uint_as_float(v[8 * q + 2]), __uint_as_float(v[8 * q + 3])),
                           pack_bf16x2(__uint_as_float(v[8 * q + 4]), __uint_as_float(v[8 * q + 5])),
                           pack_bf16x2(__uint_as_float(v[8 * q + 6]), __uint_as_float(v[8 * q + 7])));
          }
          __syncwarp();
          const int j = lane;  // value index within the chunk
          uint32_t col[16];
#pragma unroll
          for (int r = 0; r < 32; r += 2) {
            const int o0 = r * 64 + (((j >> 3) ^ ((r >> 1) & 3)) << 4) + (j & 7) * 2;
            const int o1 = (r + 1) * 64 + (((j >> 3) ^ (((r + 1) >> 1) & 3)) << 4) + (j & 7) * 2;
            const uint32_t lo = *reinterpret_cast<const uint16_t*>(stage + o0);
            const uint32_t hi = *reinterpret_cast<const uint16_t*>(stage + o1);
            col[r >> 1] = lo | (hi << 16);
          }
          (void)st32;
          uint16_t* dst = p.vt + (size_t(head) * d + c * 32 + j) * p.Rp + row0 + p.row_off;
          if (row0 + 32 <= row_end && ((row0 + p.row_off) & 7) == 0) {
            uint4* d4 = reinterpret_cast<uint4*>(dst);  // (row0 + row_off) % 8 == 0, Rp % 8 == 0: 16-byte aligned
#pragma unroll
            for (int q = 0; q < 4; ++q) d4[q] = make_uint4(col[4 * q], col[4 * q + 1], col[4 * q + 2], col[4 * q + 3]);
          } else {
#pragma unroll
            for (int r = 0; r < 32; ++r)
              if (row0 + r < row_end) dst[r] = uint16_t(r & 1 ? col[r >> 1] >> 16 : col[r >> 1] & 0xffffu);
          }
        }
        continue;
      }
      // pass 1: sum of squares of the head
      float ss = 0.f;
      for (int c = 0; c < d / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(ta + c * 32, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float f = __uint_as_float(v[j]);
          ss = fmaf(f, f, ss);
        }
      }
      const float rstd = rsqrtf(ss / float(d) + p.qk_eps);
      const bool g2 = p.m_split > 0 && row >= p.m_split;  // second row group: its own head norms
      const float* wn = which == 0 ? (g2 ? p.q_norm2 : p.q_norm) : (g2 ? p.k_norm2 : p.k_norm);
      const float4* cs = reinterpret_cast<const float4*>(srow < p.L ? p.txt_cos + size_t(srow) * tw
                                                                      : p.img_cos + size_t(srow - p.L) * tw);
      const float4* sn = reinterpret_cast<const float4*>(srow < p.L ? p.txt_sin + size_t(srow) * tw
                                                                      : p.img_sin + size_t(srow - p.L) * tw);
      uint16_t* dst = (which == 0 ? p.q : p.k) + (size_t(head) * R + srow) * d;
      if (p.rope_split) {
        // pass 2, split halves: values i and i + hr (i < hr = 3d/8) turned by angle i, eight pairs
        // at a time; the last d/4 values are normalised and weighted only
        const int hr = 3 * d / 8;
        for (int i0 = 0; i0 < hr; i0 += 8) {
          uint32_t va[8], vb[8];
          tmem_ld8(ta + i0, va);
          tmem_ld8(ta + i0 + hr, vb);
          tmem_ld_wait();
          if (!row_ok) continue;
          const float4 c0 = __ldg(cs + i0 / 4), c1 = __ldg(cs + i0 / 4 + 1);
          const float4 s0 = __ldg(sn + i0 / 4), s1 = __ldg(sn + i0 / 4 + 1);
          const float cf[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
          const float sf[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
          uint32_t pa[4], pb[4];
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float a[2], b[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              a[u] = __uint_as_float(va[j + u]) * rstd;
              b[u] = __uint_as_float(vb[j + u]) * rstd;
              if (wn) {
                a[u] *= __ldg(wn + i0 + j + u);
                b[u] *= __ldg(wn + i0 + hr + j + u);
              }
            }
            pa[j / 2] = pack_bf16x2(a[0] * cf[j] - b[0] * sf[j], a[1] * cf[j + 1] - b[1] * sf[j + 1]);
            pb[j / 2] = pack_bf16x2(a[0] * sf[j] + b[0] * cf[j], a[1] * sf[j + 1] + b[1] * cf[j + 1]);
          }
          *reinterpret_cast<uint4*>(dst + i0) = make_uint4(pa[0], pa[1], pa[2], pa[3]);
          *reinterpret_cast<uint4*>(dst + i0 + hr) = make_uint4(pb[0], pb[1], pb[2], pb[3]);
        }
        for (int i0 = 2 * hr; i0 < d; i0 += 8) {
          uint32_t va[8];
          tmem_ld8(ta + i0, va);
          tmem_ld_wait();
          if (!row_ok) continue;
          uint32_t pa[4];
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float a0 = __uint_as_float(va[j]) * rstd, a1 = __uint_as_float(va[j + 1]) * rstd;
            if (wn) {
              a0 *= __ldg(wn + i0 + j);
              a1 *= __ldg(wn + i0 + j + 1);
            }
            pa[j / 2] = pack_bf16x2(a0, a1);
          }
          *reinterpret_cast<uint4*>(dst + i0) = make_uint4(pa[0], pa[1], pa[2], pa[3]);
        }
        continue;
      }
      // pass 2: normalise, weight, rotate adjacent pairs, store
      for (int c = 0; c < d / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(ta + c * 32, v);
        tmem_ld_wait();
        if (!row_ok) continue;
        float y[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          float f = __uint_as_float(v[j]) * rstd;
          if (wn) f *= __ldg(wn + c * 32 + j);
          y[j] = f;
        }
        float cf[16], sf[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 c4 = __ldg(cs + c * 4 + q);
          const float4 s4 = __ldg(sn + c * 4 + q);
          cf[4 * q] = c4.x; cf[4 * q + 1] = c4.y; cf[4 * q + 2] = c4.z; cf[4 * q + 3] = c4.w;
          sf[4 * q] = s4.x; sf[4 * q + 1] = s4.y; sf[4 * q + 2] = s4.z; sf[4 * q + 3] = s4.w;
        }
        float o[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float a = y[2 * i], b = y[2 * i + 1];
          o[2 * i] = a * cf[i] - b * sf[i];
          o[2 * i + 1] = a * sf[i] + b * cf[i];
        }
        store_bf16x32(dst + c * 32, o);
      }
    }
  } else if constexpr (EPI == kEpiGated && kRowPerThread) {
    // x[r, n] += gate[map[r], n] * acc, one row per thread: the form for the int8 in-mainloop
    // kernel, whose 320 threads leave 168 registers each (the coalesced form below would spill).
    const int grow = (row_ok ? row : 0) + p.row_off;  // sequence row
    float* x = grow < p.L ? p.txt + size_t(grow) * p.N : p.img + size_t(grow - p.L) * p.N;
    const int m = (p.map && row_ok) ? __ldg(p.map + grow) : 0;
    const float* g = p.gate + size_t(m) * p.gate_stride;
#pragma unroll 1
    for (int c = 0; c < BN / 32; ++c) {
      uint32_t v[32];
      tmem_ld32(taddr + c * 32, v);
      const int n = n0 + c * 32;
      float4 xq[8], gq[8];
      const float4* xv = reinterpret_cast<const float4*>(x + n);
      const float4* gv = reinterpret_cast<const float4*>(g + n);
      if (row_ok) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          xq[q] = xv[q];
          gq[q] = __ldg(gv + q);
        }
      }
      tmem_ld_wait();
      if (row_ok) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          xq[q].x = fmaf(gq[q].x, __uint_as_float(v[4 * q + 0]), xq[q].x);
          xq[q].y = fmaf(gq[q].y, __uint_as_float(v[4 * q + 1]), xq[q].y);
          xq[q].z = fmaf(gq[q].z, __uint_as_float(v[4 * q + 2]), xq[q].z);
          xq[q].w = fmaf(gq[q].w, __uint_as_float(v[4 * q + 3]), xq[q].w);
        }
        float4* xo = reinterpret_cast<float4*>(x + n);
#pragma unroll
        for (int q = 0; q < 8; ++q) xo[q] = xq[q];
      }
    }
  } else if constexpr (EPI == kEpiGated) {
    // x[r, n] += gate[map[r], n] * acc. The accumulator chunk (32 rows x 32 columns, thread = row)
    // goes through the warp's 4 KB shared tile (16-byte chunks XOR-swizzled by row & 7), so the
    // global accesses are coalesced: lane handles rows (lane >> 3) + 4 i, i = 0..7, 16-byte column
    // chunk lane & 7, and every warp instruction moves four whole 128-byte lines of x or the gate.
    // The loads of chunk c + 1 are issued as soon as chunk c is stored. Every lane runs every
    // tcgen05.ld (warp-collective); only the global accesses are predicated.
    (void)row_ok;
    const int cq = lane & 7;
    float* xr[8];
    const float* gr[8];
    bool ok[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = row0 + (lane >> 3) + 4 * i;
      ok[i] = r < row_end;
      const int rr = (ok[i] ? r : 0) + p.row_off;  // sequence row
      xr[i] = (rr < p.L ? p.txt + size_t(rr) * p.N : p.img + size_t(rr - p.L) * p.N) + n0 + cq * 4;
      gr[i] = p.gate + size_t(p.map ? __ldg(p.map + rr) : 0) * p.gate_stride + n0 + cq * 4;
    }
    float4 xq[8], gq[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (ok[i]) {
        xq[i] = *reinterpret_cast<const float4*>(xr[i]);
        gq[i] = __ldg(reinterpret_cast<const float4*>(gr[i]));
      }
#pragma unroll 1
    for (int c = 0; c < BN / 32; ++c) {
      uint32_t v[32];
      tmem_ld32(taddr + c * 32, v);
      tmem_ld_wait();
#pragma unroll
      for (int q = 0; q < 8; ++q)
        *reinterpret_cast<uint4*>(stage + lane * 128 + ((q ^ (lane & 7)) << 4)) =
            make_uint4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rl = (lane >> 3) + 4 * i;
        const float4 a = *reinterpret_cast<const float4*>(stage + rl * 128 + ((cq ^ (rl & 7)) << 4));
        if (ok[i]) {
          float4 o;
          o.x = fmaf(gq[i].x, a.x, xq[i].x);
          o.y = fmaf(gq[i].y, a.y, xq[i].y);
          o.z = fmaf(gq[i].z, a.z, xq[i].z);
          o.w = fmaf(gq[i].w, a.w, xq[i].w);
          *reinterpret_cast<float4*>(xr[i] + c * 32) = o;
        }
      }
      __syncwarp();
      if (c + 1 < BN / 32) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (ok[i]) {
            xq[i] = *reinterpret_cast<const float4*>(xr[i] + (c + 1) * 32);
            gq[i] = __ldg(reinterpret_cast<const float4*>(gr[i] + (c + 1) * 32));
          }
      }
    }
  } else {
#pragma unroll 1
    for (int c = 0; c < BN / 32; ++c) {
      uint32_t v[32];
      tmem_ld32(taddr + c * 32, v);
      tmem_ld_wait();
      if (!row_ok) continue;
      const int n = n0 + c * 32;
      if constexpr (EPI == kEpiStoreF32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + size_t(row) * p.ldo + n);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          dst[q] = make_float4(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]),
                               __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]));
      } else if constexpr (EPI == kEpiStoreBF16 || EPI == kEpiSiluBF16) {
        float f[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          f[j] = __uint_as_float(v[j]);
          if constexpr (EPI == kEpiSiluBF16) f[j] = silu_f(f[j]);
        }
        store_bf16x32(static_cast<uint16_t*>(p.out) + size_t(row) * p.ldo + n, f);
      } else if constexpr (EPI == kEpiSwiGLU) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float a0 = silu_f(__uint_as_float(v[4 * j + 0])) * __uint_as_float(v[4 * j + 1]);
          const float a1 = silu_f(__uint_as_float(v[4 * j + 2])) * __uint_as_float(v[4 * j + 3]);
          w[j] = pack_bf16x2(a0, a1);
        }
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + size_t(row) * p.ldo + n / 2);
        dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
        dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
  }
}

}  // namespace
}  // namespace dit
