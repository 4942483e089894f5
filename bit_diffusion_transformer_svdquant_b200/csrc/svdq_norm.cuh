// Block norms: the normalisation in front of a block's linear, and a block's end -- an optional norm of
// its output, the gate and the residual -- in one pass over each row, optionally with the result
// quantized to MXFP4 for the next layer (declared in svdq.h as svdq_block_norm*).
//   x' = skip x + res gate_s . P(y),   h = Norm(x') . (1 + scale_s) + shift_s
// A row's x, y and x' stay in registers, so x and y cross HBM once and nothing else is read but the
// per-sample and per-channel vectors, which the rows of a sample share in L1. The mean and the centred
// second moment are summed in fp32 in two register passes: no cancellation, whatever the mean.
// DRAM traffic bounds it; a group of G threads shares a row, so that a row's values and its vectors fit
// in registers and several rows are in flight per SM.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "svdq_mx.cuh"
#include "svdq_ptx.cuh"
#include "svdq_quant.cuh"

namespace svdq {
namespace norm {

struct Vec {          // a per-channel or per-sample vector
  const void* p;      // null: absent
  long long ld;       // elements between samples (0: shared)
  int f32;
};
struct Norm {
  int kind;           // 0 none, 1 RMS, 2 LayerNorm
  float eps;
  Vec w, b;
};
struct Args {
  const void* x;
  const void* y;
  void* x_out;
  void* h;
  long long ldx, ldy, ld_out, ldh;
  int x_f32, y_f32, h_f32;
  int M, D, rows;     // rows: M, or the padded rows of a quantized output
  int samples, rows_per_sample;
  const int* offsets;
  float skip, res;
  Vec gate, scale, shift;
  Norm post, pre;
  // quantized output
  const float* inv_lambda;
  uint8_t* codes;
  uint8_t* sf;
  int K_pad;
};

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}
__device__ __forceinline__ uint4 pack8_bf16(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&b2);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Thread t of a group of G owns, of every chunk c, the 8 consecutive elements from 8 (c G + t) (VEC: one
// or two 16-byte accesses) or the elements (8 c + e) G + t, e = 0..7 (any alignment).
template <int C, bool VEC>
struct Row {
  static __device__ __forceinline__ int index(int c, int e, int G, int t) {
    return VEC ? 8 * (c * G + t) + e : (8 * c + e) * G + t;
  }
  static __device__ __forceinline__ float load1(const void* p, long long i, int f32) {
    return f32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  }
  // a row of streamed data from element `base` of p; elements past D are 0
  static __device__ __forceinline__ void load(float (&v)[C][8], const void* p, long long base, int f32, int D, int G,
                                              int t) {
    if constexpr (VEC) {
      if (f32) {
        const float* s = static_cast<const float*>(p) + base;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int i = index(c, 0, G, t);
          uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
          if (i < D) {
            a = ld_stream(s + i);
            b = ld_stream(s + i + 4);
          }
          const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) v[c][e] = __uint_as_float(w[e]);
        }
      } else {
        const __nv_bfloat16* s = static_cast<const __nv_bfloat16*>(p) + base;
        uint4 raw[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int i = index(c, 0, G, t);
          raw[c] = i < D ? ld_stream(s + i) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) bf16x8_to_f32(raw[c], v[c]);
      }
    } else {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = index(c, e, G, t);
          v[c][e] = i < D ? load1(p, base + i, f32) : 0.0f;
        }
    }
  }
  // 8 elements of a shared vector for chunk c (0 past D)
  static __device__ __forceinline__ void vec8(float (&v)[8], const Vec& a, long long s, int c, int D, int G, int t) {
    const long long base = s * a.ld;
    if constexpr (VEC) {
      const int i = index(c, 0, G, t);
      if (i >= D) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.0f;
      } else if (a.f32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(a.p) + base + i);
        const float4 l = __ldg(q), r = __ldg(q + 1);
        v[0] = l.x; v[1] = l.y; v[2] = l.z; v[3] = l.w;
        v[4] = r.x; v[5] = r.y; v[6] = r.z; v[7] = r.w;
      } else {
        bf16x8_to_f32(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.p) + base + i)), v);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = index(c, e, G, t);
        v[e] = i < D ? load1(a.p, base + i, a.f32) : 0.0f;
      }
    }
  }
  static __device__ __forceinline__ void store(const float (&v)[8], void* p, long long base, int f32, int c, int D,
                                               int G, int t) {
    if constexpr (VEC) {
      const int i = index(c, 0, G, t);
      if (i >= D) return;
      if (f32) {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(p) + base + i);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p) + base + i) = pack8_bf16(v);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = index(c, e, G, t);
        if (i < D) {
          if (f32) static_cast<float*>(p)[base + i] = v[e];
          else static_cast<__nv_bfloat16*>(p)[base + i] = __float2bfloat16_rn(v[e]);
        }
      }
    }
  }
};

// Sum over the group's threads. Groups of one warp need only shuffles; larger groups exchange one
// partial per warp through shared memory behind the group's named barrier. `red` alternates between two
// buffers, so that one barrier per sum is enough: before a buffer is written again every thread of the
// group has passed the next sum's barrier, hence read it.
struct Reducer {
  float* red;   // [2][warps]
  int warps, w, lane, bar, flip;
  __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps == 1) return v;
    float* r = red + flip * warps;
    flip ^= 1;
    if (lane == 0) r[w] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
    v = lane < warps ? r[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
};

// In place: v <- Norm(v) over the row's D elements (those past D come out as 0 or are not used).
template <int C, bool VEC>
__device__ __forceinline__ void normalise(float (&v)[C][8], const Norm& n, int D, int G, int t, Reducer& red) {
  using R = Row<C, VEC>;
  const float inv_d = 1.0f / static_cast<float>(D);
  float mean = 0.0f;
  if (n.kind == 2) {
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[c][e];
    mean = red.sum(s) * inv_d;
  }
  float q = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = R::index(c, e, G, t) < D ? v[c][e] - mean : 0.0f;
      v[c][e] = d;
      q = fmaf(d, d, q);
    }
  // sqrt and divide in IEEE rounding: once per row
  const float rstd = __frcp_rn(__fsqrt_rn(fmaf(red.sum(q), inv_d, n.eps)));
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[c][e] *= rstd;
    if (n.w.p != nullptr) {
      float w[8];
      R::vec8(w, n.w, 0, c, D, G, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] *= w[e];
    }
    if (n.b.p != nullptr) {
      float b[8];
      R::vec8(b, n.b, 0, c, D, G, t);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] += b[e];
    }
  }
}

// The sample of row m, or -1 for a row outside every sample. Indexes stay in [0, samples) whatever the
// offsets hold.
__device__ __forceinline__ int sample_of(const Args& a, int m) {
  if (a.offsets == nullptr) return m < a.M ? m / a.rows_per_sample : -1;
  if (m >= a.M || m < __ldg(a.offsets) || m >= __ldg(a.offsets + a.samples)) return -1;
  int lo = 0, hi = a.samples - 1;  // the last sample that starts at or before m (empty ones precede it)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(a.offsets + mid) <= m) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Blocks of blockDim.x / G row groups; a group takes rows g, g + groups, ... C chunks of 8 per thread
// cover the row (a quantized row: its padded length). QUANT: h is rounded to bf16 and quantized.
template <int C, bool VEC, bool QUANT>
__global__ void __launch_bounds__(512) block_norm_kernel(const __grid_constant__ Args a, int G) {
  using R = Row<C, VEC>;
  __shared__ float red_smem[2 * 16 + 8];
  grid_dependency_wait();
  grid_launch_dependents();
  const int D = a.D;
  const int group = threadIdx.x / G, t = threadIdx.x - group * G;
  const int per_block = blockDim.x / G;
  Reducer red;
  red.warps = G >> 5;
  red.w = t >> 5;
  red.lane = t & 31;
  red.bar = 1 + group;
  red.flip = 0;
  red.red = red_smem + 2 * red.warps * group;
  for (int m = blockIdx.x * per_block + group; m < a.rows; m += gridDim.x * per_block) {
    const int s = sample_of(a, m);
    if (s < 0) {  // uniform over the group
      if constexpr (QUANT) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int i = R::index(c, 0, G, t);
          if (i < a.K_pad) {
            *reinterpret_cast<uint32_t*>(a.codes + static_cast<size_t>(m) * (a.K_pad >> 1) + (i >> 1)) = 0u;
            if ((i & 31) == 0) a.sf[mx::act_sf_offset(m, i >> 5, a.K_pad)] = 0;
          }
        }
      }
      continue;
    }
    float v[C][8];
    if (a.y != nullptr) {
      float y[C][8];
      R::load(y, a.y, m * a.ldy, a.y_f32, D, G, t);
      R::load(v, a.x, m * a.ldx, a.x_f32, D, G, t);
      if (a.post.kind) normalise<C, VEC>(y, a.post, D, G, t, red);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (a.gate.p != nullptr) {
          float g[8];
          R::vec8(g, a.gate, s, c, D, G, t);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[c][e] *= g[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] = fmaf(a.res, y[c][e], a.skip * v[c][e]);
        if (a.x_out != nullptr) R::store(v[c], a.x_out, m * a.ld_out, a.x_f32, c, D, G, t);
      }
    } else {
      R::load(v, a.x, m * a.ldx, a.x_f32, D, G, t);
    }
    if (!a.pre.kind) continue;
    normalise<C, VEC>(v, a.pre, D, G, t, red);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (a.scale.p != nullptr) {
        float g[8];
        R::vec8(g, a.scale, s, c, D, G, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] = fmaf(v[c][e], g[e], v[c][e]);
      }
      if (a.shift.p != nullptr) {
        float g[8];
        R::vec8(g, a.shift, s, c, D, G, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[c][e] += g[e];
      }
      if (a.h != nullptr) R::store(v[c], a.h, m * a.ldh, a.h_f32, c, D, G, t);
      if constexpr (QUANT) {
        // the codes svdq_mx_quantize_act makes of bf16(h): smoothing in fp32, blocks of four lanes
        const int i = R::index(c, 0, G, t);
        float q[8];
        bf16x8_to_f32(pack8_bf16(v[c]), q);
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = i < D ? q[e] : 0.0f;
        if (i < D) {
          const float4 l0 = __ldg(reinterpret_cast<const float4*>(a.inv_lambda + i));
          const float4 l1 = __ldg(reinterpret_cast<const float4*>(a.inv_lambda + i + 4));
          const float l[8] = {l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) q[e] = __fmul_rn(q[e], l[e]);
        }
        uint32_t sc;
        const uint32_t codes = mx::quarter_block(q, sc);
        if (i < a.K_pad) {
          *reinterpret_cast<uint32_t*>(a.codes + static_cast<size_t>(m) * (a.K_pad >> 1) + (i >> 1)) = codes;
          if ((i & 31) == 0) a.sf[mx::act_sf_offset(m, i >> 5, a.K_pad)] = static_cast<uint8_t>(sc);
        }
      }
    }
  }
}

}  // namespace norm
}  // namespace svdq
