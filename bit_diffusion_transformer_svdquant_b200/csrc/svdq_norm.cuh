// Block norms: the normalisation in front of a block's linear, and a block's end -- an optional norm of
// its output, the gate and the residual -- in one pass over each row, optionally with the result
// quantized to MXFP4 for the next layer (declared in svdq.h as svdq_block_norm*).
//   x' = skip x + res gate_s . P(y),   h = Norm(x') . (1 + scale_s) + shift_s
// Rows of x and y arrive in a shared-memory ring as bulk copies and cross HBM once; y is read from the ring
// for each of its sums and for x', which then stays in registers. The per-sample and per-channel vectors
// are multiplied into factors that lie in shared memory for all rows of a sample (for few rows and very
// wide ones they are read from global memory per row). The mean and the centred second moment are summed
// in fp32 one after the other: no cancellation, whatever the mean.
// DRAM traffic bounds it; a group of G threads shares a row, so that several rows are in flight per SM.
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
  long long ldx, ldy, ld_out, ldh;   // row m of sample s: element m ld + s adj
  long long adj_x, adj_y, adj_out, adj_h;
  int x_f32, y_f32, h_f32;
  int M, D, rows;     // rows: M, or the padded rows of a quantized output
  int samples, rows_per_sample;
  unsigned long long per_sample;  // ceil(2^64 / rows per sample), 0 for one row per sample
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

// Pairs of fp32 values in one instruction (each half rounds as the scalar operation).
__device__ __forceinline__ uint64_t bits2(float2 v) { return *reinterpret_cast<const uint64_t*>(&v); }
__device__ __forceinline__ float2 from2(uint64_t b) { return *reinterpret_cast<const float2*>(&b); }
__device__ __forceinline__ float2 dup2(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return from2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return from2(r);
}
struct F8 {
  float2 p[4];
};
__device__ __forceinline__ F8 pair8(const float (&v)[8]) {
  F8 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r.p[j] = make_float2(v[2 * j], v[2 * j + 1]);
  return r;
}
__device__ __forceinline__ F8 bf16x8(const uint4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  F8 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r.p[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
  return r;
}
__device__ __forceinline__ uint4 pack8_bf16(const F8& v) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(v.p[j].x, v.p[j].y);
    w[j] = *reinterpret_cast<const uint32_t*>(&b2);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A group of G threads shares a row; thread t owns, of every chunk c, the elements index(c, e) for e in
// 0..7: VEC (D a multiple of 8, 16-byte aligned rows and vectors) the 8 consecutive ones from
// 8 (c G + t), else the strided (8 c + e) G + t.
template <bool VEC>
__device__ __forceinline__ int index(int c, int e, int G, int t) {
  return VEC ? 8 * (c * G + t) + e : (8 * c + e) * G + t;
}
__device__ __forceinline__ float load1(const void* p, long long i, int f32) {
  return f32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
// 8 elements (chunk c) of a shared vector of sample s; 0 past D
template <bool VEC>
__device__ __forceinline__ void vec8(float (&v)[8], const Vec& a, long long s, int c, int D, int G, int t) {
  const long long base = s * a.ld;
  if constexpr (VEC) {
    const int i = index<true>(c, 0, G, t);
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
      const int i = index<false>(c, e, G, t);
      v[e] = i < D ? load1(a.p, base + i, a.f32) : 0.0f;
    }
  }
}
__device__ __forceinline__ void store8(const F8& v, void* row, int f32, int i) {
  if (f32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(row) + i);
    o[0] = make_float4(v.p[0].x, v.p[0].y, v.p[1].x, v.p[1].y);
    o[1] = make_float4(v.p[2].x, v.p[2].y, v.p[3].x, v.p[3].y);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(row) + i) = pack8_bf16(v);
  }
}
__device__ __forceinline__ void store_strided(const float (&v)[8], void* p, long long base, int f32, int c, int D, int G,
                                              int t) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = index<false>(c, e, G, t);
    if (i < D) {
      if (f32) static_cast<float*>(p)[base + i] = v[e];
      else static_cast<__nv_bfloat16*>(p)[base + i] = __float2bfloat16_rn(v[e]);
    }
  }
}

// Per-channel factors of chunk c for sample s: x' = skip x + t a1 (+ b1) with t = y or its normalised
// value, h = n a2 + b2 with n the normalised x'. Products of the vectors, so that a row costs one
// multiply-add per element whatever is present. b1 (only with a bias in the norm of y) is separate.
template <bool VEC>
__device__ __forceinline__ void post_factors(const Args& a, int s, int c, int G, int t, float (&a1)[8]) {
  float p[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) a1[e] = a.res;
  if (a.gate.p != nullptr) {
    vec8<VEC>(p, a.gate, s, c, a.D, G, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) a1[e] *= p[e];
  }
  if (a.post.w.p != nullptr) {
    vec8<VEC>(p, a.post.w, 0, c, a.D, G, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) a1[e] *= p[e];
  }
}
template <bool VEC>
__device__ __forceinline__ void post_bias(const Args& a, int s, int c, int G, int t, float (&b1)[8]) {
  float p[8];
  vec8<VEC>(b1, a.post.b, 0, c, a.D, G, t);
#pragma unroll
  for (int e = 0; e < 8; ++e) b1[e] *= a.res;
  if (a.gate.p != nullptr) {
    vec8<VEC>(p, a.gate, s, c, a.D, G, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) b1[e] *= p[e];
  }
}
template <bool VEC>
__device__ __forceinline__ void pre_factors(const Args& a, int s, int c, int G, int t, float (&a2)[8], float (&b2)[8]) {
  const int D = a.D;
  float p[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    a2[e] = 1.0f;
    b2[e] = 0.0f;
  }
  if (a.scale.p != nullptr) {
    vec8<VEC>(p, a.scale, s, c, D, G, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) a2[e] += p[e];
  }
  if (a.shift.p != nullptr) vec8<VEC>(b2, a.shift, s, c, D, G, t);
  if (a.pre.b.p != nullptr) {
    vec8<VEC>(p, a.pre.b, 0, c, D, G, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) b2[e] = fmaf(a2[e], p[e], b2[e]);
  }
  if (a.pre.w.p != nullptr) {
    vec8<VEC>(p, a.pre.w, 0, c, D, G, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) a2[e] *= p[e];
  }
}

// Sums of R rows over the group's threads at once. Inside a warp the R values are halved against one
// another (R / 2 + R / 4 + ... shuffles instead of 5 R), so that lane l ends up with the sum of row
// l / (32 / R); groups of several warps then exchange one partial per warp and row through shared memory
// behind the group's named barrier. `red` alternates between two buffers, so that one barrier per sum is
// enough: before a buffer is written again every thread of the group has passed the next sum's barrier,
// hence read it.
template <int R>
struct Reducer {
  float* red;   // [2][R][16]
  int warps, w, lane, bar, flip;
  __device__ __forceinline__ void sync() const {
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(warps * 32) : "memory");
  }
  __device__ __forceinline__ void sum(float (&v)[R]) {
    constexpr int kSpan = 32 / R;  // lanes that share a row
    float x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = v[r];
#pragma unroll
    for (int n = R / 2, o = 16; n > 0; n /= 2, o /= 2) {
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int r = 0; r < n; ++r) {
        const float mine = up ? x[r + n] : x[r], other = up ? x[r] : x[r + n];
        x[r] = mine + __shfl_xor_sync(0xffffffffu, other, o);
      }
    }
    float y = x[0];
#pragma unroll
    for (int o = kSpan / 2; o > 0; o /= 2) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (warps > 1) {
      const int mine = lane / kSpan, i = lane & (kSpan - 1);
      float* q = red + flip * R * 16;
      flip ^= 1;
      if (i == 0) q[mine * 16 + w] = y;
      sync();
      y = 0.0f;
#pragma unroll
      for (int k = 0; k < 16; k += kSpan)
        if (i + k < warps) y += q[mine * 16 + i + k];
#pragma unroll
      for (int o = kSpan / 2; o > 0; o /= 2) y += __shfl_xor_sync(0xffffffffu, y, o);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] = __shfl_sync(0xffffffffu, y, r * kSpan);
  }
};

// 1 / sqrt(q / D + eps): rsqrtf and one step of Newton's method, within about 1.5 units in the last
// place (every thread of a group computes it, so it is kept to a few instructions). 0 (an all-equal row
// with eps = 0) and infinity keep rsqrtf's value, which the step would turn into a NaN.
__device__ __forceinline__ float root(float q, float inv_d, float eps) {
  const float v = fmaf(q, inv_d, eps), r = rsqrtf(v);
  const float n = fmaf(fmaf(-v * r, r, 1.0f), 0.5f * r, r);
  return v > 0.0f && v < __uint_as_float(0x7F800000u) ? n : r;
}

// The sample of row m, or -1 for a row outside every sample. Indexes stay in [0, samples) whatever the
// offsets hold.
__device__ __forceinline__ int sample_of(const Args& a, int m) {
  if (a.offsets == nullptr)
    return m >= a.M ? -1 : a.per_sample ? static_cast<int>(__umul64hi(m, a.per_sample)) : m;  // m / rows per sample
  if (m >= a.M || m < __ldg(a.offsets) || m >= __ldg(a.offsets + a.samples)) return -1;
  int lo = 0, hi = a.samples - 1;  // the last sample that starts at or before m (empty ones precede it)
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(a.offsets + mid) <= m) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

constexpr int kMaxWarps = 16;     // per block, and per row
constexpr int kMaxStages = 2;     // batches a group holds or has in flight

// Rows of any alignment, one at a time straight from global memory, element by element: the path of
// misaligned or odd-sized rows, and of fp32 x and y too wide for the ring. Moments as in block_norm_kernel.
// Nothing is in flight from the next row and every vector is read again for each, so that the latency of
// these loads bounds it, far from DRAM: on B200 a modulated LayerNorm of 4608 rows of 3071, bf16, takes 168 us
// (the same at 3072 on the 16-byte path 13.2), with y, gate and post-norm 333 us (24.1), one row 6.3 us. Above 4096
// values a row (two chunks and more) its values spill to local memory, 312 bytes a thread at two chunks and
// 2.5 to 8.7 KB from four on.
template <int C>
__global__ void __launch_bounds__(32 * kMaxWarps) block_norm_any_kernel(const __grid_constant__ Args a, int G) {
  __shared__ float red_smem[2 * 16 * kMaxWarps];
  grid_dependency_wait();
  grid_launch_dependents();
  const int D = a.D;
  const float inv_d = 1.0f / static_cast<float>(D);
  const int group = threadIdx.x / G, t = threadIdx.x - group * G, groups = blockDim.x / G;
  Reducer<1> red{red_smem + 2 * 16 * group, G >> 5, t >> 5, t & 31, 1 + group, 0};
  auto load = [&](float (&v)[C][8], const void* p, long long base, int f32) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = index<false>(c, e, G, t);
        v[c][e] = i < D ? load1(p, base + i, f32) : 0.0f;
      }
  };
  // v <- (v - mean) rstd; elements past D stay 0
  auto normalise = [&](float (&v)[C][8], const Norm& n) {
    float s[1] = {0.0f};
    if (n.kind == 2) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += v[c][e];
      red.sum(s);
    }
    const float mean = s[0] * inv_d;
    float q[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[c][e] = index<false>(c, e, G, t) < D ? v[c][e] - mean : 0.0f;
        q[0] = fmaf(v[c][e], v[c][e], q[0]);
      }
    red.sum(q);
    const float rstd = root(q[0], inv_d, n.eps);
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] *= rstd;
  };
  for (int m = blockIdx.x * groups + group; m < a.rows; m += gridDim.x * groups) {
    const int s = sample_of(a, m);
    if (s < 0) continue;
    float v[C][8];
    if (a.y != nullptr) {
      load(v, a.y, m * a.ldy + s * a.adj_y, a.y_f32);
      if (a.post.kind) normalise(v, a.post);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float f[8], b[8] = {};
        post_factors<false>(a, s, c, G, t, f);
        if (a.post.b.p != nullptr) post_bias<false>(a, s, c, G, t, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = index<false>(c, e, G, t);
          const float x = i < D ? load1(a.x, m * a.ldx + s * a.adj_x + i, a.x_f32) : 0.0f;
          v[c][e] = fmaf(v[c][e], f[e], fmaf(a.skip, x, b[e]));
        }
        if (a.x_out != nullptr) store_strided(v[c], a.x_out, m * a.ld_out + s * a.adj_out, a.x_f32, c, D, G, t);
      }
    } else {
      load(v, a.x, m * a.ldx + s * a.adj_x, a.x_f32);
    }
    if (!a.pre.kind) continue;
    normalise(v, a.pre);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float f[8], b[8];
      pre_factors<false>(a, s, c, G, t, f, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[c][e] = fmaf(v[c][e], f[e], b[e]);
      store_strided(v[c], a.h, m * a.ldh + s * a.adj_h, a.h_f32, c, D, G, t);
    }
  }
}

enum { kNoY = 0, kBf16Y = 1, kF32Y = 2 };  // the template's Y: no y, or its type

// A run of rows of one sample (s >= 0), or of rows outside every sample (s = -1).
struct Run {
  int s, end;
};
__device__ __forceinline__ Run run_at(const Args& a, int m, int limit) {
  Run r;
  r.s = sample_of(a, m);
  r.end = limit;
  if (a.offsets == nullptr) {
    // rows per sample come with the run: the sample's end is the first row of the next
    if (r.s >= 0) r.end = min(limit, min(a.M, (r.s + 1) * a.rows_per_sample));
  } else if (r.s >= 0) {
    r.end = min(min(limit, a.M), __ldg(a.offsets + r.s + 1));  // a quantized output has rows of padding behind M
  } else if (m < __ldg(a.offsets)) {
    r.end = min(limit, __ldg(a.offsets));
  }
  r.end = max(r.end, m + 1);  // offsets of any content: a run holds a row at least
  return r;
}

// Each block takes a contiguous share of the rows and goes through it run by run; inside a run its groups
// of G threads take batches of R rows in turn.
//   - A group's first warp keeps `stages` batches in flight as bulk copies into the group's ring in shared
//     memory (across runs), so that DRAM latency is covered by bytes in flight and not by registers; a
//     batch's stage is filled again as soon as x' is in registers.
//   - Groups are small (a thread holds up to 48 values of a row), so that many rows are in flight per SM
//     and the latency of one row's sums is covered by the others'.
//   - SHARE: the factors of the run's sample are laid in shared memory once per run, because reading the
//     vectors for every row came to twice the bytes of the row itself. Where runs are too short for that
//     (or rows too long) every row reads them from global memory.
//     A quantized output's smoothing reciprocals lie behind them (LAMBDAS) where they fit, else they are
//     read per row: whether factors are shared must not depend on them, because the order of a row's sums
//     goes with it and the codes are those of the h that the unquantized call stores.
//   - A stage holds rows of C G 8 values, zero past D, and so do the factors: the sums need no test for
//     the row's end (a test per chunk and use was a fifth of the instructions).
// Measured on B200, D = 3072, bf16: gate, post-norm, residual and modulated LayerNorm of two samples of 16896 rows
// 137 us (6.1 TB/s, 0.93 of a copy), of 4608 rows 24.1 us; a modulated LayerNorm of 4608 rows 13.2 us, of one row 4.2.
// Quantized, 4608 rows with y 26.8 us: no unit is full (issue 59 %, DRAM 42 % at 16896 rows); about four warps a
// scheduler wait for shared memory and shuffles and for the instruction before. Rows of 12288 with y, 4608 of them:
// 111 us, quantized 166 us; fp32 x and y, whose vectors are read per row there, 310 and 344 us.
// Every wait is bounded: one that runs out sets the status word and the block's abort flag, later waits
// then return at once, and the group's remaining copies are waited for before it leaves.
template <int C, int R, bool XF32, int Y, bool QUANT, bool SHARE, bool LAMBDAS = QUANT && SHARE>
__global__ void __launch_bounds__(32 * kMaxWarps, 1)
    block_norm_kernel(const __grid_constant__ Args a, int G, int stages, int factor_sets, unsigned long long wait_ns) {
  constexpr bool has_y = Y != kNoY;
  constexpr int xs = XF32 ? 4 : 2, ys = Y == kNoY ? 0 : Y == kF32Y ? 4 : 2;
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ float red_smem[2 * R * 16 * kMaxWarps];
  __shared__ __align__(8) uint64_t bars[kMaxWarps * kMaxStages];
  __shared__ int abort_smem;
  const int D = a.D, span = C * G * 8;
  const int group = threadIdx.x / G, t = threadIdx.x - group * G, groups = blockDim.x / G;
  const uint32_t bar0 = smem_addr(bars + group * kMaxStages);
  const int x_span = span * xs, row_bytes = span * (xs + ys), stage_bytes = R * row_bytes;
  uint8_t* const ring = ring_smem + static_cast<size_t>(group) * stages * stage_bytes;
  float* factors = reinterpret_cast<float*>(ring_smem + static_cast<size_t>(groups) * stages * stage_bytes);
  if (threadIdx.x == 0) abort_smem = 0;
  if (t == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(bar0 + 8 * i, 1);
    fence_barrier_init();
  }
  // zeros behind the rows, where the copies never write
  for (int r = 0; r < stages * R; ++r) {
    uint8_t* row = ring + r * row_bytes;
    for (int i = D * xs + 16 * t; i < x_span; i += 16 * G) *reinterpret_cast<uint4*>(row + i) = make_uint4(0u, 0u, 0u, 0u);
    for (int i = D * ys + 16 * t; i < span * ys; i += 16 * G)
      *reinterpret_cast<uint4*>(row + x_span + i) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  volatile int* abort_flag = &abort_smem;
  Reducer<R> red{red_smem + 2 * R * 16 * group, G >> 5, t >> 5, t & 31, 1 + group, 0};
  const int lane = t & 31;
  const int step = groups * R;
  // this block's share of the rows
  const int beg = static_cast<int>(static_cast<long long>(a.rows) * blockIdx.x / gridDim.x);
  const int end = static_cast<int>(static_cast<long long>(a.rows) * (blockIdx.x + 1) / gridDim.x);

  // the first warp's place in the group's batches, `stages` ahead of the group's
  uint32_t pending = 0;  // stages whose copies are under way and not yet seen to land
  int f_m = beg + group * R, f_end = beg, f_s = 0;
  auto fetch = [&](int stage) {
    if (t >= 32) return;
    while (f_m >= f_end) {  // into the next run that holds a batch of this group
      if (f_end >= end) return;
      const Run r = run_at(a, f_end, end);
      f_m = r.s >= 0 ? f_end + group * R : r.end;
      f_end = r.end;
      f_s = r.s;
    }
    if (*abort_flag) return;
    const uint32_t n = min(R, f_end - f_m);
    const uint32_t bar = bar0 + 8 * stage;
    if (lane == 0) mbar_arrive_expect_tx(bar, n * static_cast<uint32_t>(D) * (xs + ys));
    __syncwarp();
    if (lane < n) {
      const uint32_t dst = smem_addr(ring + stage * stage_bytes + lane * row_bytes);
      const long long m = f_m + lane;
      bulk_load(dst, static_cast<const uint8_t*>(a.x) + (m * a.ldx + f_s * a.adj_x) * xs, D * xs, bar);
      if (has_y) bulk_load(dst + x_span, static_cast<const uint8_t*>(a.y) + (m * a.ldy + f_s * a.adj_y) * ys, D * ys, bar);
    }
    pending |= 1u << stage;
    f_m += step;
  };
  auto join = [](const float4& l, const float4& h) -> F8 {
    return F8{{make_float2(l.x, l.y), make_float2(l.z, l.w), make_float2(h.x, h.y), make_float2(h.z, h.w)}};
  };
  // this thread's 8 elements of chunk c of a row in the stage
  auto get8 = [&](const uint8_t* p, bool f32, int c) -> F8 {
    if (f32) {
      const float4* q = reinterpret_cast<const float4*>(p) + 2 * (c * G + t);
      return join(q[0], q[1]);
    }
    return bf16x8(reinterpret_cast<const uint4*>(p)[c * G + t]);
  };
  // factors a2, b2 and, with y, a1: of every chunk first the low four, then the high four values of all
  // threads, so that 16-byte accesses of neighbouring threads meet no bank twice
  auto factor = [&](int which, int c) -> F8 {
    const float4* q = reinterpret_cast<const float4*>(factors + which * span) + 2 * c * G + t;
    return join(q[0], q[G]);
  };
  auto put_factor = [&](float* set, int which, int c, const float (&v)[8]) {
    float4* q = reinterpret_cast<float4*>(set + which * span) + 2 * c * G + t;
    q[0] = make_float4(v[0], v[1], v[2], v[3]);
    q[G] = make_float4(v[4], v[5], v[6], v[7]);
  };
  // the smoothing reciprocals of a quantized output: LAMBDAS laid out like a factor behind the factor sets
  float* const lambdas = factors + factor_sets * (has_y ? 3 : 2) * span;
  auto smooth = [&](int c) -> F8 {
    if constexpr (LAMBDAS) {
      const float4* q = reinterpret_cast<const float4*>(lambdas) + 2 * c * G + t;
      return join(q[0], q[G]);
    } else {
      float l[8];
      vec8<true>(l, Vec{a.inv_lambda, 0, 1}, 0, c, D, G, t);
      return pair8(l);
    }
  };
  const float inv_d = 1.0f / static_cast<float>(D);
  const int chunks = (D - 8 * t + 8 * G - 1) / (8 * G);  // of this thread that hold elements of the row
  const long long out_step = a.ld_out * xs, h_step = a.ldh * (a.h_f32 ? 4 : 2);
  const bool store_x = a.x_out != nullptr, store_h = a.h != nullptr, post_b = has_y && a.post.b.p != nullptr;
  const int post = a.post.kind, pre = a.pre.kind;
  const bool h_f32 = a.h_f32 != 0, skip_1 = a.skip == 1.0f;

  // the factors of sample s into set `set` (of factor_sets); the groups share the chunks
  float* const set0 = factors;
  const int set_len = (has_y ? 3 : 2) * span;
  auto build = [&](int s, int set) {
    float* const to = set0 + set * set_len;
    for (int c = group; c < C; c += groups) {
      float f[8], g[8];
      if (has_y) {
        post_factors<true>(a, s, c, G, t, f);
        put_factor(to, 2, c, f);
      }
      if (pre) {
        pre_factors<true>(a, s, c, G, t, f, g);
        const bool live = c < chunks;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          f[e] = live ? f[e] : 0.0f;
          g[e] = live ? g[e] : 0.0f;
        }
        put_factor(to, 0, c, f);
        put_factor(to, 1, c, g);
      }
    }
  };

  for (int i = 0; i < stages; ++i) fetch(i);
  if constexpr (LAMBDAS) {
    for (int c = group; c < C; c += groups) {
      float l[8];
      vec8<true>(l, Vec{a.inv_lambda, 0, 1}, 0, c, D, G, t);
      put_factor(lambdas, 0, c, l);
    }
  }
  int built = 0, seen = 0;  // runs of samples: with factors in shared memory, entered
  if constexpr (SHARE) {
    // the first factor_sets runs' factors at once: most blocks have no more, and entering a run then
    // waits for nobody (with one set a second run cost its block about 4 us)
    for (int m = beg; m < end && built < factor_sets;) {
      const Run r = run_at(a, m, end);
      if (r.s >= 0) build(r.s, built++);
      m = r.end;
    }
    __syncthreads();
  }
  int stage = 0;
  uint32_t phases = 0;
  for (int run_beg = beg; run_beg < end;) {
    const Run run = run_at(a, run_beg, end);
    const int s = run.s;
    if (SHARE && s >= 0) {
      if (seen == built) {
        __syncthreads();  // every group is through the runs before this one
        build(s, seen % factor_sets);
        ++built;
        __syncthreads();
      }
      factors = set0 + seen % factor_sets * set_len;
      ++seen;
    }
    for (int m = run_beg + group * R; m < run.end; m += step) {
      if (s < 0) {
        if constexpr (QUANT) {  // rows outside every sample (padding too) are quantized as zero
#pragma unroll
          for (int r = 0; r < R; ++r)
            if (m + r < run.end)
              for (int c = 0; c < C; ++c) {
                const int i = index<true>(c, 0, G, t);
                if (i < a.K_pad) {
                  *reinterpret_cast<uint32_t*>(a.codes + static_cast<size_t>(m + r) * (a.K_pad >> 1) + (i >> 1)) = 0u;
                  if ((i & 31) == 0) a.sf[mx::act_sf_offset(m + r, i >> 5, a.K_pad)] = 0;
                }
              }
        }
        continue;
      }
      const uint8_t* const buf = ring + stage * stage_bytes;
      // the waiting warps sleep: spinning ones would take issue slots from the groups at work
      if (mbar_wait_bounded(bar0 + 8 * stage, (phases >> stage) & 1u, wait_ns, &g_svdq_status, kStatusProducer,
                            abort_flag, true)) {
        pending &= ~(1u << stage);
        phases ^= 1u << stage;
      }
      F8 v[R][C];
      float mean[R], rstd[R];
      if constexpr (has_y) {
        const uint8_t* const yb = buf + x_span;
#pragma unroll
        for (int r = 0; r < R; ++r) mean[r] = 0.0f, rstd[r] = 1.0f;
        if (post == 2) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float2 q = dup2(0.0f);
#pragma unroll
            for (int c = 0; c < C; ++c) {
              const F8 u = get8(yb + r * row_bytes, Y == kF32Y, c);
              q = add2(q, add2(add2(u.p[0], u.p[1]), add2(u.p[2], u.p[3])));
            }
            mean[r] = q.x + q.y;
          }
          red.sum(mean);
#pragma unroll
          for (int r = 0; r < R; ++r) mean[r] *= inv_d;
        }
        if (post) {
#pragma unroll
          for (int r = 0; r < R; ++r) {
            float2 q[2] = {dup2(0.0f), dup2(0.0f)};
#pragma unroll
            for (int c = 0; c < C; ++c) {
              F8 u = get8(yb + r * row_bytes, Y == kF32Y, c);
              if (post == 2) {
                const float2 neg = dup2(c < chunks ? -mean[r] : 0.0f);
#pragma unroll
                for (int j = 0; j < 4; ++j) u.p[j] = add2(u.p[j], neg);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) q[j & 1] = fma2(u.p[j], u.p[j], q[j & 1]);
            }
            q[0] = add2(q[0], q[1]);
            rstd[r] = q[0].x + q[0].y;
          }
          red.sum(rstd);
#pragma unroll
          for (int r = 0; r < R; ++r) rstd[r] = root(rstd[r], inv_d, a.post.eps);
        }
        uint8_t* const x_row = static_cast<uint8_t*>(a.x_out) + m * out_step + s * a.adj_out * xs;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          F8 f;
          if constexpr (SHARE) {
            f = factor(2, c);
          } else {
            float f8[8];
            post_factors<true>(a, s, c, G, t, f8);
            f = pair8(f8);
          }
#pragma unroll
          for (int r = 0; r < R; ++r) {
            F8 u = get8(yb + r * row_bytes, Y == kF32Y, c), x = get8(buf + r * row_bytes, XF32, c);
            if (post == 2) {
              const float2 neg = dup2(c < chunks ? -mean[r] : 0.0f);
#pragma unroll
              for (int j = 0; j < 4; ++j) u.p[j] = add2(u.p[j], neg);
            }
            if (!skip_1) {
              const float2 skip = dup2(a.skip);
#pragma unroll
              for (int j = 0; j < 4; ++j) x.p[j] = mul2_rn(skip, x.p[j]);
            }
            const float2 k = dup2(rstd[r]);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[r][c].p[j] = fma2(mul2_rn(u.p[j], k), f.p[j], x.p[j]);
            if (post_b) {
              float b[8];
              post_bias<true>(a, s, c, G, t, b);
              const F8 b8 = pair8(b);
#pragma unroll
              for (int j = 0; j < 4; ++j) v[r][c].p[j] = add2(v[r][c].p[j], b8.p[j]);
            }
            if (store_x && c < chunks && (R == 1 || m + r < run.end))
              store8(v[r][c], x_row + r * out_step, XF32, index<true>(c, 0, G, t));
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int r = 0; r < R; ++r) v[r][c] = get8(buf + r * row_bytes, XF32, c);
      }
      red.sync();  // the group has read the stage
      fetch(stage);
      if (++stage == stages) stage = 0;
      if (!pre) continue;
      if (pre == 2) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          float2 q = dup2(0.0f);
#pragma unroll
          for (int c = 0; c < C; ++c) q = add2(q, add2(add2(v[r][c].p[0], v[r][c].p[1]), add2(v[r][c].p[2], v[r][c].p[3])));
          mean[r] = q.x + q.y;
        }
        red.sum(mean);
#pragma unroll
        for (int r = 0; r < R; ++r) {
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const float2 neg = dup2(c < chunks ? -mean[r] * inv_d : 0.0f);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[r][c].p[j] = add2(v[r][c].p[j], neg);
          }
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float2 q[2] = {dup2(0.0f), dup2(0.0f)};
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) q[j & 1] = fma2(v[r][c].p[j], v[r][c].p[j], q[j & 1]);
        q[0] = add2(q[0], q[1]);
        rstd[r] = q[0].x + q[0].y;
      }
      red.sum(rstd);
#pragma unroll
      for (int r = 0; r < R; ++r) rstd[r] = root(rstd[r], inv_d, a.pre.eps);
      uint8_t* const h_row = static_cast<uint8_t*>(a.h) + m * h_step + s * a.adj_h * (h_f32 ? 4 : 2);
      const long long code_step = a.K_pad >> 1;
      uint8_t* const code_row = a.codes + m * code_step;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int i = index<true>(c, 0, G, t);
        const bool on = c < chunks;
        F8 f, g;
        if constexpr (SHARE) {
          f = factor(0, c);
          g = factor(1, c);
        } else {
          float f8[8], g8[8];
          pre_factors<true>(a, s, c, G, t, f8, g8);
          f = pair8(f8);
          g = pair8(g8);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float2 k = dup2(rstd[r]);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[r][c].p[j] = fma2(mul2_rn(v[r][c].p[j], k), f.p[j], g.p[j]);
          if (store_h && on && (R == 1 || m + r < run.end)) store8(v[r][c], h_row + r * h_step, h_f32, i);
          if constexpr (QUANT) {
            // the codes svdq_mx_quantize_act makes of bf16(h): smoothing in fp32, blocks of four lanes
            F8 q = bf16x8(pack8_bf16(v[r][c]));
            const F8 l = smooth(c);
#pragma unroll
            for (int j = 0; j < 4; ++j) q.p[j] = mul2_rn(q.p[j], l.p[j]);  // past D: 0, or NaN in a row of NaN
            uint32_t sc;
            const uint32_t codes = mx::quarter_block(q.p, sc);
            // the scales of four blocks (16 lanes) go out as one word
            sc <<= 2 * (lane & 12);
            sc |= __shfl_xor_sync(0xffffffffu, sc, 4);
            sc |= __shfl_xor_sync(0xffffffffu, sc, 8);
            if (i < a.K_pad && (R == 1 || m + r < run.end)) {
              *reinterpret_cast<uint32_t*>(code_row + r * code_step + (i >> 1)) = codes;
              if ((lane & 15) == 0)
                *reinterpret_cast<uint32_t*>(a.sf + mx::act_sf_offset(m + r, 0, a.K_pad) + ((i >> 7) << 9)) = sc;
            }
          }
        }
      }
    }
    run_beg = run.end;
  }
  if (t == 0)
    for (int i = 0; i < stages; ++i)
      if (pending & (1u << i))
        mbar_wait_bounded(bar0 + 8 * i, (phases >> i) & 1u, wait_ns, &g_svdq_status, kStatusDrain, nullptr);
}

}  // namespace norm
}  // namespace svdq
