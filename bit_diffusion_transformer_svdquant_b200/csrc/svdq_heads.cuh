// What stands between a fused QKV product and attention: the norm over each head, rotary positions, and a paged
// key/value cache in 8 or 4 bits that is quantized as it is written and read back as values.
//
// Rotation of the first `dim` values of a head, pair p of dim / 2 on axis a(p), by the angle pos[a] f_p:
//   o0 = A (x0 cos - x1 sin),  o1 = A (x1 cos + x0 sin)
// on (x[2p], x[2p + 1]) (interleaved) or (x[p], x[p + dim/2]) (half). The frequency comes as turns per position
// in 64-bit fixed point, F = round(f / 2 pi 2^64): the low 64 bits of pos F are the turns modulo one, off by |pos| 2^-65 at
// most, of which the kernel keeps the upper 32 (in fp32, pos f is off by 0.03 rad at a position of 10^6). So an angle
// is that of f to |pos| 2^-65 + 2^-32 turns; the first term passes the second beyond |pos| = 2^33.
//
// Everything between a load and its store is fp32; norm statistics too.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "svdq_fp8b.cuh"
#include "svdq_mx.cuh"
#include "svdq_ptx.cuh"
#include "svdq_quant.cuh"

namespace svdq {
namespace heads {

constexpr int kMaxAxes = 4;
constexpr int kMaxD = 256;
constexpr int kThreads = 256;

struct Rope {
  const unsigned long long* turns;  // [dim / 2]
  const void* pos;                  // row (b, t), axis a at b pb + t pt + a
  long long pb, pt;
  int dim, half, pos_i64, inverse;
  int axis_end[kMaxAxes];           // pairs up to the end of each axis
  float amplitude;
};
// One tensor's heads: row (b, t), head h at b sb + t st + h sh; out the same way, or a plane of the cache.
struct Part {
  const void* x;
  long long sb, st, sh;
  void* out;
  long long ob, ot, oh;
  const void* weight;
  const void* bias;
  float eps;
  int heads, norm, nf32, rotate, quant;  // norm: 0 none, 1 rms, 2 layer
  uint8_t* codes;
  uint8_t* scales;
};
struct Cache {
  int page_size, heads, D, mx;   // mx: 1 MXFP4, 0 FP8
  int code_bytes, scale_bytes;   // per head
  long long slots;               // pages x page_size
};
struct Args {
  Part part[3];
  Rope rope;
  Cache cache;
  const void* slots;
  int slots_i64;
  int samples, rows_per_sample, D, out_f32, parts;
  int strip;  // rows per block
};

__device__ __forceinline__ long long load_index(const void* p, long long i, int i64) {
  return i64 ? __ldg(static_cast<const long long*>(p) + i) : __ldg(static_cast<const int*>(p) + i);
}

__device__ __forceinline__ float2 fma2_rn(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
        "l"(*reinterpret_cast<const uint64_t*>(&c)));
  return *reinterpret_cast<const float2*>(&r);
}
__device__ __forceinline__ float2 sub2_rn(float2 a, float2 b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&r);
}

// Cosine and sine of `turn` of 2^32 parts of a circle. The nearest quarter circle is taken off exactly, in integers; of
// the rest, x within +-pi/4, both Taylor series to x^8 and x^9 (their next terms are below 2.5e-8 and 1.8e-9), in one
// packed chain.
__device__ __forceinline__ float2 cos_sin(uint32_t turn) {
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float x = static_cast<float>(static_cast<int>(turn - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float x2 = x * x;
  const float2 y = make_float2(x2, x2);
  float2 p = fma2_rn(y, make_float2(1.0f / 40320.0f, 1.0f / 362880.0f), make_float2(-1.0f / 720.0f, -1.0f / 5040.0f));
  p = fma2_rn(p, y, make_float2(1.0f / 24.0f, 1.0f / 120.0f));
  p = fma2_rn(p, y, make_float2(-0.5f, -1.0f / 6.0f));
  const float c = fmaf(p.x, x2, 1.0f), s = fmaf(p.y * x2, x, x);
  // a quarter turn takes (c, s) to (-s, c), a half to (-c, -s)
  const float u = quarter & 1u ? s : c, v = quarter & 1u ? c : s;
  return make_float2(__uint_as_float(__float_as_uint(u) ^ (((quarter + 1u) & 2u) << 30)),
                     __uint_as_float(__float_as_uint(v) ^ ((quarter & 2u) << 30)));
}
__device__ __forceinline__ int axis_of(const Rope& r, int p) {
  int a = 0;
#pragma unroll
  for (int i = 0; i + 1 < kMaxAxes; ++i) a += p >= r.axis_end[i] ? 1 : 0;
  return a;
}
// cos and sin of a position times a frequency, times the amplitude
__device__ __forceinline__ float2 rotation(const Rope& r, long long position, unsigned long long turns) {
  const float2 cs = cos_sin(static_cast<uint32_t>((static_cast<unsigned long long>(position) * turns) >> 32));
  return make_float2(r.amplitude * cs.x, (r.inverse ? -r.amplitude : r.amplitude) * cs.y);
}

// ---------------------------------------------------------------- a lane's 8 values
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 w = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                     __uint_as_float(w.y & 0xFFFF0000u));
}
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 vector4(const void* p, int at, int f32) {
  return f32 ? load4(static_cast<const float*>(p) + at) : load4(static_cast<const __nv_bfloat16*>(p) + at);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
// The 8 values of a lane as the pairs that rotate, two pairs to a register pair for packed fp32 arithmetic: x0 holds
// the first values of pairs 0, 1 | 2, 3, x1 the second ones. In memory the lane's values are two runs of 4 (at o0 and
// o1, o0 + 4 where they are contiguous): pairs across the runs in the half layout, within a run otherwise.
struct Pairs {
  float2 x0[2], x1[2];
};
template <bool HALF>
__device__ __forceinline__ Pairs to_pairs(const float4& r0, const float4& r1) {
  Pairs v;
  if constexpr (HALF) {
    v.x0[0] = make_float2(r0.x, r0.y), v.x0[1] = make_float2(r0.z, r0.w);
    v.x1[0] = make_float2(r1.x, r1.y), v.x1[1] = make_float2(r1.z, r1.w);
  } else {
    v.x0[0] = make_float2(r0.x, r0.z), v.x1[0] = make_float2(r0.y, r0.w);
    v.x0[1] = make_float2(r1.x, r1.z), v.x1[1] = make_float2(r1.y, r1.w);
  }
  return v;
}
template <bool HALF>
__device__ __forceinline__ void to_runs(const Pairs& v, float (&x)[8]) {
  if constexpr (HALF) {
    x[0] = v.x0[0].x, x[1] = v.x0[0].y, x[2] = v.x0[1].x, x[3] = v.x0[1].y;
    x[4] = v.x1[0].x, x[5] = v.x1[0].y, x[6] = v.x1[1].x, x[7] = v.x1[1].y;
  } else {
    x[0] = v.x0[0].x, x[1] = v.x1[0].x, x[2] = v.x0[0].y, x[3] = v.x1[0].y;
    x[4] = v.x0[1].x, x[5] = v.x1[1].x, x[6] = v.x0[1].y, x[7] = v.x1[1].y;
  }
}
// The values as they were loaded
template <class T, bool HALF>
struct Raw;
template <bool HALF>
struct Raw<__nv_bfloat16, HALF> {
  uint4 w;
  __device__ void load(const __nv_bfloat16* p, int o0, int o1) {
    if constexpr (HALF) {
      const uint2 lo = *reinterpret_cast<const uint2*>(p + o0), hi = *reinterpret_cast<const uint2*>(p + o1);
      w = make_uint4(lo.x, lo.y, hi.x, hi.y);
    } else {
      w = *reinterpret_cast<const uint4*>(p + o0);
    }
  }
  __device__ void zero() { w = make_uint4(0u, 0u, 0u, 0u); }
  __device__ Pairs pairs() const {
    auto lo = [](uint32_t u) { return __uint_as_float(u << 16); };
    auto hi = [](uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); };
    return to_pairs<HALF>(make_float4(lo(w.x), hi(w.x), lo(w.y), hi(w.y)), make_float4(lo(w.z), hi(w.z), lo(w.w), hi(w.w)));
  }
};
template <bool HALF>
struct Raw<float, HALF> {
  float4 w[2];
  __device__ void load(const float* p, int o0, int o1) {
    w[0] = load4(p + o0);
    w[1] = load4(p + o1);
  }
  __device__ void zero() { w[0] = w[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ Pairs pairs() const { return to_pairs<HALF>(w[0], w[1]); }
};

// ---------------------------------------------------------------- heads of whole groups of 8 values
// A head is a group of G lanes (D / 8, up to a power of two, at least 4), 8 values each: contiguous ones, or, of the
// rotated values in the half layout, 4 of each half, so that a lane holds both values of its pairs: pairs 4 l ..
// 4 l + 3 either way. A warp owns 32 / G heads of one part and a block the heads of up to 8 warps (blockIdx.y); both go down a
// strip of rows (blockIdx.x) of one sample (blockIdx.z). So a lane's columns, weights and strides are fixed and a row
// costs it a load, a store and the arithmetic; kAhead rows of loads are in flight. The cosines and sines of kBatch
// rows are computed by the whole block at a time, into one half of a table while the heads read the other.
// Measured on B200: q and k of 16896 rows of 24 heads of 128 with norms 69.7 us (6.0 TB/s, 0.91 of the copy rate), 4608 rows
// 22.5 us, without norms 21.3; 16384 tokens written in FP8 with q 103 us (4.9 TB/s); one token 3.0 us. What bounds it is the
// latency that 32 warps an SM leave uncovered (of 13 warps per issue 5.3 wait for memory in the first) together with
// instruction issue (56 %; in the write 63 %). With a warp per row and its heads in turn (coefficients in registers,
// pointers per head) the first took 83 us. Heads of other sizes, 16896 rows of as many bytes: 64 70.6 us; 256 81.9, 96 89.0,
// 80 103, 40 104, 72 117: all in the form with branches, and lanes past D / 8 idle (3 of 8 at 40, 7 of 16 at 72).
template <class T>
constexpr int kAhead = sizeof(T) == 2 ? 4 : 2;
constexpr int kBatch = 8;
enum Destination { kBf16, kF32, kFp8, kMx };

// What a lane knows of its head
struct Place {
  int G, l, h;
  bool in;       // inside the head, and the head exists
  bool turns;    // its pairs rotate
  int o0, run;   // its first 4 values, and the other 4 from there
};
struct Strip {
  int b, t0, rows;
};

// KG: G where it is known at compile time, else 0
template <int KG, class F>
__device__ __forceinline__ float across(int G, float v, F f) {
  if constexpr (KG > 0) {
#pragma unroll
    for (int o = KG >> 1; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  } else {
    for (int o = G >> 1; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
  }
  return v;
}

// Shared memory: of two batches of rows, the cosines, then the sines of each row (kMaxD / 2 places each, so that
// offsets are constants), and where its token goes in the cache: byte offsets of the slot's codes and scales, -1 for
// none.
struct Tables {
  float angles[2][kBatch][kMaxD];
  longlong2 slots[2][kBatch];
  ulonglong2 pairs[kMaxD / 2];  // frequency and axis
};

// The tables of the rows from `first` on of a strip (one batch), a warp per row
__device__ __forceinline__ void fill_tables(const Args& a, Tables& tb, const Strip& st, int first, bool angles) {
  const int lane = threadIdx.x & 31, half = first / kBatch & 1;
  for (int r = threadIdx.x >> 5; r < kBatch && first + r < st.rows; r += blockDim.x >> 5) {
    if (angles) {
      const long long row = st.b * a.rope.pb + (st.t0 + first + r) * a.rope.pt;
      for (int p = lane; p < a.rope.dim >> 1; p += 32) {
        const ulonglong2 pair = tb.pairs[p];
        const float2 cs = rotation(a.rope, load_index(a.rope.pos, row + static_cast<int>(pair.y), a.rope.pos_i64), pair.x);
        tb.angles[half][r][p] = cs.x;
        tb.angles[half][r][kMaxD / 2 + p] = cs.y;
      }
    }
    if (a.slots != nullptr && lane == 0) {
      const long long row = static_cast<long long>(st.b) * a.rows_per_sample + st.t0 + first + r;
      const long long slot = load_index(a.slots, row, a.slots_i64);
      const bool is = slot >= 0 && slot < a.cache.slots;
      const long long head = slot * a.cache.heads;
      tb.slots[half][r] = make_longlong2(is ? head * a.cache.code_bytes : -1, is ? head * a.cache.scale_bytes : -1);
    }
  }
}

// This warp's heads down the strip. What a part may ask for (kAny), or without the branches that keep the compiler from
// running rows side by side: no norm or an rms norm without a bias, and all lanes rotate (kTurn) or none (kStay). With kAny for all, q and k of 16896
// rows take 72.7 us instead of 69.6, and the write of 16384 tokens 110 instead of 103.
enum Form { kAny, kTurn, kStay };
template <class T, bool HALF, int KG, int DST, bool NORM, int FORM>
__device__ __forceinline__ void run_strip(const Args& a, const Part& p, const Place& at, const Strip& st, Tables& tb,
                                          bool angles) {
  constexpr bool kQuant = DST == kFp8 || DST == kMx;
  constexpr int N = kAhead<T>, kSize = DST == kF32 ? 4 : 2;
  const auto add = [](float x, float y) { return x + y; };
  const T* src = static_cast<const T*>(p.x) + st.b * p.sb + st.t0 * p.st + at.h * p.sh + at.o0;
  Raw<T, HALF> raw[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    raw[u].zero();  // lanes past the head stay zero
    if (at.in) raw[u].load(src + min(u, st.rows - 1) * p.st, 0, at.run);
  }
  src += min(N, st.rows - 1) * p.st;
  Pairs w;
  if constexpr (NORM) {
    const float4 one = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    const bool has = at.in && p.weight != nullptr;
    w = to_pairs<HALF>(has ? vector4(p.weight, at.o0, p.nf32) : one, has ? vector4(p.weight, at.o0 + at.run, p.nf32) : one);
  }
  const float inv_d = NORM ? 1.0f / static_cast<float>(a.D) : 0.0f;
  char* out = nullptr;
  if constexpr (kQuant) out = reinterpret_cast<char*>(p.codes) + at.h * a.cache.code_bytes + (DST == kMx ? 4 * at.l : at.o0);
  else out = static_cast<char*>(p.out) + (st.b * p.ob + st.t0 * p.ot + at.h * p.oh + at.o0) * kSize;
  const bool layer = p.norm == 2, has_bias = p.bias != nullptr && at.in;
  const long long src_step = p.st, out_step = p.ot * kSize;
  // row i of the strip, r of its batch; past the end (the rest of a group of N) the last row's values go nowhere
  const int last = st.rows - 1;
  auto row = [&](int i, int r, int half, Raw<T, HALF>& mine) {
    Pairs v = mine.pairs();
    if (at.in) mine.load(src, 0, at.run);
    src += i + N < last ? src_step : 0;
    const bool stored = at.in && i <= last;
    float k = 1.0f;
    if constexpr (NORM) {
      if (FORM == kAny && layer) {
        float2 q = mx::add2_rn(mx::add2_rn(v.x0[0], v.x0[1]), mx::add2_rn(v.x1[0], v.x1[1]));
        const float mean = across<KG>(at.G, q.x + q.y, add) * inv_d;
        const float m = at.in ? -mean : 0.0f;  // lanes past the head stay zero
        const float2 m2 = make_float2(m, m);
#pragma unroll
        for (int i = 0; i < 2; ++i) v.x0[i] = mx::add2_rn(v.x0[i], m2), v.x1[i] = mx::add2_rn(v.x1[i], m2);
      }
      float2 q = mul2_rn(v.x0[0], v.x0[0]);
      q = fma2_rn(v.x0[1], v.x0[1], q);
      q = fma2_rn(v.x1[0], v.x1[0], q);
      q = fma2_rn(v.x1[1], v.x1[1], q);
      k = rsqrtf(fmaf(across<KG>(at.G, q.x + q.y, add), inv_d, p.eps));  // off by 2 steps at most
      // the factor follows the rotation where no bias stands between: the sum is then waited for last
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (FORM == kAny) {
          v.x0[i] = mul2_rn(v.x0[i], make_float2(k, k));
          v.x1[i] = mul2_rn(v.x1[i], make_float2(k, k));
        }
        v.x0[i] = mul2_rn(v.x0[i], w.x0[i]);
        v.x1[i] = mul2_rn(v.x1[i], w.x1[i]);
      }
      if (FORM == kAny && has_bias) {
        const Pairs z = to_pairs<HALF>(vector4(p.bias, at.o0, p.nf32), vector4(p.bias, at.o0 + at.run, p.nf32));
#pragma unroll
        for (int i = 0; i < 2; ++i) v.x0[i] = mx::add2_rn(v.x0[i], z.x0[i]), v.x1[i] = mx::add2_rn(v.x1[i], z.x1[i]);
      }
    }
    if (FORM == kTurn || (FORM == kAny && at.turns)) {
      const float4 c = load4(&tb.angles[half][r][4 * at.l]), s = load4(&tb.angles[half][r][kMaxD / 2 + 4 * at.l]);
      const float2 c2[2] = {make_float2(c.x, c.y), make_float2(c.z, c.w)};
      const float2 s2[2] = {make_float2(s.x, s.y), make_float2(s.z, s.w)};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 x0 = v.x0[i], x1 = v.x1[i];
        v.x0[i] = sub2_rn(mul2_rn(x0, c2[i]), mul2_rn(x1, s2[i]));
        v.x1[i] = fma2_rn(x1, c2[i], mul2_rn(x0, s2[i]));
      }
    }
    if constexpr (NORM && FORM != kAny) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        v.x0[i] = mul2_rn(v.x0[i], make_float2(k, k));
        v.x1[i] = mul2_rn(v.x1[i], make_float2(k, k));
      }
    }
    if constexpr (!kQuant) {
      float x[8];
      to_runs<HALF>(v, x);
      if (stored) {
        if constexpr (DST == kBf16) {
          __nv_bfloat16* const o = reinterpret_cast<__nv_bfloat16*>(out);
          const uint2 lo = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
          const uint2 hi = make_uint2(pack2(x[4], x[5]), pack2(x[6], x[7]));
          if constexpr (HALF) {
            *reinterpret_cast<uint2*>(o) = lo;
            *reinterpret_cast<uint2*>(o + at.run) = hi;
          } else {
            *reinterpret_cast<uint4*>(o) = make_uint4(lo.x, lo.y, hi.x, hi.y);
          }
        } else {
          float* const o = reinterpret_cast<float*>(out);
          *reinterpret_cast<float4*>(o) = make_float4(x[0], x[1], x[2], x[3]);
          *reinterpret_cast<float4*>(o + at.run) = make_float4(x[4], x[5], x[6], x[7]);
        }
      }
      out += out_step;
    } else if constexpr (DST == kFp8) {
      const float m0 = mx::max3_nan_abs(v.x0[0].x, v.x0[0].y, v.x0[1].x);
      const float m1 = mx::max3_nan_abs(v.x0[1].y, v.x1[0].x, v.x1[0].y);
      float am = mx::max_nan_abs(mx::max3_nan_abs(m0, m1, v.x1[1].x), v.x1[1].y);
      am = across<KG>(at.G, am, [](float x, float y) { return mx::max_nan_abs(x, y); });
      const uint32_t s = fp8b::scale_code(am);
      const float f = mx::scale_inverse(s);
      const float2 f2 = make_float2(f, f);
#pragma unroll
      for (int i = 0; i < 2; ++i) v.x0[i] = mul2_rn(v.x0[i], f2), v.x1[i] = mul2_rn(v.x1[i], f2);
      float x[8];
      to_runs<HALF>(v, x);
      uint2 q = make_uint2(fp8r::cvt_e4m3x2(x[0], x[1]) | (fp8r::cvt_e4m3x2(x[2], x[3]) << 16),
                           fp8r::cvt_e4m3x2(x[4], x[5]) | (fp8r::cvt_e4m3x2(x[6], x[7]) << 16));
      if (s == 255u) q = make_uint2(0u, 0u);
      const longlong2 to = tb.slots[half][r];
      if (stored && to.x >= 0) {
        char* const o = out + to.x;
        if constexpr (HALF) {
          *reinterpret_cast<uint32_t*>(o) = q.x;
          *reinterpret_cast<uint32_t*>(o + at.run) = q.y;
        } else {
          *reinterpret_cast<uint2*>(o) = q;
        }
        if (at.l == 0) p.scales[to.y + at.h] = static_cast<uint8_t>(s);
      }
    } else {
      float x[8];
      to_runs<HALF>(v, x);
      if (HALF && p.rotate != 0) {
        // blocks are of consecutive values: from runs of 4 in two halves to 8 in a row. Run c is lane c's first,
        // lane c - dim/8's second, or past the rotated values where it lies.
        const int eighth = a.rope.dim >> 3;
        float y[8];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = 2 * at.l + j;
          const int from = c < eighth ? c : c < 2 * eighth ? c - eighth : at.l;
          const bool second = c < eighth ? false : c < 2 * eighth ? true : j == 1;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float lo = __shfl_sync(0xffffffffu, x[i], from, at.G), hi = __shfl_sync(0xffffffffu, x[4 + i], from, at.G);
            y[4 * j + i] = second ? hi : lo;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = at.in ? y[i] : 0.0f;
      }
      const float2 v2[4] = {make_float2(x[0], x[1]), make_float2(x[2], x[3]), make_float2(x[4], x[5]),
                            make_float2(x[6], x[7])};
      uint32_t s;
      const uint32_t q = mx::quarter_block(v2, s);
      const longlong2 to = tb.slots[half][r];
      if (stored && to.x >= 0) {
        *reinterpret_cast<uint32_t*>(out + to.x) = q;
        if ((at.l & 3) == 0) p.scales[to.y + at.h * a.cache.scale_bytes + (at.l >> 2)] = static_cast<uint8_t>(s);
      }
    }
  };
  fill_tables(a, tb, st, 0, angles);
  __syncthreads();
  if (st.rows == 1) {  // few rows: one body instead of N (one token, q and k of 24 heads of 128: 3.7 -> 2.5 us)
    row(0, 0, 0, raw[0]);
    return;
  }
  for (int first = 0; first < st.rows; first += kBatch) {
    if (first + kBatch < st.rows) fill_tables(a, tb, st, first + kBatch, angles);
    const int half = first / kBatch & 1;
    // N bodies without a branch between them: with the whole batch unrolled, and a form of its own for the strip's end,
    // the parts' code did not fit the instruction cache (16384 tokens written: of 13 stalled warps 1.45 waited for
    // instructions)
#pragma unroll 1
    for (int r0 = 0; r0 < kBatch && first + r0 < st.rows; r0 += N)
#pragma unroll
      for (int u = 0; u < N; ++u) row(first + r0 + u, r0 + u, half, raw[u]);
    __syncthreads();
  }
}

// CACHE: where quantized parts go, kFp8 or kMx; kBf16 without any
template <class T, bool HALF, int KG, int CACHE>
__global__ void __launch_bounds__(kThreads, 4) heads_kernel(const __grid_constant__ Args a, int G) {
  __shared__ __align__(16) Tables tb;
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  Place at;
  at.G = KG > 0 ? KG : G;
  const int per_warp = 32 / at.G;
  at.l = lane & (at.G - 1);
  // this warp's part and heads: parts take whole warps each
  int unit = blockIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5), pi = 0;
  while (pi + 1 < a.parts && unit * per_warp >= a.part[pi].heads) {
    unit -= (a.part[pi].heads + per_warp - 1) / per_warp;
    ++pi;
  }
  const Part& p = a.part[pi];
  at.h = unit * per_warp + lane / at.G;
  at.in = 8 * at.l < a.D && at.h < p.heads;
  at.turns = p.rotate != 0 && 8 * at.l < a.rope.dim;
  const bool split = HALF && at.turns;
  at.o0 = (split ? 4 : 8) * at.l, at.run = split ? a.rope.dim >> 1 : 4;
  Strip st;
  st.b = blockIdx.z, st.t0 = blockIdx.x * a.strip;
  st.rows = min(a.strip, a.rows_per_sample - st.t0);
  const bool idle = unit * per_warp >= p.heads;
  for (int i = threadIdx.x; i < a.rope.dim >> 1; i += blockDim.x)
    tb.pairs[i] = make_ulonglong2(__ldg(a.rope.turns + i), axis_of(a.rope, i));
  const bool angles = __syncthreads_or(p.rotate && !idle) != 0;  // whether a head of the block rotates
  if (idle) {  // no head left for this warp: it takes its part of the tables only
    fill_tables(a, tb, st, 0, angles);
    __syncthreads();
    for (int first = 0; first < st.rows && st.rows > 1; first += kBatch) {
      if (first + kBatch < st.rows) fill_tables(a, tb, st, first + kBatch, angles);
      __syncthreads();
    }
    return;
  }
  auto run = [&](auto norm, auto form) {
    constexpr bool kNorm = decltype(norm)::value;
    constexpr int kForm = decltype(form)::value;
    if constexpr (CACHE != kBf16) {
      if (p.quant) return run_strip<T, HALF, KG, CACHE, kNorm, kForm>(a, p, at, st, tb, angles);
    }
    if (a.out_f32) run_strip<T, HALF, KG, kF32, kNorm, kForm>(a, p, at, st, tb, angles);
    else run_strip<T, HALF, KG, kBf16, kNorm, kForm>(a, p, at, st, tb, angles);
  };
  if constexpr (KG > 0) {
    if (a.D == 8 * KG && p.norm != 2 && p.bias == nullptr) {
      if (p.rotate != 0 && a.rope.dim == a.D) {
        if (p.norm != 0) return run(std::true_type{}, std::integral_constant<int, kTurn>{});
        return run(std::false_type{}, std::integral_constant<int, kTurn>{});
      }
      if (p.rotate == 0 && p.norm == 0) return run(std::false_type{}, std::integral_constant<int, kStay>{});
    }
  }
  if (p.norm != 0) run(std::true_type{}, std::integral_constant<int, kAny>{});
  else run(std::false_type{}, std::integral_constant<int, kAny>{});
}

// ---------------------------------------------------------------- any head size, stride and alignment
// A warp per head; value d is lane d % 32's, and its partner comes through shared memory. Not fast: one head in
// flight per warp, element by element, angles by each head (4608 rows, q and k of 24 heads of 126, or of 128 off 16 bytes:
// 197 us with norms, 151 without; of 128 by the kernel above 22.5 and 21.3).
template <class T>
__global__ void __launch_bounds__(kThreads) heads_any_kernel(const __grid_constant__ Args a) {
  constexpr int kPer = kMaxD / 32;
  __shared__ float buf[kThreads / 32][kMaxD];
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x, b = row / a.rows_per_sample, t = row - b * a.rows_per_sample;
  const int pairs = a.rope.dim >> 1;
  float* const x = buf[warp];
  auto value = [&](const void* p, int at, int f32) {
    return f32 ? static_cast<const float*>(p)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
  };
  auto sum = [&](float s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  };
  for (int pi = 0; pi < a.parts; ++pi) {
    const Part& p = a.part[pi];
    for (int h = blockIdx.y * (kThreads / 32) + warp; h < p.heads; h += gridDim.y * (kThreads / 32)) {
      const T* src = static_cast<const T*>(p.x) + b * p.sb + t * p.st + h * p.sh;
      float v[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int d = 32 * i + lane;
        v[i] = d < a.D ? static_cast<float>(src[d]) : 0.0f;
      }
      if (p.norm != 0) {
        if (p.norm == 2) {
          float s = 0.0f;
#pragma unroll
          for (int i = 0; i < kPer; ++i) s += v[i];
          const float mean = sum(s) / static_cast<float>(a.D);
#pragma unroll
          for (int i = 0; i < kPer; ++i) v[i] = 32 * i + lane < a.D ? v[i] - mean : 0.0f;
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) s = fmaf(v[i], v[i], s);
        const float k = 1.0f / sqrtf(sum(s) / static_cast<float>(a.D) + p.eps);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int d = 32 * i + lane;
          if (d < a.D)
            v[i] = fmaf(v[i] * k, p.weight != nullptr ? value(p.weight, d, p.nf32) : 1.0f,
                        p.bias != nullptr ? value(p.bias, d, p.nf32) : 0.0f);
        }
      }
      if (p.rotate) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[32 * i + lane] = v[i];
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int d = 32 * i + lane;
          if (d >= a.rope.dim) continue;
          const bool second = a.rope.half ? d >= pairs : (d & 1) != 0;
          const int pair = a.rope.half ? (second ? d - pairs : d) : d >> 1;
          const int other = a.rope.half ? (second ? d - pairs : d + pairs) : d ^ 1;
          const float2 cs = rotation(a.rope, load_index(a.rope.pos, b * a.rope.pb + t * a.rope.pt + axis_of(a.rope, pair),
                                                        a.rope.pos_i64), __ldg(a.rope.turns + pair));
          v[i] = second ? v[i] * cs.x + x[other] * cs.y : v[i] * cs.x - x[other] * cs.y;
        }
      }
      if (!p.quant) {
        const long long at = b * p.ob + t * p.ot + h * p.oh;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int d = 32 * i + lane;
          if (d >= a.D) continue;
          if (a.out_f32) static_cast<float*>(p.out)[at + d] = v[i];
          else static_cast<__nv_bfloat16*>(p.out)[at + d] = __float2bfloat16_rn(v[i]);
        }
        continue;
      }
      const long long slot = load_index(a.slots, row, a.slots_i64);
      const bool stored = slot >= 0 && slot < a.cache.slots;
      const long long head = slot * p.heads + h;
      if (!a.cache.mx) {
        float am = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) am = mx::max_nan_abs(am, v[i]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) am = mx::max_nan_abs(am, __shfl_xor_sync(0xffffffffu, am, o));
        const uint32_t s = fp8b::scale_code(am);
        const float f = mx::scale_inverse(s);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int d = 32 * i + lane;
          if (stored && d < a.D)
            p.codes[head * a.cache.code_bytes + d] = s == 255u ? 0 : static_cast<uint8_t>(cvt_e4m3(__fmul_rn(v[i], f)));
        }
        if (stored && lane == 0) p.scales[head] = static_cast<uint8_t>(s);
      } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          if (32 * i >= a.D) break;
          float am = fabsf(v[i]);
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) am = mx::max_nan_abs(am, __shfl_xor_sync(0xffffffffu, am, o));
          const uint32_t s = mx::scale_code(am);
          const float q[8] = {__fmul_rn(v[i], mx::scale_inverse(s)), 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
          const uint32_t c = s == 255u ? 0u : cvt_e2m1x8(q) & 15u;
          const uint32_t next = __shfl_down_sync(0xffffffffu, c, 1);
          const int d = 32 * i + lane;
          if (stored && d < a.D && (lane & 1) == 0)
            p.codes[head * a.cache.code_bytes + (d >> 1)] = static_cast<uint8_t>(c | (next << 4));
          if (stored && lane == 0) p.scales[head * a.cache.scale_bytes + i] = static_cast<uint8_t>(s);
        }
      }
    }
  }
}

// ---------------------------------------------------------------- reading the cache
struct ReadArgs {
  const uint8_t* codes[2];
  const uint8_t* scales[2];
  void* out[2];
  long long ot[2], oh[2];  // row and head strides
  Cache cache;
  const int* table;        // [samples][width] pages
  const int* offsets;      // [samples + 1]
  long long ld_table;
  int width, samples, rows, chunks, per_head;  // chunks of W values per row and per head
  int block_rows;          // 1 to kReadRows
  unsigned magic, magic_row;  // ceil(2^32 / per_head), ceil(2^32 / chunks)
};
constexpr int kReadRows = 64;
// i / d by ceil(2^32 / d), exact while i d < 2^32
__device__ __forceinline__ int divided(int i, int d, unsigned magic) {
  return d == 1 ? i : static_cast<int>(__umulhi(static_cast<unsigned>(i), magic));
}

// Packed rows of the sequences: row i belongs to the sequence s with offsets[s] <= i < offsets[s + 1] and is its token
// i - offsets[s]. A block finds the slots of block_rows rows, then its threads take their chunks of W values of one
// plane (blockIdx.y), kReadAhead loads in flight each. W = 16: heads of whole groups of 16 values, outputs on 32 bytes,
// stored 32 bytes at a time; W = 8: on 16 bytes with VEC, else value by value. HBM bounds it: 16384 tokens of 24 heads of
// 128 on B200 49.6 us (6.1 TB/s of codes and values; 8 values a load 54.6 us), 6006 rows of 3 heads of 96 in MXFP4 4.4 us.
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
template <bool F32, int W, bool VEC>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const __grid_constant__ ReadArgs a) {
  constexpr int kReadAhead = 64 / W;
  __shared__ long long slots[kReadRows];
  grid_dependency_wait();
  grid_launch_dependents();
  const int row0 = blockIdx.x * a.block_rows, plane = blockIdx.y;
  if (threadIdx.x < a.block_rows) {
    const int row = row0 + threadIdx.x;
    long long slot = -2;  // not a row of any sequence
    const int last = __ldg(a.offsets + a.samples);
    if (row < a.rows && row < last && row >= __ldg(a.offsets)) {
      int lo = 0, hi = a.samples;  // offsets[lo] <= row < offsets[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.offsets + mid) <= row) lo = mid;
        else hi = mid;
      }
      const int at = row - __ldg(a.offsets + lo), col = at / a.cache.page_size;
      slot = -1;  // no page: zeros
      if (at >= 0 && col < a.width) {
        const long long page = __ldg(a.table + lo * a.ld_table + col);
        const long long s = page * a.cache.page_size + (at - col * a.cache.page_size);
        if (page >= 0 && s < a.cache.slots) slot = s;
      }
    }
    slots[threadIdx.x] = slot;
  }
  __syncthreads();
  const uint8_t* const codes = a.codes[plane];
  const uint8_t* const scales = a.scales[plane];
  const int items = a.block_rows * a.chunks;
  for (int i0 = threadIdx.x; i0 < items; i0 += kThreads * kReadAhead) {
    uint4 q[kReadAhead];
    uint32_t e[kReadAhead];
    long long to[kReadAhead];
#pragma unroll
    for (int u = 0; u < kReadAhead; ++u) {
      const int i = i0 + u * kThreads;
      q[u] = make_uint4(0u, 0u, 0u, 0u);
      e[u] = 0;
      to[u] = -1;
      if (i >= items) continue;
      const int r = a.block_rows == 1 ? 0 : divided(i, a.chunks, a.magic_row), c = i - r * a.chunks;
      const int h = divided(c, a.per_head, a.magic), k = c - h * a.per_head;
      const long long slot = slots[r];
      if (slot == -2) continue;
      to[u] = (row0 + r) * a.ot[plane] + h * a.oh[plane] + W * k;
      if (slot < 0) continue;
      const long long head = slot * a.cache.heads + h;
      const uint8_t* const from = codes + head * a.cache.code_bytes;
      if (a.cache.mx) {
        if constexpr (W == 16) {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(from) + k);
          q[u].x = w.x, q[u].y = w.y;
        } else {
          q[u].x = __ldg(reinterpret_cast<const uint32_t*>(from) + k);
        }
        e[u] = __ldg(scales + head * a.cache.scale_bytes + k / (32 / W));
      } else {
        if constexpr (W == 16) {
          q[u] = __ldg(reinterpret_cast<const uint4*>(from) + k);
        } else {
          const uint2 w = __ldg(reinterpret_cast<const uint2*>(from) + k);
          q[u].x = w.x, q[u].y = w.y;
        }
        e[u] = __ldg(scales + head);
      }
    }
#pragma unroll
    for (int u = 0; u < kReadAhead; ++u) {
      if (to[u] < 0) continue;
      const float s = mx::scale_value(e[u]);
      const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
      float v[W];
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        const float2 x = a.cache.mx ? mx::e2m1x2_value((w[j / 4] >> (8 * (j % 4))) & 0xFFu)
                                    : fp8b::e4m3x2_value((w[j / 2] >> (16 * (j % 2))) & 0xFFFFu);
        v[2 * j] = x.x * s;
        v[2 * j + 1] = x.y * s;
      }
      if constexpr (F32) {
        float* const o = static_cast<float*>(a.out[plane]) + to[u];
        if constexpr (W == 16) {
#pragma unroll
          for (int j = 0; j < 16; j += 8) store32(o + j, reinterpret_cast<const uint32_t(&)[8]>(v[j]));
        } else if constexpr (VEC) {
          *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
          *reinterpret_cast<float4*>(o + 4) = make_float4(v[4], v[5], v[6], v[7]);
        } else {
#pragma unroll
          for (int j = 0; j < W; ++j) o[j] = v[j];
        }
      } else {
        __nv_bfloat16* const o = static_cast<__nv_bfloat16*>(a.out[plane]) + to[u];
        if constexpr (VEC) {
          uint32_t b[W / 2];
#pragma unroll
          for (int j = 0; j < W / 2; ++j) b[j] = pack2(v[2 * j], v[2 * j + 1]);
          if constexpr (W == 16) store32(o, b);
          else *reinterpret_cast<uint4*>(o) = make_uint4(b[0], b[1], b[2], b[3]);
        } else {
#pragma unroll
          for (int j = 0; j < W; ++j) o[j] = __float2bfloat16_rn(v[j]);
        }
      }
    }
  }
}

}  // namespace heads
}  // namespace svdq
