// MXFP4 variant of the layer: E2M1 elements with one power-of-two scale (E8M0) per 32 elements along
// K, the microscaled 4-bit format of the OCP "Microscaling Formats (MX)" specification v1.0. Of a
// block of 32 fp32 values v:
//   e = max(floor(log2(max |v|)) - 2, -127)   (-127 for an all-zero block), scale code e + 127
//   q = E2M1_rne_sat(v 2^-e)
// floor(log2(a)) is the exponent field of a, so the scale is a shift and a subtraction and 2^-e an
// exact fp32 factor: no division, no table, no rounding before E2M1's. A subnormal maximum has field 0
// and takes the floor -127, whose factor 2^127 is exact too. A block with an infinity or a NaN
// (exponent field 255) gets scale code 255, E8M0's NaN, and zero codes: its products are NaN.
//
// The layer keeps its structure (smoothing, 16-bit low-rank branch, quantized residual), without a
// tensor scale: kernel 1 is svdq::quant_act_kernel with the Act policy below, the product is
// svdq::pair_gemm_kernel with the Gemm policy (kind::mxf4, one scale per 32: two scale atoms per
// 256-wide K step and 128 rows where NVFP4 takes four). Rows and columns of padding hold zero codes, so
// that sizes need not fill a tile.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "svdq_gemm.cuh"
#include "svdq_ptx.cuh"
#include "svdq_quant.cuh"

namespace svdq {
namespace mx {

constexpr int kBlock = 32;

// ---------------------------------------------------------------- block scales
// max of magnitudes that lets a NaN through
__device__ __forceinline__ float max_nan_abs(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}
__device__ __forceinline__ float max3_nan_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// E8M0 code of a block whose largest magnitude is `amax` (sign clear), and the factor 2^-e its elements
// take (an infinity for code 255, whose codes are then forced to zero)
__device__ __forceinline__ uint32_t scale_code(float amax) {
  const int f = static_cast<int>(__float_as_uint(amax) >> 23);
  return f == 255 ? 255u : static_cast<uint32_t>(max(f - 2, 0));
}
__device__ __forceinline__ float scale_inverse(uint32_t code) { return __uint_as_float((254u - code) << 23); }
// 2^(code - 127); code 255 is NaN, code 0 the subnormal 2^-127
__device__ __forceinline__ float scale_value(uint32_t code) {
  return code == 255u ? __uint_as_float(0x7FC00000u) : code == 0u ? __uint_as_float(0x00400000u)
                                                                  : __uint_as_float(code << 23);
}

// Byte offset of the scale of activation row m, 32-element block kb: atoms of 128 rows x 4 blocks
// (512 bytes), K-fastest. K is the padded K.
__host__ __device__ __forceinline__ size_t act_sf_offset(int m, int kb, int K) {
  return ((static_cast<size_t>(m >> 7) * (K >> 7) + (kb >> 2)) << 9) + ((m & 31) << 4) + (((m >> 5) & 3) << 2) +
         (kb & 3);
}
// Same for a packed weight row: per n_tile, per 128-wide K atom, n_tile / 128 atoms of 128 tile columns.
__host__ __device__ __forceinline__ size_t wgt_sf_offset(int p, int kb, int K, int n_tile) {
  const int atoms = n_tile >> 7;
  const int nb = p / n_tile, pl = tile_col_of_packed(p - nb * n_tile, n_tile);
  const int a = pl >> 7, pr = pl & 127;
  return (((static_cast<size_t>(nb) * (K >> 7) + (kb >> 2)) * atoms + a) << 9) + ((pr & 31) << 4) +
         ((pr >> 5) << 2) + (kb & 3);
}

// One thread's 8 consecutive values; four adjacent lanes hold one block (all 32 lanes call together).
// Returns the 8 packed codes and sets s to the block's scale code.
__device__ __forceinline__ uint32_t quarter_block(const float2 (&v)[4], uint32_t& s) {
  const float m0 = max3_nan_abs(v[0].x, v[0].y, v[1].x), m1 = max3_nan_abs(v[1].y, v[2].x, v[2].y);
  float a = max_nan_abs(max3_nan_abs(m0, m1, v[3].x), v[3].y);
  a = max_nan_abs(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = max_nan_abs(a, __shfl_xor_sync(0xffffffffu, a, 2));
  s = scale_code(a);
  const float f = scale_inverse(s);
  float q[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = mul2_rn(v[i], make_float2(f, f));
    q[2 * i] = p.x;
    q[2 * i + 1] = p.y;
  }
  const uint32_t codes = cvt_e2m1x8(q);
  return s == 255u ? 0u : codes;
}

// Two IEEE round-to-nearest fp32 sums in one instruction.
__device__ __forceinline__ float2 add2_rn(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(r)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&r);
}

// ---------------------------------------------------------------- kernel 1
struct ActArgs {
  const float* inv_lambda;  // [K] (padded K)
  uint8_t* codes;           // [M_pad][K/2]
  uint8_t* sf;
  __nv_bfloat16* U;         // [2][M_pad][r]: hi then lo
  unsigned long long wait_ns;
  int M, K, M_pad, k_per_cta;
};

// The quantizer policy of quant_act_kernel: a thread owns 16 columns of two rows of a stage, half a
// block each; the lane beside it (lane ^ 1) holds the other half, and the four lanes of a row the
// stage's two blocks, whose scales lane b = 0 stores together. Reading X bounds the kernel, as for
// NVFP4 (the same ring, TMA stages and branch MMAs); the scale costs one shift per block there.
// Measured on B200: 4608 rows of 12288, r = 0, 26.7 us (5.4 TB/s of X, codes and scales), 16896 rows of 3072, r = 32,
// 27 us (5.0 TB/s).
struct Act {
  using Args = ActArgs;
  __device__ static void prologue(const Args&, float*) {}
  struct Thread {
    int b;
    uint8_t* code_ptr[2];
    uint8_t* sf_ptr[2];
    __device__ Thread(const Args& a, const float*, int m_tile, int rl, int b_, int kbeg, int grp) : b(b_) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = m_tile * 128 + rl + 64 * i;
        code_ptr[i] = a.codes + static_cast<size_t>(row) * (a.K >> 1) + ((kbeg + (b << 4)) >> 1) + (grp << 5);
        // a group's next stage lies two K steps on: one whole scale atom
        sf_ptr[i] = a.sf + act_sf_offset(row, (kbeg >> 5) + 2 * grp, a.K);
      }
    }
    __device__ void stage(const float2 (&lam)[8], const uint4 (&x)[2][2]) {
      float2 v[2][8];
      float am[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t wx[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[i][j] = mul2_rn(make_float2(__uint_as_float(wx[j] << 16), __uint_as_float(wx[j] & 0xFFFF0000u)), lam[j]);
        const float m0 = max3_nan_abs(v[i][0].x, v[i][0].y, v[i][1].x), m1 = max3_nan_abs(v[i][1].y, v[i][2].x, v[i][2].y);
        const float m2 = max3_nan_abs(v[i][3].x, v[i][3].y, v[i][4].x), m3 = max3_nan_abs(v[i][4].y, v[i][5].x, v[i][5].y);
        const float m4 = max3_nan_abs(v[i][6].x, v[i][6].y, v[i][7].x);
        am[i] = max_nan_abs(max3_nan_abs(m0, m1, m2), max3_nan_abs(m3, m4, v[i][7].y));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) am[i] = max_nan_abs(am[i], __shfl_xor_sync(0xffffffffu, am[i], 1));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t s = scale_code(am[i]);
        const float f = scale_inverse(s);
        const float2 f2 = make_float2(f, f);
        float q[16];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 p = mul2_rn(v[i][j], f2);
          q[2 * j] = p.x;
          q[2 * j + 1] = p.y;
        }
        uint2 codes;
        codes.x = cvt_e2m1x8(*reinterpret_cast<const float(*)[8]>(q));
        codes.y = cvt_e2m1x8(*reinterpret_cast<const float(*)[8]>(q + 8));
        if (s == 255u) codes = make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(code_ptr[i]) = codes;
        const uint32_t s2 = __shfl_down_sync(0xffffffffu, s, 2);
        if (b == 0) *reinterpret_cast<uint16_t*>(sf_ptr[i]) = static_cast<uint16_t>(s | (s2 << 8));
        code_ptr[i] += 64;
        sf_ptr[i] += 512;
      }
    }
  };
  __device__ static float u_scale(const Args&, int) { return 1.0f; }
  __device__ static void finish(const Args&) {}
};

// ---------------------------------------------------------------- kernel 2
// D[tmem] (+)= A[smem] x B[smem]^T, E2M1 x E2M1 with one UE8M0 scale per 32 K-elements of A and B,
// M = 256 across the CTA pair, K = 64 per instruction (warp-wide call; elect.sync picks the lane).
__device__ __forceinline__ void mma_mxf4_pair_warp(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                   uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb));
}
// Instruction descriptor, kind::mxf4: A, B = E2M1, K-major, UE8M0 scales. An MMA of K = 64 takes two of
// the four scale bytes of a TMEM column: data id 0 (bytes 0, 1) or 2 (bytes 2, 3), the same for A and B.
__host__ __device__ constexpr uint32_t idesc_mxf4(int m, int n, uint32_t sf_id) {
  return idesc_nvfp4(m, n) | (1u << 23) | (sf_id << 4) | (sf_id << 29);
}

struct GemmArgs {
  const uint8_t* sfa;
  const uint8_t* sfb;
  const __nv_bfloat16* bias;
  unsigned long long wait_ns;
  int M, M_pad, N, K, r;  // N: the weight's true width (the bias length), K: padded
  int m_tiles, m_pairs, n_tiles, k_iters, num_tiles;
  int out_f32, epi;       // epi bit 0: bias, bit 1: SwiGLU
  int n_tile;             // the packed tile width; the kernel's own is this or 128
};

// The MXFP4 format of the pair GEMM. A K step's two scale atoms each serve two MMAs (data ids 0 and 2).
// Operands between L2 and the SMs bound it, as for NVFP4, with half the scale bytes: 16896 x 3072 x 9216, r = 32,
// 194-203 us on B200 (4.8-5.0 PFLOP/s), 4608 x 3072 x 24576 with SwiGLU and bias 160-166 us.
struct Gemm {
  using Args = GemmArgs;
  static constexpr bool kScales = true;
  static constexpr int kSfAtomsK = 2;
  static constexpr bool kL2HiLo = false;
  static constexpr bool kBiasSmem = true;
  // The 128-wide kernel also takes a weight packed 256 or 384 wide: a block of 128 tile columns is two runs
  // of 64 packed rows, one for each CTA of the pair, and one scale atom per 128 of K.
  template <int N_TILE>
  __device__ static int b_row(const Args& a, int n_blk, int rank) {
    if constexpr (N_TILE == 128) {
      const int per = a.n_tile >> 7, tile = n_blk / per;
      return tile * a.n_tile + packed_of_tile_col((n_blk - tile * per) * 128 + 64 * rank, a.n_tile);
    } else {
      return n_blk * N_TILE + rank * (N_TILE / 2);
    }
  }
  template <int N_TILE, int BYTES>
  __device__ static void load_sfb(const Args& a, int n_blk, int sf_row_stride, int kt, uint32_t dst, uint32_t bar) {
    if constexpr (N_TILE == 128) {
      const int per = a.n_tile >> 7, tile = n_blk / per, at = n_blk - tile * per;
#pragma unroll
      for (int i = 0; i < kSfAtomsK; ++i)
        bulk_load(dst + 512 * i,
                  a.sfb + (((static_cast<size_t>(tile) * sf_row_stride + kt * kSfAtomsK + i) * per + at) << 9), 512, bar);
    } else {
      bulk_load(dst,
                a.sfb + ((static_cast<size_t>(n_blk) * sf_row_stride + static_cast<size_t>(kt) * kSfAtomsK) *
                             (N_TILE / 128) << 9),
                BYTES, bar);
    }
  }
  template <int N_TILE, int SF_ATOMS_B>
  __device__ static void kstep(uint32_t d, uint32_t la, uint32_t lb, uint32_t hi_ab, uint32_t tsf,
                               uint32_t accumulate) {
    constexpr int kN1 = N_TILE <= 256 ? N_TILE : 256;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t sf_id = j & 1 ? 2u : 0u;
      const uint32_t ta = tsf + 4 * (j >> 1), tb = tsf + 8 + 4 * SF_ATOMS_B * (j >> 1);
      const uint64_t a = desc_join(la + 2u * j, hi_ab);
      const uint32_t acc = j == 0 ? accumulate : 1u;
      mma_mxf4_pair_warp(d, a, desc_join(lb + 2u * j, hi_ab), idesc_mxf4(256, kN1, sf_id), ta, tb, acc);
      if constexpr (N_TILE > 256) {
        // columns 256..383: the last 64 rows of each CTA's B box (16 KB on), the third SFB atom
        constexpr uint32_t kB2 = (128 * 128) >> 4;
        mma_mxf4_pair_warp(d + 256, a, desc_join(lb + kB2 + 2u * j, hi_ab), idesc_mxf4(256, N_TILE - 256, sf_id), ta,
                           tb + 8, acc);
      }
    }
  }
  // y = acc (+ bias)
  struct Epi {
    __device__ Epi(const Args&, int) {}
    template <bool BIAS, class V>
    __device__ void apply8(const Args&, V& v, int off, int, const float* bias8) const {
      if constexpr (BIAS) {
        const float4 b0 = reinterpret_cast<const float4*>(bias8)[0], b1 = reinterpret_cast<const float4*>(bias8)[1];
        const float2 b[4] = {make_float2(b0.x, b0.y), make_float2(b0.z, b0.w), make_float2(b1.x, b1.y),
                             make_float2(b1.z, b1.w)};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 y = add2_rn(make_float2(v[off + 2 * j], v[off + 2 * j + 1]), b[j]);
          v[off + 2 * j] = y.x;
          v[off + 2 * j + 1] = y.y;
        }
      }
    }
  };
};

// ---------------------------------------------------------------- offline pack, export, values
// R [N][K] fp32 -> codes and scales of the packed rows. One thread per 8 values of a padded row
// (K_pad / 8 is a multiple of 32, so a warp stays in one row); values past K count as zero. Padded rows
// keep the zeros the blob was cleared to.
__global__ void pack_quant_kernel(const float* __restrict__ R, int N, int K, int K_pad, int n_tile, int swiglu,
                                  uint8_t* __restrict__ codes, uint8_t* __restrict__ sf) {
  const int per_row = K_pad >> 3;
  const size_t total = static_cast<size_t>(N) * per_row;
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<size_t>(gridDim.x) * blockDim.x) {
    const int n = static_cast<int>(i / per_row);
    const int k = static_cast<int>(i - static_cast<size_t>(n) * per_row) * 8;
    float2 v[4] = {};
    if (k < K) {
      const float4* src = reinterpret_cast<const float4*>(R + static_cast<size_t>(n) * K + k);
      const float4 a0 = __ldg(src), a1 = __ldg(src + 1);
      v[0] = make_float2(a0.x, a0.y);
      v[1] = make_float2(a0.z, a0.w);
      v[2] = make_float2(a1.x, a1.y);
      v[3] = make_float2(a1.z, a1.w);
    }
    uint32_t s;
    const uint32_t q = quarter_block(v, s);
    const int p = gemm_row_of(n, N, n_tile, swiglu);
    *reinterpret_cast<uint32_t*>(codes + static_cast<size_t>(p) * (K_pad >> 1) + (k >> 1)) = q;
    if ((k & 31) == 0) sf[wgt_sf_offset(p, k >> 5, K_pad, n_tile)] = static_cast<uint8_t>(s);
  }
}

__global__ void fill_inv_lambda_kernel(const float* __restrict__ src, int K, int K_pad, float* __restrict__ dst) {
  for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < K_pad; i += gridDim.x * blockDim.x)
    dst[i] = src != nullptr && i < K ? src[i] : 1.0f;
}

// L1s [K][r] -> L1s_t [r][K_pad], zero past K
__global__ void transpose_l1_kernel(const __nv_bfloat16* __restrict__ L1s, int K, int K_pad, int r,
                                    __nv_bfloat16* __restrict__ out) {
  const size_t total = static_cast<size_t>(K_pad) * r;
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<size_t>(gridDim.x) * blockDim.x) {
    const int j = static_cast<int>(i / K_pad), k = static_cast<int>(i - static_cast<size_t>(j) * K_pad);
    out[i] = k < K ? L1s[static_cast<size_t>(k) * r + j] : __float2bfloat16_rn(0.0f);
  }
}

// L2 [r][N] -> L2_t [N_pad][r], rows in GEMM order (padded rows keep the blob's zeros)
__global__ void pack_l2_kernel(const __nv_bfloat16* __restrict__ L2, int N, int r, int n_tile, int swiglu,
                               __nv_bfloat16* __restrict__ out) {
  const size_t total = static_cast<size_t>(N) * r;
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<size_t>(gridDim.x) * blockDim.x) {
    const int n = static_cast<int>(i / r), j = static_cast<int>(i - static_cast<size_t>(n) * r);
    out[static_cast<size_t>(gemm_row_of(n, N, n_tile, swiglu)) * r + j] = L2[static_cast<size_t>(j) * N + n];
  }
}

// Canonical export, one thread per 8 values: 4 bytes of codes, and the block's scale from its first.
// n_tile 0: an activation.
__global__ void export_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ sf, int rows, int K,
                              int K_pad, int n_tile, int swiglu, uint8_t* __restrict__ out_codes,
                              uint8_t* __restrict__ out_sf) {
  const int per_row = K >> 3, blocks = (K + 31) >> 5;
  const size_t total = static_cast<size_t>(rows) * per_row;
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<size_t>(gridDim.x) * blockDim.x) {
    const int n = static_cast<int>(i / per_row), c = static_cast<int>(i - static_cast<size_t>(n) * per_row);
    const int p = n_tile ? gemm_row_of(n, rows, n_tile, swiglu) : n;
    *reinterpret_cast<uint32_t*>(out_codes + static_cast<size_t>(n) * (K >> 1) + 4 * c) =
        *reinterpret_cast<const uint32_t*>(codes + static_cast<size_t>(p) * (K_pad >> 1) + 4 * c);
    if ((c & 3) == 0)
      out_sf[static_cast<size_t>(n) * blocks + (c >> 2)] =
          sf[n_tile ? wgt_sf_offset(p, c >> 2, K_pad, n_tile) : act_sf_offset(p, c >> 2, K_pad)];
  }
}

// Two E2M1 codes (a byte, low nibble first) -> their values.
__device__ __forceinline__ float2 e2m1x2_value(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 b;\n\tcvt.u8.u32 b, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(h) : "r"(byte));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The values of a quantized activation: dec(q) 2^e, exact in fp32. A thread takes 8 columns of kDeqRows
// rows, whose loads go out together; writing the values bounds it (4608 rows of 12288 to bf16 in 25.2 us, 5.7 TB/s;
// one row per thread 33 us).
constexpr int kDeqRows = 4;
template <bool F32>
__global__ void __launch_bounds__(256) dequantize_act_kernel(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ sf, int M, int K, int K_pad,
                                                             void* __restrict__ out, long long ld) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int m0 = blockIdx.x * kDeqRows, c = blockIdx.y * 256 + threadIdx.x;
  if (8 * c >= K) return;
  uint32_t q[kDeqRows], e[kDeqRows];
#pragma unroll
  for (int r = 0; r < kDeqRows; ++r) {
    const int m = m0 + r;  // a row of padding (allocated up to M_pad) may be read
    q[r] = __ldg(reinterpret_cast<const uint32_t*>(codes + static_cast<size_t>(m) * (K_pad >> 1) + 4 * c));
    e[r] = __ldg(sf + act_sf_offset(m, c >> 2, K_pad));
  }
#pragma unroll
  for (int r = 0; r < kDeqRows; ++r) {
    const long long m = m0 + r;
    if (m >= M) break;
    const float s = scale_value(e[r]);
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = mul2_rn(e2m1x2_value((q[r] >> (8 * j)) & 0xFFu), make_float2(s, s));
    if constexpr (F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + m * ld + 8 * c);
      o[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
      o[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[j].x, v[j].y);
        w[j] = *reinterpret_cast<const uint32_t*>(&b2);
      }
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + m * ld + 8 * c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

}  // namespace mx
}  // namespace svdq
