// Block-scaled FP8 variant of the layer: E4M3 elements with one power-of-two scale (E8M0) per block of 128:
// of an activation row 128 elements along K, of the weight 128 x 128. Of a block of fp32 values v:
//   e = the smallest integer >= -127 with max |v| <= 448 2^e   (-127 for an all-zero block), scale code e + 127
//   q = E4M3_rne(v 2^-e)
// 448 = 1.75 x 2^8 is E4M3's largest value, so e + 127 is the exponent field of max |v|, one more where its
// mantissa exceeds 1.75, minus 8: an addition and a shift, and 2^-e an exact fp32 factor (no division, no
// rounding before E4M3's). Nothing saturates. A block with an infinity or a NaN gets scale code 255,
// E8M0's NaN, and zero codes: what reads it is NaN.
//
// Why powers of two: the tensor cores take an E8M0 scale per 32 elements of K and row beside the operands
// (kind::mxf8f6f4), at the rate of the product without scales. fp32 scales would have to be applied to each
// 128-wide partial sum outside the tensor cores, an fp32 multiply-add per output and 128 of K; against them a
// power of two costs nothing in precision, E4M3's steps being relative (its smallest normal magnitude, relative to the
// block's largest, moves by up to a factor of 2).
//
// The layer keeps its structure (smoothing, 16-bit low-rank branch, quantized residual): kernel 1 is
// svdq::quant_act_kernel with the Act policy below, the product svdq::pair_gemm_kernel with the Gemm policy.
// Columns past K and the weight's rows past N hold zero codes, so that sizes need not fill a tile. Activation rows past M
// are not written: what they hold reaches only their own outputs, which are not stored.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "svdq_fp8r.cuh"
#include "svdq_gemm.cuh"
#include "svdq_mx.cuh"
#include "svdq_mx_few.cuh"
#include "svdq_ptx.cuh"
#include "svdq_quant.cuh"

namespace svdq {
namespace fp8b {

constexpr int kBlock = 128;

// ---------------------------------------------------------------- block scales
// E8M0 code of a block whose largest magnitude is `amax` (sign clear). mx::scale_inverse and mx::scale_value give
// 2^-e and 2^e.
__device__ __forceinline__ uint32_t scale_code(float amax) {
  const uint32_t u = __float_as_uint(amax);
  return u >= 0x7F800000u ? 255u : static_cast<uint32_t>(max(static_cast<int>((u + 0x1FFFFFu) >> 23) - 8, 0));
}
// 8 values -> 8 codes; f: 2^-e of their block
__device__ __forceinline__ uint2 encode8(const float2 (&v)[4], float f) {
  const float2 f2 = make_float2(f, f);
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = mul2_rn(v[i], f2);
    h[i] = fp8r::cvt_e4m3x2(p.x, p.y);
  }
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}
// Two E4M3 codes (low byte first) -> their values, exact.
__device__ __forceinline__ float2 e4m3x2_value(uint32_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(pair)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float amax8(const float2 (&v)[4]) {
  const float m0 = mx::max3_nan_abs(v[0].x, v[0].y, v[1].x), m1 = mx::max3_nan_abs(v[1].y, v[2].x, v[2].y);
  return mx::max_nan_abs(mx::max3_nan_abs(m0, m1, v[3].x), v[3].y);
}

// Scale atoms: 128 rows x 4 blocks of K (512 bytes). Byte offset of the scale of activation row m, block kb of
// K_pad / 128, and of a packed weight row (per n_tile, per 4 blocks, n_tile / 128 atoms of 128 tile columns).
__host__ __device__ __forceinline__ int sf_atoms(int K_pad) { return (K_pad + 511) >> 9; }
__host__ __device__ __forceinline__ size_t act_sf_offset(int m, int kb, int K_pad) {
  return ((static_cast<size_t>(m >> 7) * sf_atoms(K_pad) + (kb >> 2)) << 9) + ((m & 31) << 4) + (((m >> 5) & 3) << 2) +
         (kb & 3);
}
__host__ __device__ __forceinline__ size_t wgt_sf_offset(int p, int kb, int K_pad, int n_tile) {
  const int atoms = n_tile >> 7, nb = p / n_tile, pl = tile_col_of_packed(p - nb * n_tile, n_tile), a = pl >> 7, pr = pl & 127;
  return (((static_cast<size_t>(nb) * sf_atoms(K_pad) + (kb >> 2)) * atoms + a) << 9) + ((pr & 31) << 4) +
         ((pr >> 5) << 2) + (kb & 3);
}

// ---------------------------------------------------------------- kernel 1
struct ActArgs {
  const float* inv_lambda;  // [K_pad]
  uint8_t* codes;           // [M_pad][K_pad]
  uint8_t* sf;
  __nv_bfloat16* U;         // [2][M_pad][r]: hi then lo
  unsigned long long wait_ns;
  int M, K, M_pad, k_per_cta;  // K padded
};

// The quantizer policy of quant_act_kernel: a block spans two 64-wide stages, so a group of quantizer warps takes
// two at a time; a thread owns 16 columns of both stages in two rows, the four lanes of a row its block. Latency
// bounds it: on B200 4608 rows of 3072, r = 32, 13.9 us (3.1 TB/s of X, codes and scales, 0.47 of the copy rate), where clusters
// of three put 108 of 148 SMs to work, each goes through 16 stages once and no unit is half full (issue 35 %, ALU 33 %);
// 512 rows 11.5 us, of K = 1608, r = 16, 8.4 us with K in shares of 4, 4, 4 and 1 blocks (15.4 us unsplit).
struct Act {
  using Args = ActArgs;
  static constexpr int kRun = 2;
  __device__ static void prologue(const Args&, float*) {}
  struct Thread {
    int b;
    uint8_t* code_ptr[2];
    uint8_t* sf_row[2];
    int kb;
    float2 v[2][2][8];  // stage, row
    float am[2];
    __device__ Thread(const Args& a, const float*, int m_tile, int rl, int b_, int kbeg, int grp) : b(b_) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = m_tile * 128 + rl + 64 * i;
        code_ptr[i] = a.codes + static_cast<size_t>(row) * a.K + kbeg + (b << 4) + (grp << 7);
        sf_row[i] = a.sf + act_sf_offset(row, 0, a.K);
      }
      kb = (kbeg >> 7) + grp;
    }
    __device__ void take(int p, const float2 (&lam)[8], const uint4 (&x)[2][2]) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t wx[8] = {x[i][0].x, x[i][0].y, x[i][0].z, x[i][0].w, x[i][1].x, x[i][1].y, x[i][1].z, x[i][1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[p][i][j] = mul2_rn(make_float2(__uint_as_float(wx[j] << 16), __uint_as_float(wx[j] & 0xFFFF0000u)), lam[j]);
        const float m = mx::max_nan_abs(amax8(reinterpret_cast<const float2(&)[4]>(v[p][i][0])),
                                        amax8(reinterpret_cast<const float2(&)[4]>(v[p][i][4])));
        am[i] = p == 0 ? m : mx::max_nan_abs(am[i], m);
      }
    }
    __device__ void finish_run() {
#pragma unroll
      for (int i = 0; i < 2; ++i) am[i] = mx::max_nan_abs(am[i], __shfl_xor_sync(0xffffffffu, am[i], 1));
#pragma unroll
      for (int i = 0; i < 2; ++i) am[i] = mx::max_nan_abs(am[i], __shfl_xor_sync(0xffffffffu, am[i], 2));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t s = scale_code(am[i]);
        const float f = mx::scale_inverse(s);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint2 lo = encode8(reinterpret_cast<const float2(&)[4]>(v[p][i][0]), f);
          const uint2 hi = encode8(reinterpret_cast<const float2(&)[4]>(v[p][i][4]), f);
          *reinterpret_cast<uint4*>(code_ptr[i] + 64 * p) =
              s == 255u ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(lo.x, lo.y, hi.x, hi.y);
        }
        if (b == 0) sf_row[i][((kb >> 2) << 9) + (kb & 3)] = static_cast<uint8_t>(s);
        code_ptr[i] += 256;
      }
      kb += 2;
    }
  };
  __device__ static float u_scale(const Args&, int) { return 1.0f; }
  __device__ static void finish(const Args&) {}
};

// 32 bytes that are read once
__device__ __forceinline__ void ldg_stream32(const void* p, uint4& lo, uint4& hi) {
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(lo.x), "=r"(lo.y), "=r"(lo.z), "=r"(lo.w), "=r"(hi.x), "=r"(hi.y), "=r"(hi.z), "=r"(hi.w)
               : "l"(p));
}

// Without a branch nothing projects X, so that rows can be quantized straight from registers: 16 columns per
// lane, 8 lanes a block, ROWS rows per thread, whose loads go out together and share the smoothing factors. WIDE: rows
// lie on 32 bytes. HBM bounds it: on B200 16896 rows of 3072 28.3 us, 4608 of 12288 29.6 us (5.7 TB/s; with 16-byte loads
// and 8-byte stores 32.2 and 33.3 us), one row 1.6 us.
template <int ROWS, bool WIDE>
__global__ void __launch_bounds__(256) quant_rows_kernel(const __nv_bfloat16* __restrict__ X, long long ldx,
                                                         const float* __restrict__ inv_lambda, int M, int K, int K_pad,
                                                         uint8_t* __restrict__ codes, uint8_t* __restrict__ sf) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int per_row = K_pad >> 4;  // a multiple of 8: the lanes of a block stay together
  const long long at = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  const long long g = at / per_row;
  const int k = static_cast<int>(at - g * per_row) * 16;
  const long long m0 = g * ROWS;
  uint4 x[ROWS][2];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    x[r][0] = x[r][1] = make_uint4(0u, 0u, 0u, 0u);
    if (m0 + r < M) {
      const __nv_bfloat16* p = X + (m0 + r) * ldx + k;
      if (WIDE && k + 8 < K) {
        ldg_stream32(p, x[r][0], x[r][1]);
      } else {  // K may end in the middle
        if (k < K) x[r][0] = ldg_stream(p);
        if (k + 8 < K) x[r][1] = ldg_stream(p + 8);
      }
    }
  }
  float2 lam[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 l = m0 < M ? __ldg(reinterpret_cast<const float4*>(inv_lambda + k) + i) : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    lam[2 * i] = make_float2(l.x, l.y);
    lam[2 * i + 1] = make_float2(l.z, l.w);
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    float2 v[2][4];
    float a = 0.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float e[8];
      bf16x8_to_f32(x[r][h], e);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[h][i] = mul2_rn(make_float2(e[2 * i], e[2 * i + 1]), lam[4 * h + i]);
      a = mx::max_nan_abs(a, amax8(v[h]));
    }
#pragma unroll
    for (int o = 1; o < 8; o *= 2) a = mx::max_nan_abs(a, __shfl_xor_sync(0xffffffffu, a, o));
    const uint32_t s = scale_code(a);
    const float f = mx::scale_inverse(s);
    const uint2 lo = encode8(v[0], f), hi = encode8(v[1], f);
    if (m0 + r < M) {
      *reinterpret_cast<uint4*>(codes + static_cast<size_t>(m0 + r) * K_pad + k) =
          s == 255u ? make_uint4(0u, 0u, 0u, 0u) : make_uint4(lo.x, lo.y, hi.x, hi.y);
      if ((k & 127) == 0) sf[act_sf_offset(static_cast<int>(m0) + r, k >> 7, K_pad)] = static_cast<uint8_t>(s);
    }
  }
}

// ---------------------------------------------------------------- kernel 2
// D[tmem] (+)= A[smem] x B[smem]^T, E4M3 x E4M3 with one UE8M0 scale per row and 32 K-elements of A and B,
// M = 256 across the CTA pair, K = 32 per instruction (warp-wide call; elect.sync picks the lane).
__device__ __forceinline__ void mma_mxf8_pair_warp(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                   uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb));
}
// Instruction descriptor, kind::mxf8f6f4: A, B = E4M3 (format 0), K-major, UE8M0 scales. An MMA takes one of the
// four scale bytes of a TMEM column, `sf_id`, the same for A and B.
__host__ __device__ constexpr uint32_t idesc_mxf8(int m, int n, uint32_t sf_id) {
  return (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(m >> 4) << 24) | (sf_id << 4) |
         (sf_id << 29);
}

__device__ __forceinline__ void mma_mxf8(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb));
}

// This format in the few-row kernels (one token of 3072 -> 9216 on B200, weight from HBM: quantizer 1.6 us, product 9.9 us,
// 2.9 TB/s; by the pair GEMM 12.7 us): a step is one block of 128, its scale byte k % 4 of the atom that four steps share
// (loaded with each of them: 512 bytes beside 16 KB of weight)
struct Few {
  static constexpr int kStepK = 128, kAtoms = 1;
  using Codes = uint2;
  __device__ static Codes encode(const float2 (&v)[4], uint32_t& s) {
    float a = amax8(v);
#pragma unroll
    for (int o = 1; o < 16; o *= 2) a = mx::max_nan_abs(a, __shfl_xor_sync(0xffffffffu, a, o));
    s = scale_code(a);
    const uint2 q = encode8(v, mx::scale_inverse(s));
    return s == 255u ? make_uint2(0u, 0u) : q;
  }
  __device__ static void store(const mx::FewQuantArgs& a, int m, int k, Codes q, uint32_t s) {
    *reinterpret_cast<uint2*>(a.codes + static_cast<size_t>(m) * a.K_pad + k) = q;
    if ((k & 127) == 0) a.sf[act_sf_offset(m, k >> 7, a.K_pad)] = static_cast<uint8_t>(s);
  }
  __host__ __device__ static int sf_atoms(int K_pad) { return fp8b::sf_atoms(K_pad); }
  __device__ static int sf_atom(int k, int) { return k >> 2; }
  __device__ static void mma(uint32_t d, uint64_t w, uint64_t x, int cols, int k, int, uint32_t sfw, uint32_t sfx,
                             uint32_t accumulate) {
    mma_mxf8(d, w, x, idesc_mxf8(128, cols, static_cast<uint32_t>(k) & 3u), sfw, sfx, accumulate);
  }
};

struct GemmArgs {
  const uint8_t* sfa;
  const uint8_t* sfb;
  const __nv_bfloat16* bias;
  unsigned long long wait_ns;
  int M, M_pad, N, K, r;  // N: the weight's true width (the bias length), K: padded
  int m_tiles, m_pairs, n_tiles, k_iters, num_tiles;
  int out_f32, epi;       // epi bit 0: bias, bit 1: SwiGLU
  int n_tile;             // the packed tile width; the kernel's own is this or less
};

// The block-scaled FP8 format of the pair GEMM. A K step is one block of 128: its four MMAs (K = 32) take the same
// scale byte, byte kt % 4 of the atom that four K steps share. The writers then hand a scale buffer over once per four
// steps; with an atom in every ring slot and a hand-over per step (512 tensor-pipe cycles), 4608 x 3072 x 9216 took 117 us on
// B200 instead of 97. An SM took in 44 to 51 bytes a cycle at every size and tile measured, with 18 SMs at work as with
// all. Hence tiles 384 wide (53 bytes of codes per tensor-pipe cycle, 64 at 256 wide, 96 at 128), issued as N = 256 and N = 128 on the
// same A; 256 wide the next took 354 us. Between tiles its one accumulator waits: 256 columns twice leave TMEM no room
// for scales. 16896 x 3072 x 9216 340 us, 4608 x 3072 x 24576 with SwiGLU (256 wide), bias and r = 32 277 us (2.8 and 2.5
// PFLOP/s). Scales read by their writers from global memory instead of bulk copies: 349 us (and 5 % less at few rows).
struct Gemm {
  using Args = GemmArgs;
  static constexpr bool kScales = true;
  static constexpr int kSfAtomsK = 1;
  static constexpr int kSfShare = 4;
  static constexpr bool kL2HiLo = false;
  static constexpr bool kBiasSmem = true;
  __device__ static int sf_atoms(const Args& a) { return fp8b::sf_atoms(a.K); }
  __device__ static int sf_atom(int kt) { return kt >> 2; }
  // The 128-wide kernel takes weights packed 256 or 384 wide too: a block of 128 tile columns is two runs of 64 packed
  // rows, one for each CTA of the pair, and an atom of its own.
  template <int N_TILE>
  static constexpr int kBBoxes = 1;
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
    const int per = a.n_tile / N_TILE, tile = n_blk / per, at = n_blk - tile * per;
    bulk_load(dst,
              a.sfb + (((static_cast<size_t>(tile) * sf_row_stride + (kt >> 2)) * (a.n_tile >> 7) + at) << 9), BYTES, bar);
  }
  template <int N_TILE, int SF_ATOMS_B>
  __device__ static void kstep(uint32_t d, uint32_t la, uint32_t lb, uint32_t hi_ab, uint32_t tsf,
                               uint32_t accumulate, int kt) {
    constexpr int kN1 = N_TILE <= 256 ? N_TILE : 256;
    const uint32_t sf_id = static_cast<uint32_t>(kt) & 3u, sf_bits = (sf_id << 4) | (sf_id << 29);
    const uint32_t id = idesc_mxf8(256, kN1, 0) | sf_bits;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t a = desc_join(la + 2u * j, hi_ab);
      const uint32_t acc = j == 0 ? accumulate : 1u;
      mma_mxf8_pair_warp(d, a, desc_join(lb + 2u * j, hi_ab), id, tsf, tsf + 4, acc);
      if constexpr (N_TILE > 256) {
        // columns 256..383: the last 64 rows of each CTA's B box (16 KB on), the third SFB atom
        constexpr uint32_t kB2 = (128 * 128) >> 4;
        mma_mxf8_pair_warp(d + 256, a, desc_join(lb + kB2 + 2u * j, hi_ab), idesc_mxf8(256, N_TILE - 256, 0) | sf_bits, tsf,
                           tsf + 12, acc);
      }
    }
  }
  struct Epi : mx::Gemm::Epi {  // y = acc (+ bias)
    __device__ Epi(const Args&, int) : mx::Gemm::Epi(mx::GemmArgs{}, 0) {}
    template <bool BIAS, class V>
    __device__ void apply8(const Args&, V& v, int off, int g0, const float* bias8) const {
      mx::Gemm::Epi::apply8<BIAS>(mx::GemmArgs{}, v, off, g0, bias8);
    }
  };
};

// 256-wide tiles of a weight packed 384 wide: a CTA's B rows are two runs of 64 packed rows, and the tile's two atoms may
// lie in two packed tiles. 1024 x 3072 -> 9216 25.3 us, as if it were packed 256 wide; 384-wide tiles take 31.2. (With the
// packed width as a variable of one kernel, its divisions in the copying thread cost 27.1.)
struct Gemm256Of384 : Gemm {
  template <int N_TILE>
  static constexpr int kBBoxes = 2;
  template <int N_TILE>
  __device__ static int b_row(const Args&, int n_blk, int at) {
    static_assert(N_TILE == 256);
    const int col = n_blk * 256 + 64 * at, tile = col / 384;
    return tile * 384 + packed_of_tile_col(col - tile * 384, 384);
  }
  template <int N_TILE, int BYTES>
  __device__ static void load_sfb(const Args& a, int n_blk, int sf_row_stride, int kt, uint32_t dst, uint32_t bar) {
    auto atom = [&](int block) {  // of 128 columns
      const int tile = block / 3, at = block - tile * 3;
      return a.sfb + (((static_cast<size_t>(tile) * sf_row_stride + (kt >> 2)) * 3 + at) << 9);
    };
    const int block = 2 * n_blk;
    if (block % 3 == 2) {  // the second atom is the next packed tile's first, if there is one
      bulk_load(dst, atom(block), 512, bar);
      bulk_load(dst + 512, atom(min(block + 1, (a.N - 1) >> 7)), 512, bar);
    } else {
      bulk_load(dst, atom(block), BYTES, bar);
    }
  }
};

// ---------------------------------------------------------------- offline pack, export, values
// R [N][K] fp32 -> codes and scales of the packed rows. A CTA of 256 threads per block of 128 rows x 128 columns of
// R: eight rows of 32 lanes at a time, four columns per lane. Values past N and K count as zero; padded rows keep the
// zeros the blob was cleared to.
template <class = void>
__global__ void __launch_bounds__(256) pack_quant_kernel(const float* __restrict__ R, int N, int K, int K_pad,
                                                         int n_tile, int swiglu, uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ sf) {
  __shared__ float part[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int kbs = K_pad / kBlock, kb = static_cast<int>(blockIdx.x % kbs), n0 = static_cast<int>(blockIdx.x / kbs) * kBlock;
  const int k = kb * kBlock + 4 * lane;
  float4 v[16];
  float am = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int n = n0 + 8 * i + warp;
    v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (n < N && k < K) v[i] = __ldg(reinterpret_cast<const float4*>(R + static_cast<size_t>(n) * K + k));
    am = mx::max3_nan_abs(am, v[i].x, v[i].y);
    am = mx::max3_nan_abs(am, v[i].z, v[i].w);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) am = mx::max_nan_abs(am, __shfl_xor_sync(0xffffffffu, am, o));
  if (lane == 0) part[warp] = am;
  __syncthreads();
  am = part[0];
#pragma unroll
  for (int w = 1; w < 8; ++w) am = mx::max_nan_abs(am, part[w]);
  const uint32_t s = scale_code(am);
  const float f = mx::scale_inverse(s);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int n = n0 + 8 * i + warp;
    if (n >= N) continue;
    const int p = gemm_row_of(n, N, n_tile, swiglu);
    const uint32_t q = fp8r::cvt_e4m3x2(__fmul_rn(v[i].x, f), __fmul_rn(v[i].y, f)) |
                       (fp8r::cvt_e4m3x2(__fmul_rn(v[i].z, f), __fmul_rn(v[i].w, f)) << 16);
    *reinterpret_cast<uint32_t*>(codes + static_cast<size_t>(p) * K_pad + k) = s == 255u ? 0u : q;
    if (lane == 0) sf[wgt_sf_offset(p, kb, K_pad, n_tile)] = static_cast<uint8_t>(s);
  }
}

// Canonical export, one thread per 8 codes: codes [rows][K], and the scale of a block from its first thread (of its
// first row, for a weight). n_tile 0: an activation.
template <class = void>
__global__ void export_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ sf, int rows, int K,
                              int K_pad, int n_tile, int swiglu, uint8_t* __restrict__ out_codes,
                              uint8_t* __restrict__ out_sf) {
  const int per_row = K >> 3, blocks = (K + kBlock - 1) / kBlock;
  const size_t total = static_cast<size_t>(rows) * per_row;
  for (size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<size_t>(gridDim.x) * blockDim.x) {
    const int n = static_cast<int>(i / per_row), c = static_cast<int>(i - static_cast<size_t>(n) * per_row);
    const int p = n_tile ? gemm_row_of(n, rows, n_tile, swiglu) : n;
    *reinterpret_cast<uint2*>(out_codes + static_cast<size_t>(n) * K + 8 * c) =
        *reinterpret_cast<const uint2*>(codes + static_cast<size_t>(p) * K_pad + 8 * c);
    if ((c & 15) == 0 && (n_tile == 0 || n % kBlock == 0))
      out_sf[static_cast<size_t>(n_tile ? n / kBlock : n) * blocks + (c >> 4)] =
          sf[n_tile ? wgt_sf_offset(p, c >> 4, K_pad, n_tile) : act_sf_offset(p, c >> 4, K_pad)];
  }
}

// The values of a quantized activation: dec(q) 2^e, exact in fp32. A thread takes 8 columns of kDeqRows rows, whose
// loads go out together; HBM bounds it (4608 rows of 12288 to bf16 in 28.4 us, 6.0 TB/s).
constexpr int kDeqRows = 4;
template <bool F32>
__global__ void __launch_bounds__(256) dequantize_act_kernel(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ sf, int M, int K,
                                                             int K_pad, void* __restrict__ out, long long ld) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int m0 = blockIdx.x * kDeqRows, c = blockIdx.y * 256 + threadIdx.x;
  if (8 * c >= K) return;
  uint2 q[kDeqRows];
  uint32_t e[kDeqRows];
#pragma unroll
  for (int r = 0; r < kDeqRows; ++r) {
    const int m = m0 + r;  // a row of padding (allocated up to M_pad) may be read
    q[r] = __ldg(reinterpret_cast<const uint2*>(codes + static_cast<size_t>(m) * K_pad + 8 * c));
    e[r] = __ldg(sf + act_sf_offset(m, c >> 4, K_pad));
  }
#pragma unroll
  for (int r = 0; r < kDeqRows; ++r) {
    const long long m = m0 + r;
    if (m >= M) break;
    const float s = mx::scale_value(e[r]);
    const uint32_t pair[4] = {q[r].x & 0xFFFFu, q[r].x >> 16, q[r].y & 0xFFFFu, q[r].y >> 16};
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = mul2_rn(e4m3x2_value(pair[j]), make_float2(s, s));
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

}  // namespace fp8b
}  // namespace svdq
