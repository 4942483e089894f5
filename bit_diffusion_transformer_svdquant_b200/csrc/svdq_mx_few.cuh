// The MXFP4 layer for few rows (single tokens, conditioning vectors, short batches).
//
// At few rows the layer streams its weight: 17/32 bytes per weight element, read once. The pair GEMM's 256-row
// tiles then leave most of the tensor pipe and, at 24 to 72 tiles, most SMs idle, so here the roles are
// exchanged: 128 weight rows are the MMA's M side, the tokens its N side (16 to 128 columns, SwiGLU to 64), and K is
// split over a thread-block cluster, so that about every SM streams a share of the weight. Each CTA sums
// its K share in TMEM; the partial sums meet in distributed shared memory, every CTA of the cluster
// finishing its part of the tokens, in rank order (the result does not depend on timing).
//
// The quantizer for few rows splits K over clusters too: a row's 32-element blocks are independent, and
// the down-projection's partial sums meet at the cluster's first CTA, in a fixed order.
//
// Measured on B200 for one token of 3072 -> 9216, r = 32, weight from HBM: quantizer 3.9 us, product 7.7 us (2.0 TB/s),
// the layer 11.8 us; for kernel 1 and the pair GEMM 11.0 and 9.3 us. Launch, cluster set-up, the first loads and the
// exchange of the sums come one after another and bound both.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "svdq_gemm.cuh"
#include "svdq_mx.cuh"
#include "svdq_ptx.cuh"
#include "svdq_quant.cuh"

namespace svdq {
namespace mx {

// The product's tokens at most, for NB blocks of weight rows per CTA: two (SwiGLU) leave room for two ring
// stages beside the sums of 64 tokens only.
__host__ __device__ constexpr int few_max_cols(int NB) { return NB == 2 ? 64 : 128; }
constexpr int kFewMaxStages = 12;

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// ---------------------------------------------------------------- quantizer
struct FewQuantArgs {
  const __nv_bfloat16* X;
  long long ldx;
  const float* inv_lambda;        // [K_pad]
  const __nv_bfloat16* L1s_t;     // [R][K_pad]
  uint8_t* codes;
  uint8_t* sf;
  __nv_bfloat16* U;
  int M, K, K_pad, M_pad, rows;   // rows per CTA: 1, 2, 4 or 8
};
constexpr int kFewQuantCluster = 8;

// Clusters of 8 CTAs over K, `rows` rows each. First the CTA's 8 warps quantize their K share of the rows
// (8 / rows warps per row, 8 columns per lane, four lanes a block), leaving the raw values in shared
// memory. Then, chunk by chunk of L1s^T in shared memory, lane j of warp w sums column j of U (R = 64:
// columns j and j + 32; R = 16: two halves of the warp's columns) over the warp's columns of the chunk
// for all rows at once. The sums of the warps, then those of the CTAs, are added in order.
// What bounds it is latency: the loads of a chunk go out together, the next chunk's before this one's
// sums (with every lane loading L1s^T as it needed it, one row took 7.7 us and eight rows 12.5 us of
// K = 3072, r = 32 on B200). Rows of padding are not written.
template <int R>
__global__ void __launch_bounds__(256) few_quant_kernel(const FewQuantArgs a) {
  constexpr int kRows = 8;
  constexpr int kFewChunk = R == 64 ? 128 : 256;           // columns of L1s^T in shared memory at a time
  constexpr int kLd = kFewChunk + 8;                       // 16-byte accesses of neighbouring rows j meet no bank twice
  constexpr int kPer = R > 0 ? (R * kFewChunk / 8 + 255) / 256 : 1;  // 16-byte pieces of a chunk per thread
  __shared__ __align__(16) __nv_bfloat16 l1[R > 0 ? R * kLd : 8];
  float* const warp_part = reinterpret_cast<float*>(l1);   // [8 warps][8 rows][R], once l1 has been read
  static_assert(R == 0 || R * kLd * 2 >= 8 * kRows * R * 4, "the warps' sums fit in l1");
  extern __shared__ __align__(16) uint8_t x_smem[];        // raw bf16 rows of this CTA's K share
  __nv_bfloat16* const xs = reinterpret_cast<__nv_bfloat16*>(x_smem);
  __shared__ float part[R > 0 ? kFewQuantCluster * kRows * R : 1];  // at the cluster's first CTA
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  if constexpr (R > 0) {
    __syncwarp();
    cluster_arrive();  // the first CTA runs before its shared memory is written
  }
  grid_dependency_wait();
  grid_launch_dependents();
  const int m0 = (blockIdx.x / kFewQuantCluster) * a.rows;
  const int per_row = 8 / a.rows, row = warp / per_row, wi = warp % per_row, m = m0 + row;
  const int share = a.K_pad / kFewQuantCluster, k_beg = static_cast<int>(rank) * share, eights = share / 8;
  uint4 next[kPer];
  auto load_chunk = [&](int c0) {  // columns [c0, c0 + kFewChunk) of the share, whole groups of 8
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = threadIdx.x + 256 * i, j = at / (kFewChunk / 8), c = c0 + 8 * (at % (kFewChunk / 8));
      next[i] = make_uint4(0u, 0u, 0u, 0u);
      if (j < R && c < share) next[i] = ldg_stream(a.L1s_t + static_cast<size_t>(j) * a.K_pad + k_beg + c);
    }
  };
  if constexpr (R > 0) load_chunk(0);
  if (m < a.M) {
    for (int c0 = 32 * wi; c0 < eights; c0 += 32 * per_row) {
      const int c = c0 + lane, k = k_beg + 8 * c;
      const bool in = c < eights;
      uint4 x = make_uint4(0u, 0u, 0u, 0u);
      if (in && k < a.K) x = ldg_stream(a.X + m * a.ldx + k);
      float v[8];
      bf16x8_to_f32(x, v);
      float4 l0 = make_float4(1.0f, 1.0f, 1.0f, 1.0f), l1v = l0;
      if (in) {
        l0 = __ldg(reinterpret_cast<const float4*>(a.inv_lambda + k));
        l1v = __ldg(reinterpret_cast<const float4*>(a.inv_lambda + k + 4));
      }
      const float2 q[4] = {mul2_rn(make_float2(v[0], v[1]), make_float2(l0.x, l0.y)),
                           mul2_rn(make_float2(v[2], v[3]), make_float2(l0.z, l0.w)),
                           mul2_rn(make_float2(v[4], v[5]), make_float2(l1v.x, l1v.y)),
                           mul2_rn(make_float2(v[6], v[7]), make_float2(l1v.z, l1v.w))};
      uint32_t s;
      const uint32_t codes = quarter_block(q, s);
      if (in) {
        *reinterpret_cast<uint32_t*>(a.codes + static_cast<size_t>(m) * (a.K_pad >> 1) + (k >> 1)) = codes;
        if ((k & 31) == 0) a.sf[act_sf_offset(m, k >> 5, a.K_pad)] = static_cast<uint8_t>(s);
        if constexpr (R > 0) *reinterpret_cast<uint4*>(xs + row * share + 8 * c) = x;
      }
    }
  }
  if constexpr (R > 0) {
    constexpr int kCols = R == 64 ? 2 : 1;                 // columns of U per lane
    constexpr int kHalves = R == 16 ? 2 : 1;               // lanes that share a column
    float u[kRows][kCols];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int j = 0; j < kCols; ++j) u[r][j] = 0.0f;
    for (int c0 = 0; c0 < share; c0 += kFewChunk) {
      __syncthreads();  // the rows are in shared memory; the last chunk has been read
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = threadIdx.x + 256 * i, j = at / (kFewChunk / 8);
        if (j < R) *reinterpret_cast<uint4*>(l1 + j * kLd + 8 * (at % (kFewChunk / 8))) = next[i];
      }
      __syncthreads();
      if (c0 + kFewChunk < share) load_chunk(c0 + kFewChunk);
      // a warp takes an eighth of the chunk's columns, in groups of 8
      const int j = R == 16 ? lane & 15 : lane;
#pragma unroll
      for (int g = 0; g < kFewChunk / 64 / kHalves; ++g) {
        const int c = kFewChunk / 8 * warp + 8 * (g * kHalves + (R == 16 ? lane >> 4 : 0));
        if (c0 + c < share) {
          float w[kCols][8];
#pragma unroll
          for (int jj = 0; jj < kCols; ++jj)
            bf16x8_to_f32(*reinterpret_cast<const uint4*>(l1 + (j + 32 * jj) * kLd + c), w[jj]);
#pragma unroll
          for (int r = 0; r < kRows; ++r) {
            if (r < a.rows) {
              float x[8];
              bf16x8_to_f32(*reinterpret_cast<const uint4*>(xs + r * share + c0 + c), x);
#pragma unroll
              for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int jj = 0; jj < kCols; ++jj) u[r][jj] = fmaf(x[e], w[jj][e], u[r][jj]);
            }
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRows; ++r)
      if (r < a.rows) {
#pragma unroll
        for (int jj = 0; jj < kCols; ++jj) {
          float v = u[r][jj];
          if constexpr (R == 16) v += __shfl_xor_sync(0xffffffffu, v, 16);
          if (R != 16 || lane < 16) warp_part[(warp * kRows + r) * R + lane + 32 * jj] = v;
        }
      }
    __syncthreads();
    cluster_wait();
    float* const dst = cluster_map_generic(part, 0) + rank * kRows * R;
    for (int i = threadIdx.x; i < a.rows * R; i += 256) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += warp_part[w * kRows * R + i];
      dst[i] = s;
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (rank == 0) {
      for (int i = threadIdx.x; i < a.rows * R; i += 256) {
        const int r = i / R, j = i - r * R;
        if (m0 + r >= a.M) break;
        float s = 0.0f;
#pragma unroll
        for (int rk = 0; rk < kFewQuantCluster; ++rk) s += part[rk * kRows * R + i];
        const __nv_bfloat16 hi = __float2bfloat16_rn(s);
        a.U[static_cast<size_t>(m0 + r) * R + j] = hi;
        a.U[(static_cast<size_t>(a.M_pad) + m0 + r) * R + j] = __float2bfloat16_rn(__fsub_rn(s, __bfloat162float(hi)));
      }
    }
  }
}

// ---------------------------------------------------------------- product
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb));
}

struct FewGemmArgs {
  const uint8_t* sfw;         // weight scales
  const uint8_t* sfx;         // activation scales
  const __nv_bfloat16* bias;
  void* Y;
  long long ldy;
  unsigned long long wait_ns;
  int M, M_pad, N, K, r;      // N: the weight's true width, K: padded
  int n_tile, cols;           // cols: token columns of the MMA (16, 32, 64 or 128)
  int stages, tmem_cols, out_f32, has_bias;
};
constexpr int kFewThreads = 192;  // warp 0: TMA, warp 1: TMEM and MMA, warps 2..5: epilogue

// A ring stage of one 256-wide K step: NB x 128 weight rows, the token rows, 2 (NB + 1) scale atoms.
__host__ __device__ constexpr int few_stage_bytes(int NB, int cols) {
  return NB * 128 * 128 + cols * 128 + 2 * 512 * (NB + 1);
}
__host__ __device__ constexpr int few_stage_tmem(int NB) { return 8 * (NB + 1); }
// the CTA's sums in shared memory: [cols][NB][128]
__host__ __device__ constexpr int few_part_bytes(int NB, int cols) { return NB * cols * 512; }

// NB = 1: block b of 128 output columns (weight rows in tile order). NB = 2 (SwiGLU, n_tile 256): gate and
// up rows of 128 outputs, in two accumulators. Cluster rank c sums K steps [c n / ranks, (c + 1) n / ranks)
// of n; rank 0 also the low-rank branch.
// Everything is read after the kernel before has completed. Reading the weight while the quantizer runs, into
// the ring (10.7 -> 11.8 us) or only into L2 (11.6 us), made a layer of one token slower, not faster (3072 ->
// 9216, r = 32, weight in L2): the quantizer's own loads wait behind it.
template <int NB>
__global__ void __launch_bounds__(kFewThreads, 1)
    few_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const __grid_constant__ CUtensorMap tmU, const __grid_constant__ CUtensorMap tmL2,
                    const FewGemmArgs a) {
  constexpr int kMaxStages = kFewMaxStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_smem;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cols = a.cols, stages = a.stages, stage_bytes = few_stage_bytes(NB, cols);
  const uint32_t sbase = smem_addr(smem), bar0 = smem_addr(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  const uint32_t acc_bar = bar0 + 8u * (2 * kMaxStages), drain_bar = acc_bar + 8u;
  float* const part = reinterpret_cast<float*>(smem + stages * stage_bytes);
  const int off_x = NB * 128 * 128, off_sfw = off_x + cols * 128, off_sfx = off_sfw + NB * 2 * 512;
  volatile int* abort_flag = &abort_smem;
  const uint32_t ranks = cluster_nctarank(), rank = cluster_ctarank();
  const int block = blockIdx.x / ranks;
  const int steps = a.K >> 8;
  const int k_beg = static_cast<int>(rank) * steps / static_cast<int>(ranks);
  const int k_end = (static_cast<int>(rank) + 1) * steps / static_cast<int>(ranks);
  // tile and 128-column block inside it, and the packed rows of its two halves
  const int atoms = a.n_tile >> 7;
  const int nb0 = NB == 2 ? block : block / atoms, at = NB == 2 ? 0 : block - nb0 * atoms;
  auto packed_row = [&](int which, int half) {
    return nb0 * a.n_tile + packed_of_tile_col((at + which) * 128 + 64 * half, a.n_tile);
  };
  const int lr_slots = rank == 0 ? (a.r + kLrChunk - 1) / kLrChunk : 0;
  const int rc = a.r < kLrChunk ? a.r : kLrChunk;

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(acc_bar, 1);
    mbar_init(drain_bar, 1);
    abort_smem = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&tmem_slot), a.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (ranks > 1) cluster_arrive();  // waited for before the first write into another CTA
  const int slots = lr_slots + k_end - k_beg;
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t tmem = tmem_slot;
  unsigned* status = &g_svdq_status;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, armed = 0, armed_parity = 0;
      for (int slot = 0; slot < slots; ++slot) {
        if (!mbar_wait_bounded(empty_bar(stage), phase ^ 1u, a.wait_ns, status, kStatusProducer, abort_flag)) break;
        const uint32_t sa = sbase + stage * stage_bytes, fb = full_bar(stage);
        armed |= 1u << stage;
        armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
        if (slot < lr_slots) {
          mbar_arrive_expect_tx(fb, static_cast<uint32_t>((NB * 128 + 2 * cols) * rc * 2));
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              tma_load_2d(sa + (b * 128 + h * 64) * rc * 2, &tmL2, slot * kLrChunk, packed_row(b, h), fb);
          tma_load_2d(sa + off_x, &tmU, slot * kLrChunk, 0, fb);
          tma_load_2d(sa + off_x + cols * rc * 2, &tmU, slot * kLrChunk, a.M_pad, fb);
        } else {
          const int k = k_beg + slot - lr_slots;
          mbar_arrive_expect_tx(fb, static_cast<uint32_t>(stage_bytes));
#pragma unroll
          for (int b = 0; b < NB; ++b) {
#pragma unroll
            for (int h = 0; h < 2; ++h) tma_load_2d(sa + b * 16384 + h * 8192, &tmW, k * 128, packed_row(b, h), fb);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              bulk_load(sa + off_sfw + (b * 2 + i) * 512,
                        a.sfw + (((static_cast<size_t>(nb0) * (a.K >> 7) + 2 * k + i) * atoms + at + b) << 9), 512, fb);
          }
          tma_load_2d(sa + off_x, &tmX, k * 128, 0, fb);
          bulk_load(sa + off_sfx, a.sfx + (static_cast<size_t>(2 * k) << 9), 1024, fb);
        }
        if (++stage == stages) { stage = 0; phase ^= 1u; }
      }
      // every copy this thread started has landed before the CTA may leave
      for (int s = 0; s < stages; ++s)
        if (armed & (1u << s))
          mbar_wait_bounded(full_bar(s), (armed_parity >> s) & 1u, a.wait_ns, status, kStatusDrain, nullptr);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, accumulate = 0;
      bool ok = true;
      const uint32_t id_lr = idesc_bf16(128, cols);
      const uint32_t id0 = idesc_mxf4(128, cols, 0), id2 = idesc_mxf4(128, cols, 2);
      for (int slot = 0; slot < slots; ++slot) {
        if (!(ok = mbar_wait_bounded(full_bar(stage), phase, a.wait_ns, status, kStatusMma, abort_flag))) break;
        tc_fence_after();
        const uint32_t sa = sbase + stage * stage_bytes;
        if (slot < lr_slots) {
          const uint32_t swz = lr_swizzle_mode(rc), sbo = 8u * rc * 2u;
          for (int j = 0; j < rc >> 4; ++j) {
            const uint64_t hi = smem_desc(sa + off_x + 32 * j, 16, sbo, swz);
            const uint64_t lo = smem_desc(sa + off_x + cols * rc * 2 + 32 * j, 16, sbo, swz);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              const uint64_t l2 = smem_desc(sa + b * 128 * rc * 2 + 32 * j, 16, sbo, swz);
              mma_bf16(tmem + b * cols, l2, hi, id_lr, accumulate);
              mma_bf16(tmem + b * cols, l2, lo, id_lr, 1u);
            }
            accumulate = 1;
          }
        } else {
          // scale factors into this stage's TMEM columns (free: the stage's last MMAs have completed)
          const uint32_t tsf = tmem + NB * cols + stage * few_stage_tmem(NB);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
              tc_cp_sf(tsf + 8 * b + 4 * i, smem_desc(sa + off_sfw + (b * 2 + i) * 512, 0, 128, 0));
            tc_cp_sf(tsf + 8 * NB + 4 * i, smem_desc(sa + off_sfx + i * 512, 0, 128, 0));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t x = smem_desc(sa + off_x + 32 * j, 16, 1024, 2);
            const uint32_t id = j & 1 ? id2 : id0, i4 = 4 * (j >> 1);
#pragma unroll
            for (int b = 0; b < NB; ++b)
              mma_mxf4(tmem + b * cols, smem_desc(sa + b * 16384 + 32 * j, 16, 1024, 2), x, id, tsf + 8 * b + i4,
                       tsf + 8 * NB + i4, accumulate);
            accumulate = 1;
          }
        }
        tc_commit(empty_bar(stage));
        if (++stage == stages) { stage = 0; phase ^= 1u; }
      }
      if (ok) tc_commit(acc_bar);
      tc_commit(drain_bar);
      mbar_wait_bounded(drain_bar, 0, a.wait_ns, status, kStatusDrain, nullptr);
    }
  }
  __syncwarp();

  // Epilogue. Warps 2..5 lay the CTA's sums out in shared memory, [token][accumulator][128 outputs];
  // then all warps finish the tokens m with m % ranks == rank, a warp per token, four outputs per lane:
  // the ranks' sums in order, bias, SwiGLU, one 8- or 16-byte store.
  if (warp >= 2) {
    const int q = warp & 3, n_l = q * 32 + lane;
    bool got = mbar_wait_bounded(acc_bar, 0, a.wait_ns, status, kStatusEpilogue, abort_flag);
    got = __all_sync(0xffffffffu, got);
    tc_fence_after();
    if (got) {
      const uint32_t td = tmem + (static_cast<uint32_t>(q * 32) << 16);
      for (int c = 0; c < a.M; c += 16)
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float v[16];
          tmem_ld_32x16(td + b * cols + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) part[((c + i) * NB + b) * 128 + n_l] = v[i];
        }
    }
  }
  __syncwarp();
  if (ranks > 1) {
    cluster_wait();  // the barrier arrived on at the start
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  {
    const int j0 = nb0 * (NB == 2 ? 128 : a.n_tile) + at * 128 + 4 * lane;  // the first of four output columns
    const int n_out = NB == 2 ? a.N >> 1 : a.N;
    const bool in = j0 < n_out;  // n_out is a multiple of 8: all four or none
    float bias[NB][4] = {};
    if (a.has_bias && in) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(a.bias + j0 + b * n_out));
        bias[b][0] = __uint_as_float(w.x << 16);
        bias[b][1] = __uint_as_float(w.x & 0xFFFF0000u);
        bias[b][2] = __uint_as_float(w.y << 16);
        bias[b][3] = __uint_as_float(w.y & 0xFFFF0000u);
      }
    }
    for (int m = static_cast<int>(rank + ranks * warp); m < a.M && !*abort_flag; m += static_cast<int>(ranks) * (kFewThreads / 32)) {
      float y[NB][4] = {};
      for (uint32_t rk = 0; rk < ranks; ++rk) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const float4* src = reinterpret_cast<const float4*>(part + (m * NB + b) * 128) + lane;
          const float4 s = ranks > 1 ? *cluster_map_generic(src, rk) : *src;
          y[b][0] += s.x;
          y[b][1] += s.y;
          y[b][2] += s.z;
          y[b][3] += s.w;
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) y[b][i] += bias[b][i];
      if constexpr (NB == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) y[0][i] = silu_times(y[0][i], y[NB - 1][i]);
      }
      if (in) {
        if (a.out_f32) {
          *reinterpret_cast<float4*>(static_cast<float*>(a.Y) + m * a.ldy + j0) = make_float4(y[0][0], y[0][1], y[0][2], y[0][3]);
        } else {
          const __nv_bfloat162 p0 = __floats2bfloat162_rn(y[0][0], y[0][1]), p1 = __floats2bfloat162_rn(y[0][2], y[0][3]);
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.Y) + m * a.ldy + j0) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&p0), *reinterpret_cast<const uint32_t*>(&p1));
        }
      }
    }
  }
  __syncwarp();
  if (ranks > 1) {  // no CTA leaves while another may read its sums
    cluster_arrive();
    cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, a.tmem_cols);
  }
}

}  // namespace mx
}  // namespace svdq
