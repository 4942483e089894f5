// C ABI of the block-scaled FP8 variant of the layer (svdq_fp8b_*): argument checks, buffer layouts, TMA
// descriptors and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>
#include <mutex>

#include "svdq.h"
#include "svdq_fp8b.cuh"
#include "svdq_host.h"

using namespace svdq::host;

namespace {

constexpr int kStages384 = 4;
constexpr int kStages256 = 5;
constexpr int kStages128 = 7;
template <int N_TILE, int STAGES>
using Layout = svdq::PairGemmLayout<true, N_TILE, STAGES, svdq::fp8b::Gemm::kSfAtomsK, svdq::fp8b::Gemm::kBiasSmem,
                                    svdq::fp8b::Gemm::kSfShare>;

struct State {
  bool ready = false;
  int max_pairs[3] = {0, 0, 0};  // co-resident CTA pairs of the GEMM for n_tile 384, 256, 128
  int few_clusters[4] = {0, 0, 0, 0};  // co-resident few-row clusters of 1, 2, 4 and 8 CTAs
};
using svdq::fp8b::Few;
std::mutex g_mu;
State g_state[kMaxDevices];

template <int N_TILE, int STAGES, class F = svdq::fp8b::Gemm>
svdq_status gemm_setup(int sms, int* max_pairs) {
  auto* kern = svdq::pair_gemm_kernel<F, N_TILE, STAGES>;
  SVDQ_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<N_TILE, STAGES>::kSmem));
  return max_cta_pairs(reinterpret_cast<const void*>(kern), Layout<N_TILE, STAGES>::kSmem, sms, max_pairs);
}
template <int R>
svdq_status quant_setup() {
  auto* kern = svdq::quant_act_kernel<R, svdq::fp8b::Act>;
  SVDQ_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, svdq::Q1Layout<R>::kSmem));
  return SVDQ_OK;
}

template <int R>
svdq_status few_quant_setup() {
  SVDQ_CUDA(cudaFuncSetAttribute(svdq::mx::few_quant_kernel<Few, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 2 * svdq::mx::kFewQuantMaxK));
  return SVDQ_OK;
}
template <int NB>
svdq_status few_setup(int sms, int* clusters) {
  auto* kern = svdq::mx::few_gemm_kernel<Few, NB>;
  SVDQ_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, svdq::mx::kFewMaxSmem));
  for (int i = 0; i < 4; ++i) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1 << i;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((sms >> i) << i, 1, 1);
    cfg.blockDim = dim3(svdq::mx::kFewThreads, 1, 1);
    cfg.dynamicSmemBytes = svdq::mx::kFewMinSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    SVDQ_CUDA(cudaOccupancyMaxActiveClusters(&clusters[i], kern, &cfg));
  }
  return SVDQ_OK;
}

// The kernels are set up on the first call on a device.
svdq_status ready(int* dev_out, int* sm_out) {
  int dev = 0, sms = 0;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;
  std::lock_guard<std::mutex> lk(g_mu);
  State& st = g_state[dev];
  if (!st.ready) {
    svdq_status s = gemm_setup<384, kStages384>(sms, &st.max_pairs[0]);
    if (s == SVDQ_OK) s = gemm_setup<256, kStages256, svdq::fp8b::Gemm256Of384>(sms, &st.max_pairs[1]);
    if (s == SVDQ_OK) s = gemm_setup<256, kStages256>(sms, &st.max_pairs[1]);
    if (s == SVDQ_OK) s = gemm_setup<128, kStages128>(sms, &st.max_pairs[2]);
    if (s == SVDQ_OK) s = quant_setup<16>();
    if (s == SVDQ_OK) s = quant_setup<32>();
    if (s == SVDQ_OK) s = quant_setup<64>();
    if (s == SVDQ_OK) s = few_quant_setup<16>();
    if (s == SVDQ_OK) s = few_quant_setup<32>();
    if (s == SVDQ_OK) s = few_quant_setup<64>();
    if (s == SVDQ_OK) s = few_setup<2>(sms, st.few_clusters);
    if (s == SVDQ_OK) s = few_setup<1>(sms, st.few_clusters);
    if (s != SVDQ_OK) return s;
    st.ready = true;
  }
  if (dev_out) *dev_out = dev;
  if (sm_out) *sm_out = sms;
  return SVDQ_OK;
}

constexpr int kMax = 1 << 20;
bool k_ok(int K) { return K > 0 && K % 8 == 0 && K <= kMax; }
bool n_ok(int N, int swiglu) { return N > 0 && N % (swiglu ? 16 : 8) == 0 && N <= kMax; }
int k_pad(int K) { return round_up(K, svdq::fp8b::kBlock); }
// Tile width that a weight is packed for: 384, which streams the fewest operand bytes per flop, unless padding N to it
// costs more than that gains over 256 (GEMM us at 256 / 384: 16896 x 3072 -> 9216 359 / 340, 4608 x 3072 -> 9216 99.5 / 94.1,
// 4608 x 12288 -> 3072 124.5 / 116.7). Narrower tiles of the same packing serve the row counts at which wide ones would
// leave SMs idle. SwiGLU pairs gate and up columns inside a tile of 256.
int n_tile_of(int N, int swiglu) {
  if (swiglu) return 256;
  return round_up(N, 384) * 100ll <= round_up(N, 256) * 103ll ? 384 : 256;
}
int n_pad(int N, int swiglu) { return swiglu ? round_up(N / 2, 128) * 2 : round_up(N, n_tile_of(N, 0)); }

struct WeightLayout {
  size_t codes, scales, inv_lambda, l1t, l2t, total;
};
WeightLayout weight_layout(int N_pad, int K_pad, int r) {
  WeightLayout l{};
  size_t off = 0;
  l.codes = off;
  off = align_up(off + static_cast<size_t>(N_pad) * K_pad);
  l.scales = off;
  off = align_up(off + static_cast<size_t>(N_pad / 128) * svdq::fp8b::sf_atoms(K_pad) * 512);
  l.inv_lambda = off;
  off = align_up(off + static_cast<size_t>(K_pad) * 4);
  l.l1t = off;
  off = align_up(off + static_cast<size_t>(r) * K_pad * 2);
  l.l2t = off;
  off = align_up(off + static_cast<size_t>(N_pad) * r * 2);
  l.total = off;
  return l;
}

struct ActLayout {
  size_t codes, scales, u, total;
  int M_pad, K_pad;
};
ActLayout act_layout(int M, int K, int r) {
  ActLayout l{};
  l.M_pad = round_up(M, 128);
  l.K_pad = k_pad(K);
  size_t off = 0;
  l.codes = off;
  off = align_up(off + static_cast<size_t>(l.M_pad) * l.K_pad);
  l.scales = off;
  off = align_up(off + static_cast<size_t>(l.M_pad / 128) * svdq::fp8b::sf_atoms(l.K_pad) * 512);
  l.u = off;
  off = align_up(off + static_cast<size_t>(l.M_pad) * r * 2 * 2);  // hi and lo halves
  l.total = off;
  return l;
}

svdq_status check_weight(const svdq_fp8b_weight* w) {
  const int sw = w->swiglu_interleaved;
  if ((sw != 0 && sw != 1) || !n_ok(w->N, sw) || !k_ok(w->K) || !valid_r(w->r) || w->n_tile != n_tile_of(w->N, sw) ||
      w->N_pad != n_pad(w->N, sw) || w->K_pad != k_pad(w->K))
    return fail(SVDQ_ERR_INVALID_ARG,
                "block-scaled FP8 weight descriptor N=%d K=%d r=%d n_tile=%d is not one svdq_fp8b_pack_weight makes",
                w->N, w->K, w->r, w->n_tile);
  if (w->codes == nullptr || w->scales == nullptr || w->inv_lambda == nullptr ||
      (w->r > 0 && (w->L1s_t == nullptr || w->L2_t == nullptr)))
    return fail(SVDQ_ERR_INVALID_ARG, "block-scaled FP8 weight descriptor has a null buffer");
  return SVDQ_OK;
}

svdq_status check_act(const svdq_fp8b_act* a) {
  if (a->M < 1 || a->M >= (1 << 24) || !k_ok(a->K) || !valid_r(a->r) || a->M_pad != round_up(a->M, 128) ||
      a->K_pad != k_pad(a->K))
    return fail(SVDQ_ERR_INVALID_ARG,
                "block-scaled FP8 act descriptor M=%d M_pad=%d K=%d r=%d is not one svdq_fp8b_act_bind makes", a->M,
                a->M_pad, a->K, a->r);
  if (a->codes == nullptr || a->scales == nullptr || (a->r > 0 && a->U == nullptr))
    return fail(SVDQ_ERR_INVALID_ARG, "block-scaled FP8 act descriptor has a null buffer");
  return SVDQ_OK;
}

svdq_status fill_weight(uint8_t* b, int N, int K, int r, int swiglu, svdq_fp8b_weight* out) {
  svdq_fp8b_weight w{};
  w.N = N;
  w.K = K;
  w.r = r;
  w.swiglu_interleaved = swiglu ? 1 : 0;
  w.n_tile = n_tile_of(N, swiglu);
  w.N_pad = n_pad(N, swiglu);
  w.K_pad = k_pad(K);
  const WeightLayout l = weight_layout(w.N_pad, w.K_pad, r);
  w.codes = b + l.codes;
  w.scales = b + l.scales;
  w.inv_lambda = reinterpret_cast<float*>(b + l.inv_lambda);
  w.L1s_t = b + l.l1t;
  w.L2_t = b + l.l2t;
  static_assert(sizeof(w.tmap) >= 5 * sizeof(CUtensorMap), "tmap storage");
  CUtensorMap tm[5];  // codes, L2_t, L1s_t; codes and L2_t in boxes of 64 rows
  std::memset(tm, 0, sizeof(tm));
  const uint64_t r2 = static_cast<uint64_t>(r) * 2;
  svdq_status s = make_tmap(&tm[0], CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, w.K_pad, w.N_pad, w.K_pad, 128, w.n_tile / 2,
                            CU_TENSOR_MAP_SWIZZLE_128B);
  if (s == SVDQ_OK)
    s = make_tmap(&tm[3], CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, w.K_pad, w.N_pad, w.K_pad, 128, 64,
                  CU_TENSOR_MAP_SWIZZLE_128B);
  if (s == SVDQ_OK && r > 0)
    s = make_tmap(&tm[1], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w.L2_t, r, w.N_pad, r2, r < 32 ? r : 32, w.n_tile / 2,
                  lr_swizzle(r));
  if (s == SVDQ_OK && r > 0)
    s = make_tmap(&tm[4], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w.L2_t, r, w.N_pad, r2, r < 32 ? r : 32, 64, lr_swizzle(r));
  if (s == SVDQ_OK && r > 0)
    s = make_tmap(&tm[2], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w.L1s_t, w.K_pad, r, static_cast<uint64_t>(w.K_pad) * 2, 64,
                  r, CU_TENSOR_MAP_SWIZZLE_128B);
  if (s != SVDQ_OK) return s;
  for (int i = 0; i < 5; ++i) std::memcpy(&w.tmap[i][0], &tm[i], sizeof(CUtensorMap));
  *out = w;
  return SVDQ_OK;
}

svdq_status check_quantize(const uint16_t* X, long long ldx, const svdq_fp8b_weight* w, const svdq_fp8b_act* act) {
  if (X == nullptr || w == nullptr || act == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (act->K != w->K || act->r != w->r)
    return fail(SVDQ_ERR_INVALID_ARG, "act (K=%d r=%d) does not match weight (K=%d r=%d)", act->K, act->r, w->K, w->r);
  if (svdq_status s = check_weight(w); s != SVDQ_OK) return s;
  if (svdq_status s = check_act(act); s != SVDQ_OK) return s;
  if (!aligned16(X)) return fail(SVDQ_ERR_UNSUPPORTED, "X must be 16-byte aligned");
  if (ldx < act->K || ldx % 8 != 0 || ldx >= (1ll << 38))
    return fail(SVDQ_ERR_UNSUPPORTED, "row stride %lld of X: a multiple of 8 and at least K=%d", ldx, act->K);
  return SVDQ_OK;
}

svdq_status check_gemm(const svdq_fp8b_act* act, const svdq_fp8b_weight* w, const uint16_t* bias, svdq_epilogue epi,
                       const void* Y, long long ldy, svdq_out_dtype out_dtype) {
  if (act == nullptr || w == nullptr || Y == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (act->K != w->K || act->r != w->r) return fail(SVDQ_ERR_INVALID_ARG, "act does not match weight");
  if (svdq_status s = check_weight(w); s != SVDQ_OK) return s;
  if (svdq_status s = check_act(act); s != SVDQ_OK) return s;
  if (epi < SVDQ_EPI_NONE || epi > SVDQ_EPI_BIAS_SWIGLU) return fail(SVDQ_ERR_INVALID_ARG, "bad epilogue %d", epi);
  if (out_dtype != SVDQ_OUT_BF16 && out_dtype != SVDQ_OUT_F32) return fail(SVDQ_ERR_INVALID_ARG, "bad out dtype");
  const bool has_bias = (epi & 1) != 0, swiglu = (epi & 2) != 0;
  if (has_bias && bias == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "epilogue needs a bias");
  if (swiglu && !w->swiglu_interleaved) return fail(SVDQ_ERR_INVALID_ARG, "SwiGLU needs a weight packed with swiglu=1");
  if (!swiglu && w->swiglu_interleaved) return fail(SVDQ_ERR_INVALID_ARG, "weight packed for SwiGLU");
  const int n_out = swiglu ? w->N / 2 : w->N;
  const int esize = out_dtype == SVDQ_OUT_F32 ? 4 : 2;
  if (!aligned16(Y) || (bias != nullptr && !aligned16(bias))) return fail(SVDQ_ERR_UNSUPPORTED, "Y / bias alignment");
  if (ldy < n_out || (ldy * esize) % 16 != 0 || ldy >= (1ll << 37))
    return fail(SVDQ_ERR_UNSUPPORTED, "row stride %lld of Y: whole 16-byte units and at least %d", ldy, n_out);
  return SVDQ_OK;
}

// Where the few-row kernels run (measured on B200 with weights from HBM, us of the few-row kernel / the other).
// The quantizer with a branch up to 384 rows: K = 3072, r = 32: 4.2 / 11.8 at one row, 9.5 / 11.7 at 384, 15.7 / 11.7 at
// 512; K = 12288: 8.1 / 27.8, 25.0 / 27.8, 42.2 / 28.0; K = 256: 3.1 / 5.2, 5.5 / 5.4, 8.6 / 5.4. The few-row one sums U on the
// CUDA cores, every row its own: at 384 x 12288 instructions bound it (issue 60 %, ALU 44 %, DRAM 4 %). Kernel 1 takes as long
// for 1 row as for 512: at most 4 CTAs go through the K of 128 rows.
bool few_quant_rows(int M, int K_pad) { return M <= 384 && K_pad <= svdq::mx::kFewQuantMaxK - 1024; }
struct FewSplit {
  int blocks, ranks;  // CTA clusters over N, and their size over K
};
FewSplit few_split(const svdq_fp8b_weight* w, bool swiglu, int dev) {
  FewSplit s{swiglu ? w->N_pad / 256 : (w->N + 127) / 128, 1};
  std::lock_guard<std::mutex> lk(g_mu);
  for (int i = 1; i < 4; ++i)
    if (s.blocks <= g_state[dev].few_clusters[i] && (1 << i) <= w->K_pad / Few::kStepK) s.ranks = 1 << i;
  return s;
}
// The product of few rows wherever K is not short, and up to 128 where splitting K over the SMs outweighs its epilogue
// of M x N sums: 3072 -> 9216 9.8 / 12.7 at one row, 12.1 / 13.0 at 64, 13.5 / 13.0 at 96; 3072 -> 3072 6.6 / 11.3, 9.7 /
// 11.6 at 128; 12288 -> 3072 14.2 / 32.9, 17.9 / 33.2 at 128; 1024 -> 1024 4.1 / 5.9, 5.9 / 6.2 at 96, 6.6 / 6.2 at 128;
// 1024 -> 9216 6.0 / 7.3, 6.8 / 7.5 at 32, 8.3 / 7.5 at 64; 256 -> 9216 4.5 / 5.1, 5.0 / 5.2 at 16, 5.9 / 5.3 at 48; 512 ->
// 3072 4.3 / 4.8, 4.5 / 4.8 at 16, 5.1 / 4.8 at 32. SwiGLU up to its 64: 3072 -> 24576 18.9 / 24.7, 23.9 / 25.1 at 64;
// 256 -> 24576 4.4 / 7.5, 7.4 / 7.9 at 64.
bool few_product_rows(int M, const svdq_fp8b_weight* w, bool swiglu) {
  if (swiglu) return M <= svdq::mx::few_max_cols(2);
  return M <= (w->K_pad >= 1024 ? 32 : 16) || (M <= svdq::mx::few_max_cols(1) && 192ll * w->K_pad >= 1ll * M * w->N);
}

// The GEMM's tile width: the one whose rounds of tiles over the resident CTA pairs take least, a round counted 8 at 384
// columns, 6 at 256 and 5 at 128, as measured (3072 -> 9216, one round of each: 16.1, 12.3 and 10.1 us past the kernel's
// fixed 3). Of a weight packed 384 wide, us at 384 / 256: 512 rows 3072 -> 9216 19.4 / 15.4, 768 rows 20.0 / 24.0, 1024 rows
// 31.2 / 25.3, 1024 rows 12288 -> 3072 48.8 / 37.9; 256 rows 3072 -> 9216 at 256 / 128 15.4 / 12.8. SwiGLU pairs columns of
// the packed tile and keeps it.
int tile_of(int m_pairs, const svdq_fp8b_weight* w, const int* most) {
  constexpr int kTile[3] = {384, 256, 128}, kCost[3] = {8, 6, 5};
  int tile = 0;
  long long best = 0;
  for (int i = w->n_tile == 384 ? 0 : 1; i < 3; ++i) {
    const long long tiles = static_cast<long long>(m_pairs) * ((w->N + kTile[i] - 1) / kTile[i]);
    const long long cost = (tiles + most[i] - 1) / most[i] * kCost[i];
    if (tile == 0 || cost < best) best = cost, tile = kTile[i];
  }
  return tile;
}

svdq_status few_gemm(const svdq_fp8b_act* act, const svdq_fp8b_weight* w, const uint16_t* bias, bool has_bias, bool swiglu,
                     void* Y, long long ldy, int esize, const FewSplit& split, cudaStream_t st) {
  using namespace svdq::mx;
  using svdq::fp8b::Few;
  static_assert(
      2 * few_stage_bytes(1, few_max_cols(1), Few::kAtoms) + few_part_bytes(1, few_max_cols(1)) + 1024 <= kFewMaxSmem &&
          2 * few_stage_bytes(2, few_max_cols(2), Few::kAtoms) + few_part_bytes(2, few_max_cols(2)) + 1024 <= kFewMaxSmem,
      "two stages always fit");
  static_assert(few_max_cols(1) + kFewMaxStages * few_stage_tmem(1, Few::kAtoms) <= 512 &&
                    2 * few_max_cols(2) + kFewMaxStages * few_stage_tmem(2, Few::kAtoms) <= 512,
                "TMEM budget");
  const int NB = swiglu ? 2 : 1, r = w->r;
  const int cols = act->M <= 16 ? 16 : act->M <= 32 ? 32 : act->M <= 64 ? 64 : 128;
  const int steps = w->K_pad / Few::kStepK, stage = few_stage_bytes(NB, cols, Few::kAtoms), part = few_part_bytes(NB, cols);
  const int slots = (steps + split.ranks - 1) / split.ranks + (r + 31) / 32;
  int stages = (kFewMaxSmem - 1024 - part) / stage;
  if (stages > slots) stages = slots;  // one, where a CTA has a single K step and no branch
  if (stages > kFewMaxStages) stages = kFewMaxStages;
  int tmem = 32;
  while (tmem < NB * cols + stages * few_stage_tmem(NB, Few::kAtoms)) tmem *= 2;
  CUtensorMap tmW, tmX, tmU, tmL2;
  std::memset(&tmU, 0, sizeof(tmU));
  std::memcpy(&tmW, &w->tmap[3][0], sizeof(CUtensorMap));
  std::memcpy(&tmL2, &w->tmap[4][0], sizeof(CUtensorMap));
  if (svdq_status s = make_tmap(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, act->codes, act->K_pad, act->M_pad, act->K_pad, 128,
                                cols, CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  if (r > 0) {
    if (svdq_status s = make_tmap(&tmU, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, act->U, r, 2 * static_cast<uint64_t>(act->M_pad),
                                  static_cast<uint64_t>(r) * 2, r < 32 ? r : 32, cols, lr_swizzle(r));
        s != SVDQ_OK)
      return s;
  }
  FewGemmArgs g{};
  g.sfw = static_cast<const uint8_t*>(w->scales);
  g.sfx = static_cast<const uint8_t*>(act->scales);
  g.bias = reinterpret_cast<const __nv_bfloat16*>(bias);
  g.Y = Y;
  g.ldy = ldy;
  g.wait_ns = wait_limit_ns();
  g.M = act->M;
  g.M_pad = act->M_pad;
  g.N = w->N;
  g.K = w->K_pad;
  g.r = r;
  g.n_tile = w->n_tile;
  g.cols = cols;
  g.stages = stages;
  g.tmem_cols = tmem;
  g.out_f32 = esize == 4 ? 1 : 0;
  g.has_bias = has_bias ? 1 : 0;
  const int smem = stages * stage + part + 1024;
  const cudaError_t e = launch(NB == 2 ? few_gemm_kernel<Few, 2> : few_gemm_kernel<Few, 1>,
                               dim3(split.blocks * split.ranks), kFewThreads, smem < kFewMinSmem ? kFewMinSmem : smem,
                               split.ranks, st, tmW, tmX, tmU, tmL2, g);
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of few_gemm_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("few_gemm_kernel (block-scaled FP8)");
}

// svdq_fp8b_quantize_act on checked arguments.
svdq_status quantize(const uint16_t* X, long long ldx, const svdq_fp8b_weight* w, const svdq_fp8b_act* act,
                     svdq_stream_t stream) {
  int dev, sms;
  if (svdq_status s = ready(&dev, &sms); s != SVDQ_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int r = w->r;
  if (r == 0) {
    const long long chunks = act->K_pad / 16;
    const int rows = static_cast<long long>(act->M) * chunks > 4ll * 256 * 4 * sms ? 4 : 1;
    const long long blocks = ((act->M + rows - 1) / rows * chunks + 255) / 256;
    if (blocks > 0x7FFFFFFFll) return fail(SVDQ_ERR_UNSUPPORTED, "M=%d K=%d: too many blocks", act->M, act->K);
    const bool wide = ((reinterpret_cast<uintptr_t>(X) | static_cast<uintptr_t>(ldx * 2)) & 31u) == 0;
    auto* kern = rows == 4 ? (wide ? svdq::fp8b::quant_rows_kernel<4, true> : svdq::fp8b::quant_rows_kernel<4, false>)
                           : (wide ? svdq::fp8b::quant_rows_kernel<1, true> : svdq::fp8b::quant_rows_kernel<1, false>);
    const cudaError_t e = launch(kern,
                                 dim3(static_cast<unsigned>(blocks)), 256, 0, 0, st,
                                 reinterpret_cast<const __nv_bfloat16*>(X), ldx, static_cast<const float*>(w->inv_lambda),
                                 act->M, act->K, act->K_pad, static_cast<uint8_t*>(act->codes),
                                 static_cast<uint8_t*>(act->scales));
    if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of fp8b::quant_rows_kernel failed: %s", cudaGetErrorString(e));
    return check_launch("fp8b::quant_rows_kernel");
  }
  if (few_quant_rows(act->M, act->K_pad)) {
    svdq::mx::FewQuantArgs f{};
    f.X = reinterpret_cast<const __nv_bfloat16*>(X);
    f.ldx = ldx;
    f.inv_lambda = w->inv_lambda;
    f.L1s_t = static_cast<const __nv_bfloat16*>(w->L1s_t);
    f.codes = static_cast<uint8_t*>(act->codes);
    f.sf = static_cast<uint8_t*>(act->scales);
    f.U = static_cast<__nv_bfloat16*>(act->U);
    f.M = act->M;
    f.K = act->K;
    f.K_pad = act->K_pad;
    f.M_pad = act->M_pad;
    constexpr int kCluster = svdq::mx::kFewQuantCluster;
    f.share = round_up((act->K_pad + kCluster - 1) / kCluster, svdq::fp8b::kBlock);
    // rows per cluster: the fewest that keep all clusters on the SMs at once, as for MXFP4
    f.rows = 1;
    while (f.rows < 8 && (act->M + f.rows - 1) / f.rows * kCluster > sms) f.rows *= 2;
    auto* kern = r == 16   ? svdq::mx::few_quant_kernel<Few, 16>
                 : r == 32 ? svdq::mx::few_quant_kernel<Few, 32>
                           : svdq::mx::few_quant_kernel<Few, 64>;
    const cudaError_t e = launch(kern, dim3((act->M + f.rows - 1) / f.rows * kCluster), 256, f.rows * f.share * 2, kCluster,
                                 st, f);
    if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of few_quant_kernel failed: %s", cudaGetErrorString(e));
    return check_launch("few_quant_kernel (block-scaled FP8)");
  }
  CUtensorMap tmX, tmL1;
  std::memcpy(&tmL1, &w->tmap[2][0], sizeof(CUtensorMap));
  if (svdq_status s = make_tmap(&tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, act->K, act->M,
                                static_cast<uint64_t>(ldx) * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  // K split over a cluster as for the NVFP4 kernel 1 (the same kernel body and resources), in whole blocks, the last
  // CTA's share being what is left
  const int m_tiles = act->M_pad / 128, blocks = act->K_pad / svdq::fp8b::kBlock;
  int csize = 1;
  for (int c = 2; c <= 4; ++c)
    if (m_tiles <= k1_clusters(dev, r, c) && (c - 1) * ((blocks + c - 1) / c) < blocks) csize = c;
  svdq::fp8b::ActArgs a;
  a.inv_lambda = w->inv_lambda;
  a.codes = static_cast<uint8_t*>(act->codes);
  a.sf = static_cast<uint8_t*>(act->scales);
  a.U = static_cast<__nv_bfloat16*>(act->U);
  a.wait_ns = wait_limit_ns();
  a.M = act->M;
  a.K = act->K_pad;
  a.M_pad = act->M_pad;
  a.k_per_cta = (blocks + csize - 1) / csize * svdq::fp8b::kBlock;
  const dim3 grid(m_tiles * csize);
  cudaError_t e;
  if (r == 16)
    e = launch(svdq::quant_act_kernel<16, svdq::fp8b::Act>, grid, svdq::kQ1Threads, svdq::Q1Layout<16>::kSmem, csize, st,
               tmX, tmL1, a);
  else if (r == 32)
    e = launch(svdq::quant_act_kernel<32, svdq::fp8b::Act>, grid, svdq::kQ1Threads, svdq::Q1Layout<32>::kSmem, csize, st,
               tmX, tmL1, a);
  else
    e = launch(svdq::quant_act_kernel<64, svdq::fp8b::Act>, grid, svdq::kQ1Threads, svdq::Q1Layout<64>::kSmem, csize, st,
               tmX, tmL1, a);
  if (e != cudaSuccess)
    return fail(SVDQ_ERR_CUDA, "launch of the block-scaled FP8 quant_act_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("quant_act_kernel (block-scaled FP8)");
}

// svdq_fp8b_gemm on checked arguments.
svdq_status gemm(const svdq_fp8b_act* act, const svdq_fp8b_weight* w, const uint16_t* bias, svdq_epilogue epi, void* Y,
                 long long ldy, svdq_out_dtype out_dtype, svdq_stream_t stream) {
  const bool swiglu = (epi & 2) != 0;
  const int n_out = swiglu ? w->N / 2 : w->N, esize = out_dtype == SVDQ_OUT_F32 ? 4 : 2;
  int dev, sms;
  if (svdq_status s = ready(&dev, &sms); s != SVDQ_OK) return s;
  const int r = w->r;
  if (few_product_rows(act->M, w, swiglu))
    return few_gemm(act, w, bias, (epi & 1) != 0, swiglu, Y, ldy, esize, few_split(w, swiglu, dev),
                    static_cast<cudaStream_t>(stream));
  CUtensorMap tmA, tmU, tmB, tmL2, tmY;
  std::memset(&tmU, 0, sizeof(tmU));
  if (svdq_status s = make_tmap(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, act->codes, act->K_pad, act->M_pad, act->K_pad, 128,
                                128, CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  if (r > 0) {
    if (svdq_status s = make_tmap(&tmU, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, act->U, r, 2 * static_cast<uint64_t>(act->M_pad),
                                  static_cast<uint64_t>(r) * 2, r < 32 ? r : 32, 128, lr_swizzle(r));
        s != SVDQ_OK)
      return s;
  }
  // columns past n_out and rows past M are clipped by the store
  if (svdq_status s = make_tmap(&tmY, esize == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, Y,
                                n_out, act->M, static_cast<uint64_t>(ldy) * esize, 32, 32,
                                esize == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
      s != SVDQ_OK)
    return s;

  svdq::fp8b::GemmArgs g{};
  g.sfa = static_cast<const uint8_t*>(act->scales);
  g.sfb = static_cast<const uint8_t*>(w->scales);
  g.bias = reinterpret_cast<const __nv_bfloat16*>(bias);
  g.wait_ns = wait_limit_ns();
  g.M = act->M;
  g.M_pad = act->M_pad;
  g.N = w->N;
  g.K = w->K_pad;
  g.r = r;
  g.m_tiles = act->M_pad / 128;
  g.m_pairs = (g.m_tiles + 1) / 2;
  g.k_iters = w->K_pad / svdq::fp8b::kBlock;
  g.out_f32 = esize == 4 ? 1 : 0;
  g.epi = static_cast<int>(epi);
  g.n_tile = w->n_tile;
  int tile = w->n_tile, max_pairs = 0;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    const int* most = g_state[dev].max_pairs;
    if (!swiglu) tile = tile_of(g.m_pairs, w, most);
    max_pairs = most[tile == 384 ? 0 : tile == 256 ? 1 : 2];
  }
  g.n_tiles = swiglu ? w->N_pad / 256 : (w->N + tile - 1) / tile;
  const long long tiles = static_cast<long long>(g.m_pairs) * g.n_tiles;
  if (tiles > 0x7FFFFFFFll) return fail(SVDQ_ERR_UNSUPPORTED, "M=%d N=%d: too many tiles", act->M, w->N);
  g.num_tiles = static_cast<int>(tiles);
  std::memcpy(&tmB, &w->tmap[tile == w->n_tile ? 0 : 3][0], sizeof(CUtensorMap));
  std::memcpy(&tmL2, &w->tmap[tile == w->n_tile ? 1 : 4][0], sizeof(CUtensorMap));
  const int pairs = g.num_tiles < max_pairs ? g.num_tiles : max_pairs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto run = [&](auto* kern, int smem) {
    return launch(kern, dim3(2 * pairs), svdq::kGemmThreads, smem, 0, st, tmA, tmB, tmU, tmL2, tmY, g);
  };
  using svdq::fp8b::Gemm, svdq::fp8b::Gemm256Of384;
  const cudaError_t e =
      tile == 384        ? run(svdq::pair_gemm_kernel<Gemm, 384, kStages384>, Layout<384, kStages384>::kSmem)
      : tile == 128      ? run(svdq::pair_gemm_kernel<Gemm, 128, kStages128>, Layout<128, kStages128>::kSmem)
      : w->n_tile == 384 ? run(svdq::pair_gemm_kernel<Gemm256Of384, 256, kStages256>, Layout<256, kStages256>::kSmem)
                         : run(svdq::pair_gemm_kernel<Gemm, 256, kStages256>, Layout<256, kStages256>::kSmem);
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of pair_gemm_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("pair_gemm_kernel (block-scaled FP8)");
}

}  // namespace

svdq_status svdq::host::fp8b_device_status(unsigned* bits, bool reset) {
  SVDQ_CUDA(cudaMemcpyFromSymbol(bits, svdq::g_svdq_status, sizeof(*bits)));
  if (reset) {
    const unsigned z = 0;
    SVDQ_CUDA(cudaMemcpyToSymbol(svdq::g_svdq_status, &z, sizeof(z)));
  }
  return SVDQ_OK;
}

extern "C" {

size_t svdq_fp8b_weight_bytes(int N, int K, int r, int swiglu) {
  if (!n_ok(N, swiglu) || !k_ok(K) || !valid_r(r)) return 0;
  return weight_layout(n_pad(N, swiglu), k_pad(K), r).total;
}

size_t svdq_fp8b_act_bytes(int M, int K, int r) {
  if (M < 1 || M >= (1 << 24) || !k_ok(K) || !valid_r(r)) return 0;
  return act_layout(M, K, r).total;
}

svdq_status svdq_fp8b_act_bind(int M, int K, int r, void* dst, size_t dst_bytes, svdq_fp8b_act* out) {
  if (out == nullptr || dst == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  const size_t need = svdq_fp8b_act_bytes(M, K, r);
  if (need == 0) return fail(SVDQ_ERR_UNSUPPORTED, "block-scaled FP8 act shape M=%d K=%d r=%d unsupported", M, K, r);
  if (dst_bytes < need) return fail(SVDQ_ERR_INVALID_ARG, "block-scaled FP8 act buffer %zu bytes < %zu", dst_bytes, need);
  if (reinterpret_cast<uintptr_t>(dst) % kAlign) return fail(SVDQ_ERR_UNSUPPORTED, "act buffer not 256-byte aligned");
  const ActLayout l = act_layout(M, K, r);
  uint8_t* b = static_cast<uint8_t*>(dst);
  svdq_fp8b_act a{};
  a.M = M;
  a.K = K;
  a.r = r;
  a.M_pad = l.M_pad;
  a.K_pad = l.K_pad;
  a.codes = b + l.codes;
  a.scales = b + l.scales;
  a.U = b + l.u;
  *out = a;
  return SVDQ_OK;
}

svdq_status svdq_fp8b_pack_weight(const float* R_nk, const uint16_t* L1s_kr, const uint16_t* L2_rn,
                                  const float* inv_lambda, int N, int K, int r, int swiglu, void* dst, size_t dst_bytes,
                                  svdq_fp8b_weight* out, svdq_stream_t stream) {
  if (out == nullptr || R_nk == nullptr || dst == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (r > 0 && (L1s_kr == nullptr || L2_rn == nullptr)) return fail(SVDQ_ERR_INVALID_ARG, "null L1s / L2 with r > 0");
  const size_t need = svdq_fp8b_weight_bytes(N, K, r, swiglu);
  if (need == 0) return fail(SVDQ_ERR_UNSUPPORTED, "block-scaled FP8 weight shape N=%d K=%d r=%d unsupported", N, K, r);
  if (!aligned16(R_nk) || (r > 0 && (!aligned16(L1s_kr) || !aligned16(L2_rn))) ||
      (reinterpret_cast<uintptr_t>(inv_lambda) & 3u))
    return fail(SVDQ_ERR_UNSUPPORTED, "inputs must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(dst) % kAlign) return fail(SVDQ_ERR_UNSUPPORTED, "dst not 256-byte aligned");
  if (dst_bytes < need)
    return fail(SVDQ_ERR_INVALID_ARG, "block-scaled FP8 weight buffer %zu bytes < %zu", dst_bytes, need);
  int dev, sms;
  if (svdq_status s = ready(&dev, &sms); s != SVDQ_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  svdq_fp8b_weight w{};
  if (svdq_status s = fill_weight(static_cast<uint8_t*>(dst), N, K, r, swiglu, &w); s != SVDQ_OK) return s;
  SVDQ_CUDA(cudaMemsetAsync(dst, 0, need, st));  // padded rows and columns
  svdq::mx::fill_inv_lambda_kernel<><<<grid_for(w.K_pad, 256, sms), 256, 0, st>>>(inv_lambda, K, w.K_pad, w.inv_lambda);
  if (svdq_status s = check_launch("mx::fill_inv_lambda_kernel"); s != SVDQ_OK) return s;
  const unsigned blocks = static_cast<unsigned>((N + 127) / 128) * (w.K_pad / svdq::fp8b::kBlock);
  svdq::fp8b::pack_quant_kernel<><<<blocks, 256, 0, st>>>(R_nk, N, K, w.K_pad, w.n_tile, w.swiglu_interleaved,
                                                       static_cast<uint8_t*>(w.codes), static_cast<uint8_t*>(w.scales));
  if (svdq_status s = check_launch("fp8b::pack_quant_kernel"); s != SVDQ_OK) return s;
  if (r > 0) {
    svdq::mx::transpose_l1_kernel<><<<grid_for(static_cast<size_t>(w.K_pad) * r, 256, sms), 256, 0, st>>>(
        reinterpret_cast<const __nv_bfloat16*>(L1s_kr), K, w.K_pad, r, static_cast<__nv_bfloat16*>(w.L1s_t));
    if (svdq_status s = check_launch("mx::transpose_l1_kernel"); s != SVDQ_OK) return s;
    svdq::mx::pack_l2_kernel<><<<grid_for(static_cast<size_t>(N) * r, 256, sms), 256, 0, st>>>(
        reinterpret_cast<const __nv_bfloat16*>(L2_rn), N, r, w.n_tile, w.swiglu_interleaved,
        static_cast<__nv_bfloat16*>(w.L2_t));
    if (svdq_status s = check_launch("mx::pack_l2_kernel"); s != SVDQ_OK) return s;
  }
  *out = w;
  return SVDQ_OK;
}

svdq_status svdq_fp8b_weight_bind(int N, int K, int r, int swiglu, void* blob, size_t blob_bytes, svdq_fp8b_weight* out) {
  if (out == nullptr || blob == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  const size_t need = svdq_fp8b_weight_bytes(N, K, r, swiglu);
  if (need == 0) return fail(SVDQ_ERR_UNSUPPORTED, "block-scaled FP8 weight shape N=%d K=%d r=%d unsupported", N, K, r);
  if (reinterpret_cast<uintptr_t>(blob) % kAlign) return fail(SVDQ_ERR_UNSUPPORTED, "blob not 256-byte aligned");
  if (blob_bytes < need)
    return fail(SVDQ_ERR_INVALID_ARG, "block-scaled FP8 weight blob %zu bytes < %zu", blob_bytes, need);
  if (svdq_status s = ready(nullptr, nullptr); s != SVDQ_OK) return s;
  return fill_weight(static_cast<uint8_t*>(blob), N, K, r, swiglu, out);
}

svdq_status svdq_fp8b_quantize_act(const uint16_t* X, long long ldx, const svdq_fp8b_weight* w,
                                   const svdq_fp8b_act* act, svdq_stream_t stream) {
  if (svdq_status s = check_quantize(X, ldx, w, act); s != SVDQ_OK) return s;
  return quantize(X, ldx, w, act, stream);
}

svdq_status svdq_fp8b_gemm(const svdq_fp8b_act* act, const svdq_fp8b_weight* w, const uint16_t* bias, svdq_epilogue epi,
                           void* Y, long long ldy, svdq_out_dtype out_dtype, svdq_stream_t stream) {
  if (svdq_status s = check_gemm(act, w, bias, epi, Y, ldy, out_dtype); s != SVDQ_OK) return s;
  return gemm(act, w, bias, epi, Y, ldy, out_dtype, stream);
}

svdq_status svdq_fp8b_linear(const uint16_t* X, long long ldx, const svdq_fp8b_weight* w, const svdq_fp8b_act* act,
                             const uint16_t* bias, svdq_epilogue epi, void* Y, long long ldy, svdq_out_dtype out_dtype,
                             svdq_stream_t stream) {
  if (svdq_status s = check_quantize(X, ldx, w, act); s != SVDQ_OK) return s;
  if (svdq_status s = check_gemm(act, w, bias, epi, Y, ldy, out_dtype); s != SVDQ_OK) return s;
  if (svdq_status s = quantize(X, ldx, w, act, stream); s != SVDQ_OK) return s;
  return gemm(act, w, bias, epi, Y, ldy, out_dtype, stream);
}

svdq_status svdq_fp8b_export_weight(const svdq_fp8b_weight* w, uint8_t* codes, uint8_t* scales, svdq_stream_t stream) {
  if (w == nullptr || codes == nullptr || scales == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_weight(w); s != SVDQ_OK) return s;
  if (reinterpret_cast<uintptr_t>(codes) & 7u) return fail(SVDQ_ERR_UNSUPPORTED, "codes must be 8-byte aligned");
  int dev, sms;
  if (svdq_status s = ready(&dev, &sms); s != SVDQ_OK) return s;
  svdq::fp8b::export_kernel<><<<grid_for(static_cast<size_t>(w->N) * (w->K / 8), 256, sms), 256, 0,
                              static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(w->codes), static_cast<const uint8_t*>(w->scales), w->N, w->K, w->K_pad, w->n_tile,
      w->swiglu_interleaved, codes, scales);
  return check_launch("fp8b::export_kernel");
}

svdq_status svdq_fp8b_export_act(const svdq_fp8b_act* act, uint8_t* codes, uint8_t* scales, svdq_stream_t stream) {
  if (act == nullptr || codes == nullptr || scales == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_act(act); s != SVDQ_OK) return s;
  if (reinterpret_cast<uintptr_t>(codes) & 7u) return fail(SVDQ_ERR_UNSUPPORTED, "codes must be 8-byte aligned");
  int dev, sms;
  if (svdq_status s = ready(&dev, &sms); s != SVDQ_OK) return s;
  svdq::fp8b::export_kernel<><<<grid_for(static_cast<size_t>(act->M) * (act->K / 8), 256, sms), 256, 0,
                              static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(act->codes), static_cast<const uint8_t*>(act->scales), act->M, act->K, act->K_pad, 0, 0,
      codes, scales);
  return check_launch("fp8b::export_kernel");
}

svdq_status svdq_fp8b_dequantize_act(const svdq_fp8b_act* act, void* out, long long ld, svdq_out_dtype out_dtype,
                                     svdq_stream_t stream) {
  if (act == nullptr || out == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_act(act); s != SVDQ_OK) return s;
  if (out_dtype != SVDQ_OUT_BF16 && out_dtype != SVDQ_OUT_F32) return fail(SVDQ_ERR_INVALID_ARG, "bad out dtype");
  if (!aligned16(out)) return fail(SVDQ_ERR_UNSUPPORTED, "out must be 16-byte aligned");
  if (ld < act->K || ld % 8 != 0)
    return fail(SVDQ_ERR_UNSUPPORTED, "row stride %lld of out: a multiple of 8 and at least K=%d", ld, act->K);
  int dev, sms;
  if (svdq_status s = ready(&dev, &sms); s != SVDQ_OK) return s;
  const dim3 grid((act->M + svdq::fp8b::kDeqRows - 1) / svdq::fp8b::kDeqRows, (act->K / 8 + 255) / 256);
  const cudaError_t e = launch(
      out_dtype == SVDQ_OUT_F32 ? svdq::fp8b::dequantize_act_kernel<true> : svdq::fp8b::dequantize_act_kernel<false>, grid,
      256, 0, 0, static_cast<cudaStream_t>(stream), static_cast<const uint8_t*>(act->codes),
      static_cast<const uint8_t*>(act->scales), act->M, act->K, act->K_pad, out, ld);
  if (e != cudaSuccess)
    return fail(SVDQ_ERR_CUDA, "launch of fp8b::dequantize_act_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("fp8b::dequantize_act_kernel");
}

}  // extern "C"
