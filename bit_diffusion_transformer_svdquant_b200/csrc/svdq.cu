// C ABI of the sm_100a W4A4 + low-rank linear layer (declared in include/svdq.h): argument checks,
// buffer layouts, TMA descriptor construction and kernel launches. One translation unit.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdlib>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <utility>
#include <string>

#include "svdq.h"
#include "svdq_fp8r.cuh"
#include "svdq_fused.cuh"
#include "svdq_gemm.cuh"
#include "svdq_mx.cuh"
#include "svdq_mx_few.cuh"
#include "svdq_norm.cuh"
#include "svdq_ptx.cuh"
#include "svdq_quant.cuh"

namespace {

thread_local std::string g_last_error;
std::atomic<unsigned long long> g_wait_ns{2000000000ull};

svdq_status fail(svdq_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
svdq_status fail(svdq_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

#define SVDQ_CUDA(call)                                                                         \
  do {                                                                                          \
    cudaError_t e_ = (call);                                                                    \
    if (e_ != cudaSuccess) return fail(SVDQ_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_)); \
  } while (0)

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// ------------------------------------------------------------------ per-device state
struct DeviceState {
  bool ready = false;
  int sm_count = 0;
  int max_pairs[4] = {0, 0, 0, 0};  // co-resident CTA pairs of the GEMM kernel for n_tile 256, 192, 128, 384
  int k1_clusters[4][4] = {};     // co-resident kernel-1 clusters, by r (0/16/32/64) and size - 1 (1..4)
  svdq_status status = SVDQ_OK;
  std::string error;
};
std::mutex g_dev_mu;
DeviceState g_dev[64];

constexpr int kStagesTile256 = 5;
constexpr int kStagesTile192 = 5;
constexpr int kStagesTile128 = 6;
constexpr int kStagesTile384 = 4;

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                            const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                            CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode g_encode = nullptr;

svdq_status device_ready(int* dev_out, int* sm_out) {
  int dev = 0;
  SVDQ_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return fail(SVDQ_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceState& st = g_dev[dev];
  if (!st.ready) {
    int major = 0, minor = 0, sms = 0;
    SVDQ_CUDA(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev));
    SVDQ_CUDA(cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev));
    SVDQ_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    if (major != 10 || minor != 0)
      return fail(SVDQ_ERR_UNSUPPORTED, "device %d is sm_%d%d; this library is built for sm_100a only", dev, major,
                  minor);
    if (g_encode == nullptr) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      SVDQ_CUDA(cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q));
      if (fn == nullptr || q != cudaDriverEntryPointSuccess)
        return fail(SVDQ_ERR_CUDA, "cuTensorMapEncodeTiled not available from the driver");
      g_encode = reinterpret_cast<Encode>(fn);
    }
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::pair_gemm_kernel<svdq::Nvfp4Gemm, 256, kStagesTile256>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   svdq::GemmLayout<256, kStagesTile256>::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::pair_gemm_kernel<svdq::Nvfp4Gemm, 192, kStagesTile192>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   svdq::GemmLayout<192, kStagesTile192>::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::pair_gemm_kernel<svdq::Nvfp4Gemm, 128, kStagesTile128>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   svdq::GemmLayout<128, kStagesTile128>::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::pair_gemm_kernel<svdq::Nvfp4Gemm, 384, kStagesTile384>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   svdq::GemmLayout<384, kStagesTile384>::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::quant_act_kernel<0, svdq::Nvfp4Act>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   svdq::Q1Layout<0>::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::quant_act_kernel<16, svdq::Nvfp4Act>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   svdq::Q1Layout<16>::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::quant_act_kernel<32, svdq::Nvfp4Act>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   svdq::Q1Layout<32>::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::quant_act_kernel<64, svdq::Nvfp4Act>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   svdq::Q1Layout<64>::kSmem));
    // How many CTA pairs of each GEMM instantiation can be resident at once: the persistent grid
    // never asks for more (pairs must sit on two SMs of one GPC, so this can be below sms / 2).
    auto max_pairs = [&](const void* fn, int smem, int* out) -> svdq_status {
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(2 * (sms / 2), 1, 1);
      cfg.blockDim = dim3(svdq::kGemmThreads, 1, 1);
      cfg.dynamicSmemBytes = static_cast<size_t>(smem);
      int n = 0;
      SVDQ_CUDA(cudaOccupancyMaxActiveClusters(&n, fn, &cfg));
      if (n <= 0) return fail(SVDQ_ERR_CUDA, "GEMM kernel cannot be resident as CTA pairs");
      *out = n;
      return SVDQ_OK;
    };
    if (svdq_status s = max_pairs(reinterpret_cast<const void*>(svdq::pair_gemm_kernel<svdq::Nvfp4Gemm, 256, kStagesTile256>),
                                  svdq::GemmLayout<256, kStagesTile256>::kSmem, &st.max_pairs[0]);
        s != SVDQ_OK)
      return s;
    if (svdq_status s = max_pairs(reinterpret_cast<const void*>(svdq::pair_gemm_kernel<svdq::Nvfp4Gemm, 192, kStagesTile192>),
                                  svdq::GemmLayout<192, kStagesTile192>::kSmem, &st.max_pairs[1]);
        s != SVDQ_OK)
      return s;
    if (svdq_status s = max_pairs(reinterpret_cast<const void*>(svdq::pair_gemm_kernel<svdq::Nvfp4Gemm, 128, kStagesTile128>),
                                  svdq::GemmLayout<128, kStagesTile128>::kSmem, &st.max_pairs[2]);
        s != SVDQ_OK)
      return s;
    if (svdq_status s = max_pairs(reinterpret_cast<const void*>(svdq::pair_gemm_kernel<svdq::Nvfp4Gemm, 384, kStagesTile384>),
                                  svdq::GemmLayout<384, kStagesTile384>::kSmem, &st.max_pairs[3]);
        s != SVDQ_OK)
      return s;
    // how many kernel-1 clusters of 1, 2, 3 and 4 CTAs (one CTA per SM) can be resident at once
    // (a cluster's CTAs share a GPC, so fewer 4-clusters than sms / 4 may fit)
    auto k1_clusters = [&](const void* fn, int smem, int* out) -> svdq_status {
      for (int ci = 0; ci < 4; ++ci) {
        const int c = ci + 1;
        cudaLaunchConfig_t cfg{};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = c;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3(c * (sms / c), 1, 1);
        cfg.blockDim = dim3(svdq::kQ1Threads, 1, 1);
        cfg.dynamicSmemBytes = static_cast<size_t>(smem);
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        SVDQ_CUDA(cudaOccupancyMaxActiveClusters(&n, fn, &cfg));
        out[ci] = n;
      }
      return SVDQ_OK;
    };
    if (svdq_status s = k1_clusters(reinterpret_cast<const void*>(svdq::quant_act_kernel<0, svdq::Nvfp4Act>), svdq::Q1Layout<0>::kSmem,
                                    st.k1_clusters[0]);
        s != SVDQ_OK)
      return s;
    if (svdq_status s = k1_clusters(reinterpret_cast<const void*>(svdq::quant_act_kernel<16, svdq::Nvfp4Act>),
                                    svdq::Q1Layout<16>::kSmem, st.k1_clusters[1]);
        s != SVDQ_OK)
      return s;
    if (svdq_status s = k1_clusters(reinterpret_cast<const void*>(svdq::quant_act_kernel<32, svdq::Nvfp4Act>),
                                    svdq::Q1Layout<32>::kSmem, st.k1_clusters[2]);
        s != SVDQ_OK)
      return s;
    if (svdq_status s = k1_clusters(reinterpret_cast<const void*>(svdq::quant_act_kernel<64, svdq::Nvfp4Act>),
                                    svdq::Q1Layout<64>::kSmem, st.k1_clusters[3]);
        s != SVDQ_OK)
      return s;
    st.sm_count = sms;
    st.ready = true;
  }
  if (dev_out) *dev_out = dev;
  if (sm_out) *sm_out = st.sm_count;
  return SVDQ_OK;
}

svdq_status make_tmap(CUtensorMap* m, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t outer,
                      uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swz) {
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {box_inner, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  CUresult r = g_encode(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(SVDQ_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return SVDQ_OK;
}

// The low-rank operands travel in chunks of at most 32 columns of r (one ring slot each).
CUtensorMapSwizzle lr_swizzle(int r) { return r == 16 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B; }

bool valid_r(int r) { return r == 0 || r == 16 || r == 32 || r == 64; }

// The 384-wide NVFP4 tile (two pair MMAs per K chunk): a weight without the SwiGLU interleave whose
// N is a multiple of 768, so that its blob has the same size as at 256 (N / 128 scale atoms per K
// atom either way) and svdq_weight_bytes need not know whether a weight is SwiGLU.
bool wide_tile_ok(int N, int swiglu) { return !swiglu && N % 768 == 0; }

// GEMM tile width along N: the widest that divides N, for the fewest operand bytes streamed per
// flop: 384 (where wide_tile_ok and `wide`: the NVFP4 GEMM), else 256, 192, 128. SVDQ_N_TILE
// overrides it with another valid width.
int choose_n_tile(int N, int swiglu, bool wide) {
  const char* env = getenv("SVDQ_N_TILE");
  if (env != nullptr) {
    const int t = atoi(env);
    if ((t == 256 || t == 192 || t == 128) && N % t == 0) return t;
    if (t == 384 && wide && wide_tile_ok(N, swiglu)) return t;
  }
  if (wide && wide_tile_ok(N, swiglu)) return 384;
  if (N % 256 == 0) return 256;
  if (N % 192 == 0) return 192;
  if (N % 128 == 0) return 128;
  return 0;
}
// A GEMM tile width a descriptor of an NVFP4 weight may hold.
bool valid_n_tile(int N, int n_tile, int swiglu) {
  if (n_tile == 384) return wide_tile_ok(N, swiglu);
  return (n_tile == 256 || n_tile == 192 || n_tile == 128) && N % n_tile == 0;
}

struct WeightLayout {
  size_t codes, scales, gw, inv_lambda, l1t, l2t, total;
};
WeightLayout weight_layout(int N, int K, int r, int n_tile) {
  WeightLayout l{};
  size_t off = 0;
  l.codes = off;
  off = align_up(off + static_cast<size_t>(N) * K / 2);
  l.scales = off;
  off = align_up(off + static_cast<size_t>(N / n_tile) * (K / 64) * ((n_tile + 127) / 128) * 512);
  l.gw = off;
  off = align_up(off + 4);
  l.inv_lambda = off;
  off = align_up(off + static_cast<size_t>(K) * 4);
  l.l1t = off;
  off = align_up(off + static_cast<size_t>(r) * K * 2);
  l.l2t = off;
  off = align_up(off + static_cast<size_t>(N) * r * 2);
  l.total = off;
  return l;
}

struct ActLayout {
  size_t codes, scales, u, alpha, total;
  int M_pad;
};
ActLayout act_layout(int M, int K, int r) {
  ActLayout l{};
  l.M_pad = (M + 127) / 128 * 128;
  size_t off = 0;
  l.codes = off;
  off = align_up(off + static_cast<size_t>(l.M_pad) * K / 2);
  l.scales = off;
  off = align_up(off + static_cast<size_t>(l.M_pad / 128) * (K / 64) * 512);
  l.u = off;
  off = align_up(off + static_cast<size_t>(l.M_pad) * r * 2 * 2);  // hi and lo halves
  l.alpha = off;
  off = align_up(off + 4);
  l.total = off;
  return l;
}

bool shape_ok(int N, int K, int r) {
  return N > 0 && K > 0 && K % 256 == 0 && valid_r(r) && K <= (1 << 20) && N <= (1 << 20) &&
         choose_n_tile(N, 0, false) > 0;
}

// The descriptors are plain structs that a caller may also fill by hand: before a launch reads
// through them, check that they describe a layout that svdq_pack_weight / svdq_act_bind can produce.
svdq_status check_weight(const svdq_weight* w) {
  const int t = w->n_tile;
  if (w->N <= 0 || !valid_n_tile(w->N, t, w->swiglu_interleaved) || w->N > (1 << 20) || w->K <= 0 ||
      w->K % 256 != 0 || w->K > (1 << 20) || !valid_r(w->r))
    return fail(SVDQ_ERR_INVALID_ARG, "weight descriptor N=%d K=%d r=%d n_tile=%d is not one svdq_pack_weight makes",
                w->N, w->K, w->r, t);
  if (w->codes == nullptr || w->scales == nullptr || w->g_w == nullptr || w->inv_lambda == nullptr ||
      (w->r > 0 && (w->L1s_t == nullptr || w->L2_t == nullptr)))
    return fail(SVDQ_ERR_INVALID_ARG, "weight descriptor has a null buffer");
  return SVDQ_OK;
}

svdq_status check_act(const svdq_act* a) {
  if (a->M < 1 || a->M >= (1 << 24) || a->K <= 0 || a->K % 256 != 0 || a->K > (1 << 20) || !valid_r(a->r) ||
      a->M_pad != (a->M + 127) / 128 * 128)
    return fail(SVDQ_ERR_INVALID_ARG, "act descriptor M=%d M_pad=%d K=%d r=%d is not one svdq_act_bind makes", a->M,
                a->M_pad, a->K, a->r);
  if (a->codes == nullptr || a->scales == nullptr || a->alpha == nullptr || (a->r > 0 && a->U == nullptr))
    return fail(SVDQ_ERR_INVALID_ARG, "act descriptor has a null buffer");
  return SVDQ_OK;
}

// Descriptor of a packed weight blob at `b`: the pointers of weight_layout(N, K, r, n_tile) and
// the TMA descriptors of its codes and L2^T, which hold absolute addresses and so are encoded for
// this copy of the blob. svdq_pack_weight and svdq_weight_bind both fill descriptors here.
svdq_status fill_weight_desc(uint8_t* b, int N, int K, int r, int swiglu, int n_tile, svdq_weight* out) {
  const WeightLayout l = weight_layout(N, K, r, n_tile);
  svdq_weight w{};
  w.N = N;
  w.K = K;
  w.r = r;
  w.swiglu_interleaved = swiglu ? 1 : 0;
  w.n_tile = n_tile;
  w.codes = b + l.codes;
  w.scales = b + l.scales;
  w.g_w = reinterpret_cast<float*>(b + l.gw);
  w.inv_lambda = reinterpret_cast<float*>(b + l.inv_lambda);
  w.L1s_t = b + l.l1t;
  w.L2_t = b + l.l2t;
  static_assert(sizeof(w.tmap) >= 2 * sizeof(CUtensorMap), "tmap storage");
  CUtensorMap tmB, tmL2;
  std::memset(&tmL2, 0, sizeof(tmL2));
  // each CTA of a GEMM pair stages half of a tile's n_tile rows
  if (svdq_status s = make_tmap(&tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, K / 2, N, K / 2, 128, n_tile / 2,
                                CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  if (r > 0) {
    if (svdq_status s = make_tmap(&tmL2, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w.L2_t, r, N, static_cast<uint64_t>(r) * 2,
                                  r < 32 ? r : 32, n_tile / 2, lr_swizzle(r));
        s != SVDQ_OK)
      return s;
  }
  std::memcpy(&w.tmap[0][0], &tmB, sizeof(CUtensorMap));
  std::memcpy(&w.tmap[1][0], &tmL2, sizeof(CUtensorMap));
  *out = w;
  return SVDQ_OK;
}

int grid_for(size_t work_items, int per_block, int sm_count) {
  size_t blocks = (work_items + per_block - 1) / per_block;
  size_t cap = static_cast<size_t>(sm_count) * 16;
  if (blocks > cap) blocks = cap;
  if (blocks < 1) blocks = 1;
  return static_cast<int>(blocks);
}

svdq_status check_launch(const char* what) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of %s failed: %s", what, cudaGetErrorString(e));
  return SVDQ_OK;
}

// Both kernels of a layer are launched with programmatic stream serialization: a kernel may be
// scheduled while the previous kernel on the stream is finishing, so its barrier and TMEM set-up
// overlap that kernel's tail; its first global access waits for that grid (griddepcontrol.wait).
void set_programmatic(cudaLaunchAttribute& a) {
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
}

// The pair GEMMs: clusters of 2 CTAs are compiled into the kernel, so the one launch attribute is
// the programmatic one.
template <typename... P, typename... A>
cudaError_t launch_pair_gemm(void (*kern)(P...), int ctas, int smem, cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  set_programmatic(attr[0]);
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(svdq::kGemmThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<A>(args)...);
}

}  // namespace

extern "C" {

int svdq_abi_version(void) { return SVDQ_ABI_VERSION; }

const char* svdq_status_str(svdq_status s) {
  switch (s) {
    case SVDQ_OK: return "ok";
    case SVDQ_ERR_INVALID_ARG: return "invalid argument";
    case SVDQ_ERR_UNSUPPORTED: return "unsupported shape, alignment or device";
    case SVDQ_ERR_CUDA: return "CUDA error";
    case SVDQ_ERR_TIMEOUT: return "device-side wait timed out";
  }
  return "unknown status";
}

const char* svdq_last_error(void) { return g_last_error.c_str(); }

size_t svdq_weight_bytes(int N, int K, int r) {
  if (!shape_ok(N, K, r)) return 0;
  return weight_layout(N, K, r, choose_n_tile(N, 0, true)).total;
}

size_t svdq_weight_bytes_tiled(int N, int K, int r, int n_tile) {
  if (N <= 0 || K <= 0 || K % 256 != 0 || K > (1 << 20) || N > (1 << 20) || !valid_r(r) ||
      !valid_n_tile(N, n_tile, 0))
    return 0;
  return weight_layout(N, K, r, n_tile).total;
}

size_t svdq_act_bytes(int M, int K, int r) {
  if (M < 1 || M >= (1 << 24) || K <= 0 || K % 256 != 0 || !valid_r(r)) return 0;
  return act_layout(M, K, r).total;
}

svdq_status svdq_set_wait_limit_ns(unsigned long long ns) {
  if (ns < 1000000ull || ns > 60000000000ull) return fail(SVDQ_ERR_INVALID_ARG, "wait limit %llu ns out of range", ns);
  g_wait_ns.store(ns);
  return SVDQ_OK;
}

svdq_status svdq_act_bind(int M, int K, int r, void* dst, size_t dst_bytes, svdq_act* out) {
  if (out == nullptr || dst == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  const size_t need = svdq_act_bytes(M, K, r);
  if (need == 0) return fail(SVDQ_ERR_UNSUPPORTED, "act shape M=%d K=%d r=%d unsupported", M, K, r);
  if (dst_bytes < need) return fail(SVDQ_ERR_INVALID_ARG, "act buffer %zu bytes < %zu", dst_bytes, need);
  if (reinterpret_cast<uintptr_t>(dst) % kAlign) return fail(SVDQ_ERR_UNSUPPORTED, "act buffer not 256-byte aligned");
  const ActLayout l = act_layout(M, K, r);
  uint8_t* b = static_cast<uint8_t*>(dst);
  out->M = M;
  out->K = K;
  out->r = r;
  out->M_pad = l.M_pad;
  out->codes = b + l.codes;
  out->scales = b + l.scales;
  out->U = b + l.u;
  out->alpha = reinterpret_cast<float*>(b + l.alpha);
  return SVDQ_OK;
}

svdq_status svdq_pack_weight(const float* R_nk, const uint16_t* L1s_kr, const uint16_t* L2_rn,
                             const float* inv_lambda, int N, int K, int r, int swiglu, void* dst, size_t dst_bytes,
                             svdq_weight* out, svdq_stream_t stream) {
  if (out == nullptr || R_nk == nullptr || inv_lambda == nullptr || dst == nullptr)
    return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (r > 0 && (L1s_kr == nullptr || L2_rn == nullptr)) return fail(SVDQ_ERR_INVALID_ARG, "null L1s / L2 with r > 0");
  if (!shape_ok(N, K, r)) return fail(SVDQ_ERR_UNSUPPORTED, "weight shape N=%d K=%d r=%d unsupported", N, K, r);
  if (swiglu && (N % 2 != 0)) return fail(SVDQ_ERR_UNSUPPORTED, "SwiGLU needs N even");
  if (!aligned16(R_nk) || !aligned16(inv_lambda) || (r > 0 && (!aligned16(L1s_kr) || !aligned16(L2_rn))))
    return fail(SVDQ_ERR_UNSUPPORTED, "inputs must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(dst) % kAlign) return fail(SVDQ_ERR_UNSUPPORTED, "dst not 256-byte aligned");
  const int n_tile = choose_n_tile(N, swiglu, true);
  const WeightLayout l = weight_layout(N, K, r, n_tile);
  if (dst_bytes < l.total) return fail(SVDQ_ERR_INVALID_ARG, "weight buffer %zu bytes < %zu", dst_bytes, l.total);
  int dev, sms;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* b = static_cast<uint8_t*>(dst);

  svdq_weight w{};
  if (svdq_status s = fill_weight_desc(b, N, K, r, swiglu, n_tile, &w); s != SVDQ_OK) return s;

  SVDQ_CUDA(cudaMemsetAsync(b + l.scales, 0, l.gw - l.scales + 4, st));  // pad rows of the scale layout, amax
  SVDQ_CUDA(cudaMemcpyAsync(w.inv_lambda, inv_lambda, static_cast<size_t>(K) * 4, cudaMemcpyDeviceToDevice, st));
  const size_t n4 = static_cast<size_t>(N) * K / 4;
  svdq::amax_f32_kernel<<<grid_for(n4, 256, sms), 256, 0, st>>>(R_nk, n4, reinterpret_cast<unsigned*>(w.g_w));
  if (svdq_status s = check_launch("amax_f32_kernel"); s != SVDQ_OK) return s;
  svdq::finalize_scale_kernel<<<1, 1, 0, st>>>(w.g_w);
  if (svdq_status s = check_launch("finalize_scale_kernel"); s != SVDQ_OK) return s;
  const size_t halves = static_cast<size_t>(N) * K / 8;
  svdq::pack_quant_kernel<<<grid_for(halves, 256, sms), 256, 0, st>>>(
      R_nk, N, K, n_tile, w.swiglu_interleaved, w.g_w, static_cast<uint8_t*>(w.codes), static_cast<uint8_t*>(w.scales));
  if (svdq_status s = check_launch("pack_quant_kernel"); s != SVDQ_OK) return s;
  if (r > 0) {
    svdq::transpose_l1_kernel<<<grid_for(static_cast<size_t>(K) * r, 256, sms), 256, 0, st>>>(
        reinterpret_cast<const __nv_bfloat16*>(L1s_kr), K, r, static_cast<__nv_bfloat16*>(w.L1s_t));
    if (svdq_status s = check_launch("transpose_l1_kernel"); s != SVDQ_OK) return s;
    svdq::pack_l2_kernel<<<grid_for(static_cast<size_t>(N) * r, 256, sms), 256, 0, st>>>(
        reinterpret_cast<const __nv_bfloat16*>(L2_rn), N, r, n_tile, w.swiglu_interleaved,
        static_cast<__nv_bfloat16*>(w.L2_t));
    if (svdq_status s = check_launch("pack_l2_kernel"); s != SVDQ_OK) return s;
  }
  *out = w;
  return SVDQ_OK;
}

svdq_status svdq_weight_bind(int N, int K, int r, int swiglu, int n_tile, void* blob, size_t blob_bytes,
                             svdq_weight* out) {
  if (out == nullptr || blob == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (N <= 0 || K <= 0 || K % 256 != 0 || K > (1 << 20) || N > (1 << 20) || !valid_r(r) ||
      !valid_n_tile(N, n_tile, swiglu))
    return fail(SVDQ_ERR_UNSUPPORTED, "weight shape N=%d K=%d r=%d n_tile=%d swiglu=%d unsupported", N, K, r, n_tile,
                swiglu);
  if (reinterpret_cast<uintptr_t>(blob) % kAlign) return fail(SVDQ_ERR_UNSUPPORTED, "blob not 256-byte aligned");
  const WeightLayout l = weight_layout(N, K, r, n_tile);
  if (blob_bytes < l.total) return fail(SVDQ_ERR_INVALID_ARG, "weight blob %zu bytes < %zu", blob_bytes, l.total);
  int dev, sms;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;
  // the TMA descriptors hold absolute addresses: they are encoded for this copy of the blob
  return fill_weight_desc(static_cast<uint8_t*>(blob), N, K, r, swiglu, n_tile, out);
}

svdq_status svdq_calibrate_act(const uint16_t* X, int M, const svdq_weight* w, float* g_x_out, svdq_stream_t stream) {
  if (X == nullptr || w == nullptr || g_x_out == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_weight(w); s != SVDQ_OK) return s;
  if (M < 1 || M >= (1 << 24)) return fail(SVDQ_ERR_UNSUPPORTED, "M=%d unsupported", M);
  if (!aligned16(X)) return fail(SVDQ_ERR_UNSUPPORTED, "X must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(g_x_out) & 3u) return fail(SVDQ_ERR_UNSUPPORTED, "g_x_out must be 4-byte aligned");
  int dev, sms;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  SVDQ_CUDA(cudaMemsetAsync(g_x_out, 0, 4, st));
  // 128 column chunks of 8 per block along x; rows split over y so that ~16 blocks land per SM
  const int per_row = w->K / 8;
  const int gx = (per_row + 127) / 128;
  int gy = sms * 16 / gx;
  if (gy > M) gy = M;
  if (gy > 65535) gy = 65535;
  if (gy < 1) gy = 1;
  svdq::act_amax_kernel<<<dim3(gx, gy), 128, 0, st>>>(reinterpret_cast<const __nv_bfloat16*>(X), w->inv_lambda,
                                                      M, w->K, reinterpret_cast<unsigned*>(g_x_out));
  if (svdq_status s = check_launch("act_amax_kernel"); s != SVDQ_OK) return s;
  svdq::finalize_scale_kernel<<<1, 1, 0, st>>>(g_x_out);
  return check_launch("finalize_scale_kernel");
}

svdq_status svdq_quantize_act(const uint16_t* X, const svdq_weight* w, const float* g_x, const svdq_act* act,
                              svdq_stream_t stream) {
  if (X == nullptr || w == nullptr || g_x == nullptr || act == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (act->K != w->K || act->r != w->r)
    return fail(SVDQ_ERR_INVALID_ARG, "act (K=%d r=%d) does not match weight (K=%d r=%d)", act->K, act->r, w->K, w->r);
  if (svdq_status s = check_weight(w); s != SVDQ_OK) return s;
  if (svdq_status s = check_act(act); s != SVDQ_OK) return s;
  if (!aligned16(X)) return fail(SVDQ_ERR_UNSUPPORTED, "X must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(g_x) & 3u) return fail(SVDQ_ERR_UNSUPPORTED, "g_x must be 4-byte aligned");
  int dev, sms;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;
  const int K = act->K, r = w->r, M = act->M;
  CUtensorMap tmX, tmL1;
  std::memset(&tmL1, 0, sizeof(tmL1));
  if (svdq_status s = make_tmap(&tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, K, M, static_cast<uint64_t>(K) * 2, 64, 128,
                                CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  if (r > 0) {
    if (svdq_status s = make_tmap(&tmL1, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w->L1s_t, K, r,
                                  static_cast<uint64_t>(K) * 2, 64, r, CU_TENSOR_MAP_SWIZZLE_128B);
        s != SVDQ_OK)
      return s;
  }
  // One CTA per SM; K is split across the largest cluster of 2, 3 or 4 CTAs whose clusters for all
  // row tiles are resident at once (cudaOccupancyMaxActiveClusters: clusters must fit inside GPCs),
  // so small M fills more SMs and nothing runs as a second wave. Measured on B200 at M = 4608 (36 row
  // tiles): only 32 clusters of 4 are resident, and at K = 12288 3-CTA clusters (108 CTAs) take
  // 47 us against 57 us for 2-CTA ones (72 CTAs). SVDQ_K1_CLUSTER overrides the size; every CTA
  // keeps whole 64-column K steps.
  const int m_tiles = act->M_pad / 128;
  int csize = 1;
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    const int* mc = g_dev[dev].k1_clusters[r == 0 ? 0 : r == 16 ? 1 : r == 32 ? 2 : 3];
    for (int c = 2; c <= 4; ++c)
      if (m_tiles <= mc[c - 1] && K % (64 * c) == 0) csize = c;
  }
  if (const char* env = getenv("SVDQ_K1_CLUSTER"); env != nullptr) {
    const int c = atoi(env);
    if (c >= 1 && c <= 4 && K % (64 * c) == 0) csize = c;
  }
  svdq::QuantActArgs a;
  a.inv_lambda = w->inv_lambda;
  a.g_x = g_x;
  a.g_w = w->g_w;
  a.codes = static_cast<uint8_t*>(act->codes);
  a.sf = static_cast<uint8_t*>(act->scales);
  a.U = static_cast<__nv_bfloat16*>(act->U);
  a.alpha = act->alpha;
  a.wait_ns = g_wait_ns.load();
  a.M = M;
  a.K = K;
  a.M_pad = act->M_pad;
  a.k_per_cta = K / csize;

  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = csize;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  set_programmatic(attr[1]);
  cfg.gridDim = dim3(m_tiles * csize, 1, 1);
  cfg.blockDim = dim3(svdq::kQ1Threads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaSuccess;
  switch (r) {
    case 0:
      cfg.dynamicSmemBytes = svdq::Q1Layout<0>::kSmem;
      e = cudaLaunchKernelEx(&cfg, svdq::quant_act_kernel<0, svdq::Nvfp4Act>, tmX, tmL1, a);
      break;
    case 16:
      cfg.dynamicSmemBytes = svdq::Q1Layout<16>::kSmem;
      e = cudaLaunchKernelEx(&cfg, svdq::quant_act_kernel<16, svdq::Nvfp4Act>, tmX, tmL1, a);
      break;
    case 32:
      cfg.dynamicSmemBytes = svdq::Q1Layout<32>::kSmem;
      e = cudaLaunchKernelEx(&cfg, svdq::quant_act_kernel<32, svdq::Nvfp4Act>, tmX, tmL1, a);
      break;
    case 64:
      cfg.dynamicSmemBytes = svdq::Q1Layout<64>::kSmem;
      e = cudaLaunchKernelEx(&cfg, svdq::quant_act_kernel<64, svdq::Nvfp4Act>, tmX, tmL1, a);
      break;
    default: return fail(SVDQ_ERR_UNSUPPORTED, "r=%d unsupported", r);
  }
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of quant_act_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("quant_act_kernel");
}

svdq_status svdq_gemm(const svdq_act* act, const svdq_weight* w, const uint16_t* bias, svdq_epilogue epi, void* Y,
                      svdq_out_dtype out_dtype, svdq_stream_t stream) {
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
  if (!aligned16(Y) || (bias != nullptr && !aligned16(bias))) return fail(SVDQ_ERR_UNSUPPORTED, "Y / bias alignment");
  const int n_tile = w->n_tile;
  int dev, sms;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;

  const int K = w->K, r = w->r;
  CUtensorMap tmA, tmU;
  std::memset(&tmU, 0, sizeof(tmU));
  if (svdq_status s = make_tmap(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, act->codes, K / 2, act->M_pad, K / 2, 128, 128,
                                CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  if (r > 0) {
    if (svdq_status s = make_tmap(&tmU, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, act->U, r, 2 * static_cast<uint64_t>(act->M_pad),
                                  static_cast<uint64_t>(r) * 2, r < 32 ? r : 32, 128, lr_swizzle(r));
        s != SVDQ_OK)
      return s;
  }
  CUtensorMap tmB, tmL2;  // properly aligned copies of the descriptors cached in the weight
  std::memcpy(&tmB, &w->tmap[0][0], sizeof(CUtensorMap));
  std::memcpy(&tmL2, &w->tmap[1][0], sizeof(CUtensorMap));

  svdq::GemmArgs g{};
  g.sfa = static_cast<const uint8_t*>(act->scales);
  g.sfb = static_cast<const uint8_t*>(w->scales);
  g.alpha = act->alpha;
  g.bias = reinterpret_cast<const __nv_bfloat16*>(bias);
  g.Y = Y;
  g.wait_ns = g_wait_ns.load();
  g.M = act->M;
  g.M_pad = act->M_pad;
  g.N = w->N;
  g.K = K;
  g.r = r;
  g.m_tiles = act->M_pad / 128;
  g.m_pairs = (g.m_tiles + 1) / 2;
  g.n_tiles = w->N / n_tile;
  g.k_iters = K / 256;
  g.num_tiles = g.m_pairs * g.n_tiles;
  g.ldy = swiglu ? w->N / 2 : w->N;
  g.out_f32 = out_dtype == SVDQ_OUT_F32 ? 1 : 0;
  g.epi = static_cast<int>(epi);
  CUtensorMap tmY;
  if (svdq_status s = make_tmap(&tmY, g.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, Y,
                                static_cast<uint64_t>(g.ldy), static_cast<uint64_t>(act->M),
                                static_cast<uint64_t>(g.ldy) * (g.out_f32 ? 4 : 2), 32, 32,
                                g.out_f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
      s != SVDQ_OK)
    return s;
  int max_pairs = 0;
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    max_pairs = g_dev[dev].max_pairs[n_tile == 256 ? 0 : n_tile == 192 ? 1 : n_tile == 128 ? 2 : 3];
  }
  const int pairs = g.num_tiles < max_pairs ? g.num_tiles : max_pairs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (n_tile == 384)
    e = launch_pair_gemm(svdq::pair_gemm_kernel<svdq::Nvfp4Gemm, 384, kStagesTile384>, 2 * pairs,
                         svdq::GemmLayout<384, kStagesTile384>::kSmem, st, tmA, tmB, tmU, tmL2, tmY, g);
  else if (n_tile == 256)
    e = launch_pair_gemm(svdq::pair_gemm_kernel<svdq::Nvfp4Gemm, 256, kStagesTile256>, 2 * pairs,
                         svdq::GemmLayout<256, kStagesTile256>::kSmem, st, tmA, tmB, tmU, tmL2, tmY, g);
  else if (n_tile == 192)
    e = launch_pair_gemm(svdq::pair_gemm_kernel<svdq::Nvfp4Gemm, 192, kStagesTile192>, 2 * pairs,
                         svdq::GemmLayout<192, kStagesTile192>::kSmem, st, tmA, tmB, tmU, tmL2, tmY, g);
  else
    e = launch_pair_gemm(svdq::pair_gemm_kernel<svdq::Nvfp4Gemm, 128, kStagesTile128>, 2 * pairs,
                         svdq::GemmLayout<128, kStagesTile128>::kSmem, st, tmA, tmB, tmU, tmL2, tmY, g);
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of pair_gemm_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("pair_gemm_kernel (NVFP4)");
}

svdq_status svdq_export_weight(const svdq_weight* w, uint8_t* codes, uint8_t* scales, svdq_stream_t stream) {
  if (w == nullptr || codes == nullptr || scales == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_weight(w); s != SVDQ_OK) return s;
  int dev, sms;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;
  const size_t total = static_cast<size_t>(w->N) * (w->K / 16);
  svdq::export_weight_kernel<<<grid_for(total, 256, sms), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(w->codes), static_cast<const uint8_t*>(w->scales), w->N, w->K, w->n_tile,
      w->swiglu_interleaved, codes, scales);
  return check_launch("export_weight_kernel");
}

svdq_status svdq_export_act(const svdq_act* act, uint8_t* codes, uint8_t* scales, svdq_stream_t stream) {
  if (act == nullptr || codes == nullptr || scales == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_act(act); s != SVDQ_OK) return s;
  int dev, sms;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;
  const size_t total = static_cast<size_t>(act->M) * (act->K / 16);
  svdq::export_act_kernel<<<grid_for(total, 256, sms), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(act->codes), static_cast<const uint8_t*>(act->scales), act->M, act->K, codes,
      scales);
  return check_launch("export_act_kernel");
}

svdq_status svdq_device_status(int reset) {
  SVDQ_CUDA(cudaDeviceSynchronize());
  unsigned v = 0;
  SVDQ_CUDA(cudaMemcpyFromSymbol(&v, svdq::g_svdq_status, sizeof(v)));
  if (reset) {
    const unsigned z = 0;
    SVDQ_CUDA(cudaMemcpyToSymbol(svdq::g_svdq_status, &z, sizeof(z)));
  }
  if (v != 0) return fail(SVDQ_ERR_TIMEOUT, "device wait ran out (status bits 0x%x)", v);
  return SVDQ_OK;
}

svdq_status svdq_watchdog_selftest(unsigned long long limit_ns, svdq_stream_t stream) {
  if (limit_ns < 1000ull || limit_ns > 1000000000ull) return fail(SVDQ_ERR_INVALID_ARG, "limit out of range");
  int dev, sms;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;
  svdq::watchdog_selftest_kernel<<<1, 1, 0, static_cast<cudaStream_t>(stream)>>>(limit_ns);
  return check_launch("watchdog_selftest_kernel");
}

}  // extern "C"

// ================================================================== row-wise FP8 (W8A8) variant
namespace {

constexpr int kFp8Stages256 = 6;
constexpr int kFp8Stages192 = 6;
constexpr int kFp8Stages128 = 8;

struct Fp8rState {
  bool ready = false;
  int max_pairs[3] = {0, 0, 0};  // co-resident CTA pairs of the FP8 GEMM for n_tile 256, 192, 128
};
Fp8rState g_fp8r[64];

svdq_status fp8r_max_pairs(const void* fn, int smem, int sms, int* out) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * (sms / 2), 1, 1);
  cfg.blockDim = dim3(svdq::kGemmThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  int n = 0;
  SVDQ_CUDA(cudaOccupancyMaxActiveClusters(&n, fn, &cfg));
  if (n <= 0) return fail(SVDQ_ERR_CUDA, "FP8 GEMM kernel cannot be resident as CTA pairs");
  *out = n;
  return SVDQ_OK;
}

// The FP8 kernels are set up on the first FP8 call on a device, apart from the NVFP4 set-up (which
// never depends on them).
svdq_status fp8r_ready(int* dev_out, int* sm_out) {
  int dev = 0, sms = 0;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  Fp8rState& st = g_fp8r[dev];
  if (!st.ready) {
    using L256 = svdq::PairGemmLayout<false, 256, kFp8Stages256>;
    using L192 = svdq::PairGemmLayout<false, 192, kFp8Stages192>;
    using L128 = svdq::PairGemmLayout<false, 128, kFp8Stages128>;
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::pair_gemm_kernel<svdq::fp8r::Fp8Gemm, 256, kFp8Stages256>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, L256::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::pair_gemm_kernel<svdq::fp8r::Fp8Gemm, 192, kFp8Stages192>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, L192::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::pair_gemm_kernel<svdq::fp8r::Fp8Gemm, 128, kFp8Stages128>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, L128::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::quant_act_kernel<0, svdq::fp8r::RowAct>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, svdq::Q1Layout<0>::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::quant_act_kernel<16, svdq::fp8r::RowAct>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, svdq::Q1Layout<16>::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::quant_act_kernel<32, svdq::fp8r::RowAct>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, svdq::Q1Layout<32>::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::quant_act_kernel<64, svdq::fp8r::RowAct>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, svdq::Q1Layout<64>::kSmem));
    if (svdq_status s = fp8r_max_pairs(reinterpret_cast<const void*>(svdq::pair_gemm_kernel<svdq::fp8r::Fp8Gemm, 256, kFp8Stages256>),
                                       L256::kSmem, sms, &st.max_pairs[0]);
        s != SVDQ_OK)
      return s;
    if (svdq_status s = fp8r_max_pairs(reinterpret_cast<const void*>(svdq::pair_gemm_kernel<svdq::fp8r::Fp8Gemm, 192, kFp8Stages192>),
                                       L192::kSmem, sms, &st.max_pairs[1]);
        s != SVDQ_OK)
      return s;
    if (svdq_status s = fp8r_max_pairs(reinterpret_cast<const void*>(svdq::pair_gemm_kernel<svdq::fp8r::Fp8Gemm, 128, kFp8Stages128>),
                                       L128::kSmem, sms, &st.max_pairs[2]);
        s != SVDQ_OK)
      return s;
    st.ready = true;
  }
  if (dev_out) *dev_out = dev;
  if (sm_out) *sm_out = sms;
  return SVDQ_OK;
}

struct Fp8rWeightLayout {
  size_t codes, scales, inv_lambda, l1t, l2t, total;
};
Fp8rWeightLayout fp8r_weight_layout(int N, int K, int r) {
  Fp8rWeightLayout l{};
  size_t off = 0;
  l.codes = off;
  off = align_up(off + static_cast<size_t>(N) * K);
  l.scales = off;
  off = align_up(off + static_cast<size_t>(N) * 4);
  l.inv_lambda = off;
  off = align_up(off + static_cast<size_t>(K) * 4);
  l.l1t = off;
  off = align_up(off + static_cast<size_t>(r) * K * 2);
  l.l2t = off;
  off = align_up(off + static_cast<size_t>(N) * r * 2 * 2);  // hi and lo halves
  l.total = off;
  return l;
}

struct Fp8rActLayout {
  size_t codes, s_x, rs_x, u, total;
  int M_pad;
};
Fp8rActLayout fp8r_act_layout(int M, int K, int r) {
  Fp8rActLayout l{};
  l.M_pad = (M + 127) / 128 * 128;
  size_t off = 0;
  l.codes = off;
  off = align_up(off + static_cast<size_t>(l.M_pad) * K);
  l.s_x = off;
  off = align_up(off + static_cast<size_t>(l.M_pad) * 4);
  l.rs_x = off;
  off = align_up(off + static_cast<size_t>(l.M_pad) * 4);
  l.u = off;
  off = align_up(off + static_cast<size_t>(l.M_pad) * r * 2 * 2);  // hi and lo halves
  l.total = off;
  return l;
}

svdq_status check_fp8r_weight(const svdq_fp8r_weight* w) {
  const int t = w->n_tile;
  if ((t != 256 && t != 192 && t != 128) || w->N <= 0 || w->N % t != 0 || w->N > (1 << 20) || w->K <= 0 ||
      w->K % 256 != 0 || w->K > (1 << 20) || !valid_r(w->r))
    return fail(SVDQ_ERR_INVALID_ARG,
                "FP8 weight descriptor N=%d K=%d r=%d n_tile=%d is not one svdq_fp8r_pack_weight makes", w->N, w->K,
                w->r, t);
  if (w->codes == nullptr || w->row_scale == nullptr || w->inv_lambda == nullptr ||
      (w->r > 0 && (w->L1s_t == nullptr || w->L2_t == nullptr)))
    return fail(SVDQ_ERR_INVALID_ARG, "FP8 weight descriptor has a null buffer");
  return SVDQ_OK;
}

svdq_status check_fp8r_act(const svdq_fp8r_act* a) {
  if (a->M < 1 || a->M >= (1 << 24) || a->K <= 0 || a->K % 256 != 0 || a->K > (1 << 20) || !valid_r(a->r) ||
      a->M_pad != (a->M + 127) / 128 * 128)
    return fail(SVDQ_ERR_INVALID_ARG,
                "FP8 act descriptor M=%d M_pad=%d K=%d r=%d is not one svdq_fp8r_act_bind makes", a->M, a->M_pad,
                a->K, a->r);
  if (a->codes == nullptr || a->row_scale == nullptr || a->row_rscale == nullptr || (a->r > 0 && a->U == nullptr))
    return fail(SVDQ_ERR_INVALID_ARG, "FP8 act descriptor has a null buffer");
  return SVDQ_OK;
}

}  // namespace

extern "C" {

size_t svdq_fp8r_weight_bytes(int N, int K, int r) {
  if (!shape_ok(N, K, r)) return 0;
  return fp8r_weight_layout(N, K, r).total;
}

size_t svdq_fp8r_act_bytes(int M, int K, int r) {
  if (M < 1 || M >= (1 << 24) || K <= 0 || K % 256 != 0 || K > (1 << 20) || !valid_r(r)) return 0;
  return fp8r_act_layout(M, K, r).total;
}

svdq_status svdq_fp8r_act_bind(int M, int K, int r, void* dst, size_t dst_bytes, svdq_fp8r_act* out) {
  if (out == nullptr || dst == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  const size_t need = svdq_fp8r_act_bytes(M, K, r);
  if (need == 0) return fail(SVDQ_ERR_UNSUPPORTED, "FP8 act shape M=%d K=%d r=%d unsupported", M, K, r);
  if (dst_bytes < need) return fail(SVDQ_ERR_INVALID_ARG, "FP8 act buffer %zu bytes < %zu", dst_bytes, need);
  if (reinterpret_cast<uintptr_t>(dst) % kAlign) return fail(SVDQ_ERR_UNSUPPORTED, "act buffer not 256-byte aligned");
  const Fp8rActLayout l = fp8r_act_layout(M, K, r);
  uint8_t* b = static_cast<uint8_t*>(dst);
  out->M = M;
  out->K = K;
  out->r = r;
  out->M_pad = l.M_pad;
  out->codes = b + l.codes;
  out->row_scale = reinterpret_cast<float*>(b + l.s_x);
  out->row_rscale = reinterpret_cast<float*>(b + l.rs_x);
  out->U = b + l.u;
  return SVDQ_OK;
}

svdq_status svdq_fp8r_pack_weight(const float* R_nk, const uint16_t* L1s_kr, const uint16_t* L2_rn,
                                  const float* inv_lambda, int N, int K, int r, int swiglu, void* dst,
                                  size_t dst_bytes, svdq_fp8r_weight* out, svdq_stream_t stream) {
  if (out == nullptr || R_nk == nullptr || inv_lambda == nullptr || dst == nullptr)
    return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (r > 0 && (L1s_kr == nullptr || L2_rn == nullptr)) return fail(SVDQ_ERR_INVALID_ARG, "null L1s / L2 with r > 0");
  if (!shape_ok(N, K, r)) return fail(SVDQ_ERR_UNSUPPORTED, "weight shape N=%d K=%d r=%d unsupported", N, K, r);
  if (!aligned16(R_nk) || !aligned16(inv_lambda) || (r > 0 && (!aligned16(L1s_kr) || !aligned16(L2_rn))))
    return fail(SVDQ_ERR_UNSUPPORTED, "inputs must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(dst) % kAlign) return fail(SVDQ_ERR_UNSUPPORTED, "dst not 256-byte aligned");
  const int n_tile = choose_n_tile(N, swiglu, false);
  const Fp8rWeightLayout l = fp8r_weight_layout(N, K, r);
  if (dst_bytes < l.total) return fail(SVDQ_ERR_INVALID_ARG, "FP8 weight buffer %zu bytes < %zu", dst_bytes, l.total);
  int dev, sms;
  if (svdq_status s = fp8r_ready(&dev, &sms); s != SVDQ_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* b = static_cast<uint8_t*>(dst);

  svdq_fp8r_weight w{};
  w.N = N;
  w.K = K;
  w.r = r;
  w.swiglu_interleaved = swiglu ? 1 : 0;
  w.n_tile = n_tile;
  w.codes = b + l.codes;
  w.row_scale = reinterpret_cast<float*>(b + l.scales);
  w.inv_lambda = reinterpret_cast<float*>(b + l.inv_lambda);
  w.L1s_t = b + l.l1t;
  w.L2_t = b + l.l2t;

  SVDQ_CUDA(cudaMemcpyAsync(w.inv_lambda, inv_lambda, static_cast<size_t>(K) * 4, cudaMemcpyDeviceToDevice, st));
  svdq::fp8r::pack_weight_kernel<<<grid_for(static_cast<size_t>(N) * 32, 256, sms), 256, 0, st>>>(
      R_nk, N, K, n_tile, w.swiglu_interleaved, static_cast<uint8_t*>(w.codes), w.row_scale);
  if (svdq_status s = check_launch("fp8r::pack_weight_kernel"); s != SVDQ_OK) return s;
  if (r > 0) {
    svdq::transpose_l1_kernel<<<grid_for(static_cast<size_t>(K) * r, 256, sms), 256, 0, st>>>(
        reinterpret_cast<const __nv_bfloat16*>(L1s_kr), K, r, static_cast<__nv_bfloat16*>(w.L1s_t));
    if (svdq_status s = check_launch("transpose_l1_kernel"); s != SVDQ_OK) return s;
    svdq::fp8r::pack_l2_kernel<<<grid_for(static_cast<size_t>(N) * r, 256, sms), 256, 0, st>>>(
        reinterpret_cast<const __nv_bfloat16*>(L2_rn), w.row_scale, N, r, n_tile, w.swiglu_interleaved,
        static_cast<__nv_bfloat16*>(w.L2_t));
    if (svdq_status s = check_launch("fp8r::pack_l2_kernel"); s != SVDQ_OK) return s;
  }
  static_assert(sizeof(w.tmap) >= 2 * sizeof(CUtensorMap), "tmap storage");
  CUtensorMap tmB, tmL2;
  std::memset(&tmL2, 0, sizeof(tmL2));
  // each CTA of a GEMM pair stages half of a tile's n_tile rows; one K step is 128 bytes of a row
  if (svdq_status s = make_tmap(&tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, K, N, K, 128, n_tile / 2,
                                CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  if (r > 0) {
    // rows 0..N-1: hi halves, rows N..2N-1: lo halves
    if (svdq_status s = make_tmap(&tmL2, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w.L2_t, r, 2 * static_cast<uint64_t>(N),
                                  static_cast<uint64_t>(r) * 2, r < 32 ? r : 32, n_tile / 2, lr_swizzle(r));
        s != SVDQ_OK)
      return s;
  }
  std::memcpy(&w.tmap[0][0], &tmB, sizeof(CUtensorMap));
  std::memcpy(&w.tmap[1][0], &tmL2, sizeof(CUtensorMap));
  *out = w;
  return SVDQ_OK;
}

svdq_status svdq_fp8r_quantize_act(const uint16_t* X, const svdq_fp8r_weight* w, const svdq_fp8r_act* act,
                                   svdq_stream_t stream) {
  if (X == nullptr || w == nullptr || act == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (act->K != w->K || act->r != w->r)
    return fail(SVDQ_ERR_INVALID_ARG, "act (K=%d r=%d) does not match weight (K=%d r=%d)", act->K, act->r, w->K, w->r);
  if (svdq_status s = check_fp8r_weight(w); s != SVDQ_OK) return s;
  if (svdq_status s = check_fp8r_act(act); s != SVDQ_OK) return s;
  if (!aligned16(X)) return fail(SVDQ_ERR_UNSUPPORTED, "X must be 16-byte aligned");
  int dev, sms;
  if (svdq_status s = fp8r_ready(&dev, &sms); s != SVDQ_OK) return s;
  const int K = act->K, r = w->r, M = act->M;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // row scales first: the quantizing pass needs each row's amax before its first code
  {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    set_programmatic(attr[0]);
    cfg.gridDim = dim3(grid_for(static_cast<size_t>(act->M_pad) * 32, 256, sms), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e =
        cudaLaunchKernelEx(&cfg, svdq::fp8r::act_row_scale_kernel, reinterpret_cast<const __nv_bfloat16*>(X),
                           static_cast<const float*>(w->inv_lambda), M, act->M_pad, K, act->row_scale, act->row_rscale);
    if (e != cudaSuccess)
      return fail(SVDQ_ERR_CUDA, "launch of fp8r::act_row_scale_kernel failed: %s", cudaGetErrorString(e));
  }
  if (svdq_status s = check_launch("fp8r::act_row_scale_kernel"); s != SVDQ_OK) return s;
  CUtensorMap tmX, tmL1;
  std::memset(&tmL1, 0, sizeof(tmL1));
  if (svdq_status s = make_tmap(&tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, K, M, static_cast<uint64_t>(K) * 2, 64, 128,
                                CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  if (r > 0) {
    if (svdq_status s = make_tmap(&tmL1, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w->L1s_t, K, r,
                                  static_cast<uint64_t>(K) * 2, 64, r, CU_TENSOR_MAP_SWIZZLE_128B);
        s != SVDQ_OK)
      return s;
  }
  // K split over a cluster exactly as for the NVFP4 kernel 1 (the same kernel body and resources)
  const int m_tiles = act->M_pad / 128;
  int csize = 1;
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    const int* mc = g_dev[dev].k1_clusters[r == 0 ? 0 : r == 16 ? 1 : r == 32 ? 2 : 3];
    for (int c = 2; c <= 4; ++c)
      if (m_tiles <= mc[c - 1] && K % (64 * c) == 0) csize = c;
  }
  svdq::fp8r::ActArgs a;
  a.inv_lambda = w->inv_lambda;
  a.rs_x = act->row_rscale;
  a.codes = static_cast<uint8_t*>(act->codes);
  a.U = static_cast<__nv_bfloat16*>(act->U);
  a.wait_ns = g_wait_ns.load();
  a.M = M;
  a.K = K;
  a.M_pad = act->M_pad;
  a.k_per_cta = K / csize;

  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = csize;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  set_programmatic(attr[1]);
  cfg.gridDim = dim3(m_tiles * csize, 1, 1);
  cfg.blockDim = dim3(svdq::kQ1Threads, 1, 1);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaSuccess;
  switch (r) {
    case 0:
      cfg.dynamicSmemBytes = svdq::Q1Layout<0>::kSmem;
      e = cudaLaunchKernelEx(&cfg, svdq::quant_act_kernel<0, svdq::fp8r::RowAct>, tmX, tmL1, a);
      break;
    case 16:
      cfg.dynamicSmemBytes = svdq::Q1Layout<16>::kSmem;
      e = cudaLaunchKernelEx(&cfg, svdq::quant_act_kernel<16, svdq::fp8r::RowAct>, tmX, tmL1, a);
      break;
    case 32:
      cfg.dynamicSmemBytes = svdq::Q1Layout<32>::kSmem;
      e = cudaLaunchKernelEx(&cfg, svdq::quant_act_kernel<32, svdq::fp8r::RowAct>, tmX, tmL1, a);
      break;
    case 64:
      cfg.dynamicSmemBytes = svdq::Q1Layout<64>::kSmem;
      e = cudaLaunchKernelEx(&cfg, svdq::quant_act_kernel<64, svdq::fp8r::RowAct>, tmX, tmL1, a);
      break;
    default: return fail(SVDQ_ERR_UNSUPPORTED, "r=%d unsupported", r);
  }
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of the row-wise FP8 quant_act_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("quant_act_kernel (row-wise FP8)");
}

svdq_status svdq_fp8r_gemm(const svdq_fp8r_act* act, const svdq_fp8r_weight* w, const uint16_t* bias,
                           svdq_epilogue epi, void* Y, svdq_out_dtype out_dtype, svdq_stream_t stream) {
  if (act == nullptr || w == nullptr || Y == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (act->K != w->K || act->r != w->r) return fail(SVDQ_ERR_INVALID_ARG, "act does not match weight");
  if (svdq_status s = check_fp8r_weight(w); s != SVDQ_OK) return s;
  if (svdq_status s = check_fp8r_act(act); s != SVDQ_OK) return s;
  if (epi < SVDQ_EPI_NONE || epi > SVDQ_EPI_BIAS_SWIGLU) return fail(SVDQ_ERR_INVALID_ARG, "bad epilogue %d", epi);
  if (out_dtype != SVDQ_OUT_BF16 && out_dtype != SVDQ_OUT_F32) return fail(SVDQ_ERR_INVALID_ARG, "bad out dtype");
  const bool has_bias = (epi & 1) != 0, swiglu = (epi & 2) != 0;
  if (has_bias && bias == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "epilogue needs a bias");
  if (swiglu && !w->swiglu_interleaved) return fail(SVDQ_ERR_INVALID_ARG, "SwiGLU needs a weight packed with swiglu=1");
  if (!swiglu && w->swiglu_interleaved) return fail(SVDQ_ERR_INVALID_ARG, "weight packed for SwiGLU");
  if (!aligned16(Y) || (bias != nullptr && !aligned16(bias))) return fail(SVDQ_ERR_UNSUPPORTED, "Y / bias alignment");
  const int n_tile = w->n_tile;
  int dev, sms;
  if (svdq_status s = fp8r_ready(&dev, &sms); s != SVDQ_OK) return s;

  const int K = w->K, r = w->r;
  CUtensorMap tmA, tmU;
  std::memset(&tmU, 0, sizeof(tmU));
  if (svdq_status s = make_tmap(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, act->codes, K, act->M_pad, K, 128, 128,
                                CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  if (r > 0) {
    if (svdq_status s = make_tmap(&tmU, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, act->U, r, 2 * static_cast<uint64_t>(act->M_pad),
                                  static_cast<uint64_t>(r) * 2, r < 32 ? r : 32, 128, lr_swizzle(r));
        s != SVDQ_OK)
      return s;
  }
  CUtensorMap tmB, tmL2;  // properly aligned copies of the descriptors cached in the weight
  std::memcpy(&tmB, &w->tmap[0][0], sizeof(CUtensorMap));
  std::memcpy(&tmL2, &w->tmap[1][0], sizeof(CUtensorMap));

  svdq::fp8r::GemmArgs g{};
  g.s_x = act->row_scale;
  g.s_w = w->row_scale;
  g.bias = reinterpret_cast<const __nv_bfloat16*>(bias);
  g.Y = Y;
  g.wait_ns = g_wait_ns.load();
  g.M = act->M;
  g.M_pad = act->M_pad;
  g.N = w->N;
  g.K = K;
  g.r = r;
  g.m_tiles = act->M_pad / 128;
  g.m_pairs = (g.m_tiles + 1) / 2;
  g.n_tiles = w->N / n_tile;
  g.k_iters = K / 128;
  g.num_tiles = g.m_pairs * g.n_tiles;
  g.ldy = swiglu ? w->N / 2 : w->N;
  g.out_f32 = out_dtype == SVDQ_OUT_F32 ? 1 : 0;
  g.epi = static_cast<int>(epi);
  CUtensorMap tmY;
  if (svdq_status s = make_tmap(&tmY, g.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, Y,
                                static_cast<uint64_t>(g.ldy), static_cast<uint64_t>(act->M),
                                static_cast<uint64_t>(g.ldy) * (g.out_f32 ? 4 : 2), 32, 32,
                                g.out_f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
      s != SVDQ_OK)
    return s;
  int max_pairs = 0;
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    max_pairs = g_fp8r[dev].max_pairs[n_tile == 256 ? 0 : n_tile == 192 ? 1 : 2];
  }
  const int pairs = g.num_tiles < max_pairs ? g.num_tiles : max_pairs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (n_tile == 256)
    e = launch_pair_gemm(svdq::pair_gemm_kernel<svdq::fp8r::Fp8Gemm, 256, kFp8Stages256>, 2 * pairs,
                         svdq::PairGemmLayout<false, 256, kFp8Stages256>::kSmem, st, tmA, tmB, tmU, tmL2, tmY, g);
  else if (n_tile == 192)
    e = launch_pair_gemm(svdq::pair_gemm_kernel<svdq::fp8r::Fp8Gemm, 192, kFp8Stages192>, 2 * pairs,
                         svdq::PairGemmLayout<false, 192, kFp8Stages192>::kSmem, st, tmA, tmB, tmU, tmL2, tmY, g);
  else
    e = launch_pair_gemm(svdq::pair_gemm_kernel<svdq::fp8r::Fp8Gemm, 128, kFp8Stages128>, 2 * pairs,
                         svdq::PairGemmLayout<false, 128, kFp8Stages128>::kSmem, st, tmA, tmB, tmU, tmL2, tmY, g);
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of pair_gemm_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("pair_gemm_kernel (row-wise FP8)");
}

svdq_status svdq_fp8r_export_weight(const svdq_fp8r_weight* w, uint8_t* codes, float* scales, svdq_stream_t stream) {
  if (w == nullptr || codes == nullptr || scales == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_fp8r_weight(w); s != SVDQ_OK) return s;
  if (!aligned16(codes) || (reinterpret_cast<uintptr_t>(scales) & 3u))
    return fail(SVDQ_ERR_UNSUPPORTED, "codes must be 16-byte and scales 4-byte aligned");
  int dev, sms;
  if (svdq_status s = fp8r_ready(&dev, &sms); s != SVDQ_OK) return s;
  const size_t total = static_cast<size_t>(w->N) * (w->K / 16);
  svdq::fp8r::export_weight_kernel<<<grid_for(total, 256, sms), 256, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(w->codes), w->row_scale, w->N, w->K, w->n_tile, w->swiglu_interleaved, codes,
      scales);
  return check_launch("fp8r::export_weight_kernel");
}

svdq_status svdq_fp8r_export_act(const svdq_fp8r_act* act, uint8_t* codes, float* scales, svdq_stream_t stream) {
  if (act == nullptr || codes == nullptr || scales == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_fp8r_act(act); s != SVDQ_OK) return s;
  int dev, sms;
  if (svdq_status s = fp8r_ready(&dev, &sms); s != SVDQ_OK) return s;
  // the activation codes are already canonical row-major; rows >= M are padding
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  SVDQ_CUDA(cudaMemcpyAsync(codes, act->codes, static_cast<size_t>(act->M) * act->K, cudaMemcpyDeviceToDevice, st));
  SVDQ_CUDA(cudaMemcpyAsync(scales, act->row_scale, static_cast<size_t>(act->M) * 4, cudaMemcpyDeviceToDevice, st));
  return SVDQ_OK;
}

}  // extern "C"

// ================================================================== MLP chain: kernel 1 fused into SwiGLU
namespace {

constexpr int kFusedStages = 5;
constexpr int kMaxSplits = svdq::fused::kMaxUSplits;

struct FusedState {
  bool ready = false;
  int max_pairs[3] = {0, 0, 0};  // r_next 16, 32, 64
};
FusedState g_fused[64];

svdq_status fused_ready(int* dev_out, int* sm_out) {
  int dev = 0, sms = 0;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  FusedState& st = g_fused[dev];
  if (!st.ready) {
    using L16 = svdq::fused::Layout<kFusedStages, 16>;
    using L32 = svdq::fused::Layout<kFusedStages, 32>;
    using L64 = svdq::fused::Layout<kFusedStages, 64>;
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::fused::gemm_swiglu_quant_kernel<kFusedStages, 16>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, L16::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::fused::gemm_swiglu_quant_kernel<kFusedStages, 32>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, L32::kSmem));
    SVDQ_CUDA(cudaFuncSetAttribute(svdq::fused::gemm_swiglu_quant_kernel<kFusedStages, 64>,
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, L64::kSmem));
    if (svdq_status s = fp8r_max_pairs(
            reinterpret_cast<const void*>(svdq::fused::gemm_swiglu_quant_kernel<kFusedStages, 16>), L16::kSmem, sms,
            &st.max_pairs[0]);
        s != SVDQ_OK)
      return s;
    if (svdq_status s = fp8r_max_pairs(
            reinterpret_cast<const void*>(svdq::fused::gemm_swiglu_quant_kernel<kFusedStages, 32>), L32::kSmem, sms,
            &st.max_pairs[1]);
        s != SVDQ_OK)
      return s;
    if (svdq_status s = fp8r_max_pairs(
            reinterpret_cast<const void*>(svdq::fused::gemm_swiglu_quant_kernel<kFusedStages, 64>), L64::kSmem, sms,
            &st.max_pairs[2]);
        s != SVDQ_OK)
      return s;
    st.ready = true;
  }
  if (dev_out) *dev_out = dev;
  if (sm_out) *sm_out = sms;
  return SVDQ_OK;
}

}  // namespace

extern "C" {

size_t svdq_mlp_scratch_bytes(int M, int r_next) {
  if (M < 1 || M >= (1 << 24) || !(r_next == 16 || r_next == 32 || r_next == 64)) return 0;
  const size_t m_pad = static_cast<size_t>((M + 127) / 128 * 128);
  return static_cast<size_t>(kMaxSplits) * m_pad * static_cast<size_t>(r_next) * 4;
}

svdq_status svdq_gemm_swiglu_quant(const svdq_act* act, const svdq_weight* w, const uint16_t* bias,
                                   const svdq_weight* w_next, const float* g_x_next, const svdq_act* act_next,
                                   void* scratch, size_t scratch_bytes, uint16_t* H, svdq_stream_t stream) {
  if (act == nullptr || w == nullptr || w_next == nullptr || g_x_next == nullptr || act_next == nullptr ||
      scratch == nullptr)
    return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (act->K != w->K || act->r != w->r) return fail(SVDQ_ERR_INVALID_ARG, "act does not match weight");
  if (svdq_status s = check_weight(w); s != SVDQ_OK) return s;
  if (svdq_status s = check_act(act); s != SVDQ_OK) return s;
  if (svdq_status s = check_weight(w_next); s != SVDQ_OK) return s;
  if (svdq_status s = check_act(act_next); s != SVDQ_OK) return s;
  if (!w->swiglu_interleaved || w->n_tile != 256)
    return fail(SVDQ_ERR_UNSUPPORTED, "the fused MLP path takes a SwiGLU weight packed with 256-wide tiles");
  if (w_next->swiglu_interleaved) return fail(SVDQ_ERR_INVALID_ARG, "the next layer's weight is packed for SwiGLU");
  if (w_next->K != w->N / 2) return fail(SVDQ_ERR_INVALID_ARG, "next layer K=%d != N/2=%d", w_next->K, w->N / 2);
  if (act_next->M != act->M || act_next->K != w_next->K || act_next->r != w_next->r)
    return fail(SVDQ_ERR_INVALID_ARG, "next act (M=%d K=%d r=%d) does not match", act_next->M, act_next->K,
                act_next->r);
  const int r2 = w_next->r;
  if (r2 != 16 && r2 != 32 && r2 != 64) return fail(SVDQ_ERR_UNSUPPORTED, "next layer rank %d not in 16/32/64", r2);
  const size_t need = svdq_mlp_scratch_bytes(act->M, r2);
  if (scratch_bytes < need) return fail(SVDQ_ERR_INVALID_ARG, "scratch %zu bytes < %zu", scratch_bytes, need);
  if (!aligned16(scratch) || (bias != nullptr && !aligned16(bias)) || (H != nullptr && !aligned16(H)) ||
      (reinterpret_cast<uintptr_t>(g_x_next) & 3u))
    return fail(SVDQ_ERR_UNSUPPORTED, "scratch / bias / H / g_x_next alignment");
  int dev, sms;
  if (svdq_status s = fused_ready(&dev, &sms); s != SVDQ_OK) return s;

  const int K = w->K, r = w->r, N = w->N, K2 = w_next->K;
  CUtensorMap tmA, tmU, tmH, tmL1n;
  std::memset(&tmU, 0, sizeof(tmU));
  std::memset(&tmH, 0, sizeof(tmH));
  if (svdq_status s = make_tmap(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, act->codes, K / 2, act->M_pad, K / 2, 128, 128,
                                CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  if (r > 0) {
    if (svdq_status s = make_tmap(&tmU, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, act->U, r, 2 * static_cast<uint64_t>(act->M_pad),
                                  static_cast<uint64_t>(r) * 2, r < 32 ? r : 32, 128, lr_swizzle(r));
        s != SVDQ_OK)
      return s;
  }
  // the next layer's L1s^T [r2][K2]: per tile, 64-column boxes of this CTA's r2/2 rows
  if (svdq_status s = make_tmap(&tmL1n, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w_next->L1s_t, K2, r2,
                                static_cast<uint64_t>(K2) * 2, 64, r2 / 2, CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  if (H != nullptr) {
    // h [M][N/2] bf16, stored from the 128B-swizzled h tile in 64 x 32 boxes
    if (svdq_status s = make_tmap(&tmH, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, H, static_cast<uint64_t>(N / 2),
                                  static_cast<uint64_t>(act->M), static_cast<uint64_t>(N / 2) * 2, 64, 32,
                                  CU_TENSOR_MAP_SWIZZLE_128B);
        s != SVDQ_OK)
      return s;
  }
  CUtensorMap tmB, tmL2;
  std::memcpy(&tmB, &w->tmap[0][0], sizeof(CUtensorMap));
  std::memcpy(&tmL2, &w->tmap[1][0], sizeof(CUtensorMap));

  svdq::fused::Args a{};
  a.sfa = static_cast<const uint8_t*>(act->scales);
  a.sfb = static_cast<const uint8_t*>(w->scales);
  a.alpha = act->alpha;
  a.bias = reinterpret_cast<const __nv_bfloat16*>(bias);
  a.wait_ns = g_wait_ns.load();
  a.M = act->M;
  a.M_pad = act->M_pad;
  a.N = N;
  a.K = K;
  a.r = r;
  a.m_tiles = act->M_pad / 128;
  a.m_pairs = (a.m_tiles + 1) / 2;
  a.n_tiles = N / 256;
  a.k_iters = K / 256;
  a.store_h = H != nullptr ? 1 : 0;
  a.inv_lambda2 = w_next->inv_lambda;
  a.g_x2 = g_x_next;
  a.codes2 = static_cast<uint8_t*>(act_next->codes);
  a.sf2 = static_cast<uint8_t*>(act_next->scales);
  a.partials = static_cast<float*>(scratch);
  a.K2 = K2;
  int max_pairs = 0;
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    max_pairs = g_fused[dev].max_pairs[r2 == 16 ? 0 : r2 == 32 ? 1 : 2];
  }
  // column splits: enough units to about fill the resident pairs, each a sweep over n_tiles/splits tiles
  int splits = max_pairs / a.m_pairs;
  if (splits < 1) splits = 1;
  if (splits > kMaxSplits) splits = kMaxSplits;
  if (splits > a.n_tiles) splits = a.n_tiles;
  a.splits = splits;
  a.num_units = a.m_pairs * splits;
  const int pairs = a.num_units < max_pairs ? a.num_units : max_pairs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (r2) {
    case 16:
      e = launch_pair_gemm(svdq::fused::gemm_swiglu_quant_kernel<kFusedStages, 16>, 2 * pairs,
                           svdq::fused::Layout<kFusedStages, 16>::kSmem, st, tmA, tmB, tmU, tmL2, tmH, tmL1n, a);
      break;
    case 32:
      e = launch_pair_gemm(svdq::fused::gemm_swiglu_quant_kernel<kFusedStages, 32>, 2 * pairs,
                           svdq::fused::Layout<kFusedStages, 32>::kSmem, st, tmA, tmB, tmU, tmL2, tmH, tmL1n, a);
      break;
    default:
      e = launch_pair_gemm(svdq::fused::gemm_swiglu_quant_kernel<kFusedStages, 64>, 2 * pairs,
                           svdq::fused::Layout<kFusedStages, 64>::kSmem, st, tmA, tmB, tmU, tmL2, tmH, tmL1n, a);
      break;
  }
  if (e != cudaSuccess)
    return fail(SVDQ_ERR_CUDA, "launch of fused::gemm_swiglu_quant_kernel failed: %s", cudaGetErrorString(e));
  if (svdq_status s = check_launch("fused::gemm_swiglu_quant_kernel"); s != SVDQ_OK) return s;
  {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    set_programmatic(attr[0]);
    cfg.gridDim = dim3(grid_for(static_cast<size_t>(act_next->M_pad) * r2, 256, sms), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, svdq::fused::finalize_u_kernel, static_cast<const float*>(scratch), splits, act->M,
                           act_next->M_pad, r2, g_x_next, static_cast<const float*>(w_next->g_w),
                           static_cast<__nv_bfloat16*>(act_next->U), act_next->alpha);
  }
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of fused::finalize_u_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("fused::finalize_u_kernel");
}

}  // extern "C"


// ================================================================== MLP chain without caller scratch
// svdq_gemm_swiglu_quant needs a scratch buffer for the column-split partial sums of U'. Some
// callers have none to lend and cannot allocate one; this entry point serves them from a buffer
// that lives in the library's own device image: a file-scope array of fixed size that every GPU
// which loads the library holds until the process exits. In host code the array's name is only a
// host-side stand-in, so its device address is looked up once per device (cudaGetSymbolAddress,
// with that device current) and handed to the kernels like any caller's scratch pointer.
namespace {

constexpr size_t kMlpBuiltinScratchBytes = SVDQ_MLP_BUILTIN_SCRATCH_BYTES;  // 8 MiB
static __device__ __align__(256) unsigned char g_mlp_builtin_scratch[kMlpBuiltinScratchBytes];

struct BuiltinScratchState {
  bool ready = false;
  void* ptr = nullptr;
};
BuiltinScratchState g_builtin_scratch[64];

// The device address of g_mlp_builtin_scratch on the current device (looked up on first use).
svdq_status builtin_scratch_ptr(void** out) {
  int dev = 0;
  SVDQ_CUDA(cudaGetDevice(&dev));
  if (dev < 0 || dev >= 64) return fail(SVDQ_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
  std::lock_guard<std::mutex> lk(g_dev_mu);
  BuiltinScratchState& st = g_builtin_scratch[dev];
  if (!st.ready) {
    void* p = nullptr;
    SVDQ_CUDA(cudaGetSymbolAddress(&p, g_mlp_builtin_scratch));
    if (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 255u) != 0)
      return fail(SVDQ_ERR_CUDA, "built-in scratch has no usable device address");
    st.ptr = p;
    st.ready = true;
  }
  *out = st.ptr;
  return SVDQ_OK;
}

}  // namespace

extern "C" {

svdq_status svdq_gemm_swiglu_quant_noscratch(const svdq_act* act, const svdq_weight* w, const uint16_t* bias,
                                             const svdq_weight* w_next, const float* g_x_next,
                                             const svdq_act* act_next, uint16_t* H, svdq_stream_t stream) {
  if (act == nullptr || w == nullptr || w_next == nullptr || g_x_next == nullptr || act_next == nullptr)
    return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  const size_t need = svdq_mlp_scratch_bytes(act->M, w_next->r);
  if (need == 0)
    return fail(SVDQ_ERR_UNSUPPORTED, "M=%d with next-layer rank %d unsupported", act->M, w_next->r);
  if (need > kMlpBuiltinScratchBytes)
    return fail(SVDQ_ERR_UNSUPPORTED,
                "M=%d at next-layer rank %d needs %zu bytes of scratch, more than the %zu-byte built-in buffer; "
                "pass a buffer to svdq_gemm_swiglu_quant instead",
                act->M, w_next->r, need, kMlpBuiltinScratchBytes);
  void* scratch = nullptr;
  if (svdq_status s = builtin_scratch_ptr(&scratch); s != SVDQ_OK) return s;
  return svdq_gemm_swiglu_quant(act, w, bias, w_next, g_x_next, act_next, scratch, kMlpBuiltinScratchBytes, H,
                                stream);
}

}  // extern "C"


// ================================================================== MXFP4 variant
namespace {

constexpr int kMxStages384 = 4;
constexpr int kMxStages256 = 5;
constexpr int kMxStages128 = 7;
template <int N_TILE, int STAGES>
using MxLayout = svdq::PairGemmLayout<true, N_TILE, STAGES, svdq::mx::Gemm::kSfAtomsK, svdq::mx::Gemm::kBiasSmem>;

struct MxState {
  bool ready = false;
  int max_pairs[3] = {0, 0, 0};  // co-resident CTA pairs of the MXFP4 GEMM for n_tile 384, 256, 128
  int few_clusters[4] = {0, 0, 0, 0};  // co-resident few-row clusters of 1, 2, 4 and 8 CTAs
};
MxState g_mx[64];

// A few-row block asks for at least this much shared memory, so that an SM holds one: its TMEM columns
// (up to 512) are then free when it starts, and no cluster can wait for columns that another waiting
// cluster holds.
constexpr int kFewMinSmem = 116 * 1024;
constexpr int kFewMaxSmem = 226 * 1024;

// The few-row quantizer holds its share of up to 8 raw rows in shared memory: 2 K bytes.
constexpr int kFewQuantMaxK = 49152;
template <int R>
svdq_status mx_few_quant_setup() {
  SVDQ_CUDA(cudaFuncSetAttribute(svdq::mx::few_quant_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 2 * kFewQuantMaxK));
  return SVDQ_OK;
}

template <int NB>
svdq_status mx_few_setup(int sms, int* clusters) {
  auto* kern = svdq::mx::few_gemm_kernel<NB>;
  SVDQ_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewMaxSmem));
  for (int i = 0; i < 4; ++i) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1 << i;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3((sms >> i) << i, 1, 1);
    cfg.blockDim = dim3(svdq::mx::kFewThreads, 1, 1);
    cfg.dynamicSmemBytes = kFewMinSmem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    SVDQ_CUDA(cudaOccupancyMaxActiveClusters(&clusters[i], kern, &cfg));
  }
  return SVDQ_OK;
}

template <int N_TILE, int STAGES>
svdq_status mx_gemm_setup(int sms, int* max_pairs) {
  auto* kern = svdq::pair_gemm_kernel<svdq::mx::Gemm, N_TILE, STAGES>;
  SVDQ_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, MxLayout<N_TILE, STAGES>::kSmem));
  return fp8r_max_pairs(reinterpret_cast<const void*>(kern), MxLayout<N_TILE, STAGES>::kSmem, sms, max_pairs);
}
template <int R>
svdq_status mx_quant_setup() {
  auto* kern = svdq::quant_act_kernel<R, svdq::mx::Act>;
  SVDQ_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, svdq::Q1Layout<R>::kSmem));
  return SVDQ_OK;
}

// The MXFP4 kernels are set up on the first MXFP4 call on a device.
svdq_status mx_ready(int* dev_out, int* sm_out) {
  int dev = 0, sms = 0;
  if (svdq_status s = device_ready(&dev, &sms); s != SVDQ_OK) return s;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  MxState& st = g_mx[dev];
  if (!st.ready) {
    svdq_status s = mx_gemm_setup<384, kMxStages384>(sms, &st.max_pairs[0]);
    if (s == SVDQ_OK) s = mx_gemm_setup<256, kMxStages256>(sms, &st.max_pairs[1]);
    if (s == SVDQ_OK) s = mx_gemm_setup<128, kMxStages128>(sms, &st.max_pairs[2]);
    if (s == SVDQ_OK) s = mx_quant_setup<0>();
    if (s == SVDQ_OK) s = mx_quant_setup<16>();
    if (s == SVDQ_OK) s = mx_quant_setup<32>();
    if (s == SVDQ_OK) s = mx_quant_setup<64>();
    if (s == SVDQ_OK) s = mx_few_quant_setup<16>();
    if (s == SVDQ_OK) s = mx_few_quant_setup<32>();
    if (s == SVDQ_OK) s = mx_few_quant_setup<64>();
    if (s == SVDQ_OK) s = mx_few_setup<2>(sms, st.few_clusters);
    if (s == SVDQ_OK) s = mx_few_setup<1>(sms, st.few_clusters);
    if (s != SVDQ_OK) return s;
    st.ready = true;
  }
  if (dev_out) *dev_out = dev;
  if (sm_out) *sm_out = sms;
  return SVDQ_OK;
}

constexpr int kMxMax = 1 << 20;
bool mx_k_ok(int K) { return K > 0 && K % 8 == 0 && K <= kMxMax; }
bool mx_n_ok(int N, int swiglu) { return N > 0 && N % (swiglu ? 16 : 8) == 0 && N <= kMxMax; }
int mx_k_pad(int K) { return (K + 255) / 256 * 256; }
int round_up(int x, int to) { return (x + to - 1) / to * to; }

// Tile width a weight is packed for: 384, which streams the fewest operand bytes per flop, unless padding N
// to it costs more than that gains over 256 (large M on B200, GEMM us at 256 / 384: 16896x3072x9216 211 / 197,
// 4608x12288x3072 62.5 / 57.0). The packing serves every M, so the wide tile loses where its tiles do not fill the SMs
// and 128-wide ones, which the same packing allows, do not all run at once (1024x3072x3072 10.4 / 12.0). SwiGLU pairs
// gate and up columns inside a tile of 256.
int mx_n_tile(int N, int swiglu) {
  if (swiglu) return 256;
  return round_up(N, 384) * 100ll <= round_up(N, 256) * 103ll ? 384 : 256;
}
int mx_n_pad(int N, int swiglu) {
  return swiglu ? round_up(N / 2, 128) * 2 : round_up(N, mx_n_tile(N, 0));
}

// Where the few-row kernels run (measured on B200 with weights from HBM; quantizer, product in us).
// The quantizer up to 384 rows with a branch (every group of 8 rows reads L1s^T again), up to 1024 without:
// K = 3072, r = 32: 3.9 (one row) to 8.6 (384) against kernel 1's 11.0, 14.9 / 11.1 at 512; K = 12288, r = 32:
// 7.8 to 24.1 against 26.3, 41 / 27 at 512; K = 1024, r = 32: 5.6 / 7.0 at 384; K = 3072, r = 0: 1.5 to 4.3 against
// 6.9, 7.2 / 6.6 at 2048; K = 1024, r = 0: 3.0 / 3.6 at 1024, 3.9 / 3.6 at 1536.
bool mx_few_quant_rows(int M, int K_pad, int r) {
  return r == 0 ? M <= 1024 : M <= 384 && K_pad <= kFewQuantMaxK;
}
// The product up to 32 rows, and up to 128 (SwiGLU 64) where splitting K over the SMs outweighs its epilogue of M x N
// sums, r = 32: 3072 -> 9216 7.7 against the pair GEMM's 9.3 at one row, 9.1 / 9.4 at 40, 10.0 / 9.5 at 64; 3072 -> 3072
// 6.9 / 8.3 at 64, 8.4 / 8.5 at 128; 12288 -> 3072 10.2 / 21.3 at one row, 13.3 / 21.7 at 128; 256 -> 9216 4.0 / 4.9 at 16,
// 5.4 / 5.0 at 40; 3072 -> 24576 with SwiGLU 12.8 / 16.2 at one row, 16.3 / 16.4 at 64.
// A CTA with a single K step (no branch and K split down to that) has little but the epilogue, which its cluster shares:
// up to 8 rows per CTA of the cluster, 16 at least, and while all blocks run at once: 256 -> 9216 3.1 / 4.7 at one row,
// 3.5 / 4.7 at 16, 256 -> 128 4.2 / 3.6 at 32, 256 -> 24576 6.9 / 6.0 at one row; 512 -> 3072 3.7 / 4.2 and 4.6 / 4.2 at
// 32; 1024 -> 1024 3.7 / 4.7, 4.5 / 4.8 at 32, 5.2 / 4.9 at 64; 2048 -> 1024 4.0 / 6.3, 5.4 / 6.4 at 64, 6.5 / 6.5 at 128;
// SwiGLU 256 -> 24576 4.1 / 7.2, 2048 -> 2048 4.6 / 7.3, 7.4 / 7.5 at 64.
struct FewSplit {
  int blocks, ranks;  // CTA clusters over N, and their size over K
};
FewSplit mx_few_split(const svdq_mx_weight* w, bool swiglu, int dev) {
  FewSplit s{swiglu ? w->N_pad / 256 : (w->N + 127) / 128, 1};
  std::lock_guard<std::mutex> lk(g_dev_mu);
  for (int i = 1; i < 4; ++i)
    if (s.blocks <= g_mx[dev].few_clusters[i] && (1 << i) <= w->K_pad / 256) s.ranks = 1 << i;
  return s;
}
bool mx_few_product_rows(int M, const svdq_mx_weight* w, bool swiglu, const FewSplit& s, int sms) {
  if (w->r == 0 && w->K_pad / 256 == s.ranks) return M <= (s.ranks > 2 ? 8 * s.ranks : 16) && s.blocks <= sms;
  return M <= 32 || (M <= svdq::mx::few_max_cols(swiglu ? 2 : 1) && 128ll * w->K_pad >= 1ll * M * w->N);
}

struct MxWeightLayout {
  size_t codes, scales, inv_lambda, l1t, l2t, total;
};
MxWeightLayout mx_weight_layout(int N_pad, int K_pad, int r) {
  MxWeightLayout l{};
  size_t off = 0;
  l.codes = off;
  off = align_up(off + static_cast<size_t>(N_pad) * K_pad / 2);
  l.scales = off;
  off = align_up(off + static_cast<size_t>(N_pad) * (K_pad / 32));
  l.inv_lambda = off;
  off = align_up(off + static_cast<size_t>(K_pad) * 4);
  l.l1t = off;
  off = align_up(off + static_cast<size_t>(r) * K_pad * 2);
  l.l2t = off;
  off = align_up(off + static_cast<size_t>(N_pad) * r * 2);
  l.total = off;
  return l;
}

struct MxActLayout {
  size_t codes, scales, u, total;
  int M_pad, K_pad;
};
MxActLayout mx_act_layout(int M, int K, int r) {
  MxActLayout l{};
  l.M_pad = round_up(M, 128);
  l.K_pad = mx_k_pad(K);
  size_t off = 0;
  l.codes = off;
  off = align_up(off + static_cast<size_t>(l.M_pad) * l.K_pad / 2);
  l.scales = off;
  off = align_up(off + static_cast<size_t>(l.M_pad) * (l.K_pad / 32));
  l.u = off;
  off = align_up(off + static_cast<size_t>(l.M_pad) * r * 2 * 2);  // hi and lo halves
  l.total = off;
  return l;
}

svdq_status check_mx_weight(const svdq_mx_weight* w) {
  const int sw = w->swiglu_interleaved;
  if ((sw != 0 && sw != 1) || !mx_n_ok(w->N, sw) || !mx_k_ok(w->K) || !valid_r(w->r) || w->n_tile != mx_n_tile(w->N, sw) ||
      w->N_pad != mx_n_pad(w->N, sw) || w->K_pad != mx_k_pad(w->K))
    return fail(SVDQ_ERR_INVALID_ARG,
                "MXFP4 weight descriptor N=%d K=%d r=%d n_tile=%d is not one svdq_mx_pack_weight makes", w->N, w->K,
                w->r, w->n_tile);
  if (w->codes == nullptr || w->scales == nullptr || w->inv_lambda == nullptr ||
      (w->r > 0 && (w->L1s_t == nullptr || w->L2_t == nullptr)))
    return fail(SVDQ_ERR_INVALID_ARG, "MXFP4 weight descriptor has a null buffer");
  return SVDQ_OK;
}

svdq_status check_mx_act(const svdq_mx_act* a) {
  if (a->M < 1 || a->M >= (1 << 24) || !mx_k_ok(a->K) || !valid_r(a->r) || a->M_pad != round_up(a->M, 128) ||
      a->K_pad != mx_k_pad(a->K))
    return fail(SVDQ_ERR_INVALID_ARG, "MXFP4 act descriptor M=%d M_pad=%d K=%d r=%d is not one svdq_mx_act_bind makes",
                a->M, a->M_pad, a->K, a->r);
  if (a->codes == nullptr || a->scales == nullptr || (a->r > 0 && a->U == nullptr))
    return fail(SVDQ_ERR_INVALID_ARG, "MXFP4 act descriptor has a null buffer");
  return SVDQ_OK;
}

// The few-row product of what mx_few_product_rows takes.
svdq_status mx_few_gemm(const svdq_mx_act* act, const svdq_mx_weight* w, const uint16_t* bias, bool has_bias, bool swiglu,
                        void* Y, long long ldy, int esize, const FewSplit& split, svdq_stream_t stream) {
  using namespace svdq::mx;
  static_assert(2 * few_stage_bytes(1, few_max_cols(1)) + few_part_bytes(1, few_max_cols(1)) + 1024 <= kFewMaxSmem &&
                    2 * few_stage_bytes(2, few_max_cols(2)) + few_part_bytes(2, few_max_cols(2)) + 1024 <= kFewMaxSmem,
                "two stages always fit");
  static_assert(few_max_cols(1) + kFewMaxStages * few_stage_tmem(1) <= 512 &&
                    2 * few_max_cols(2) + kFewMaxStages * few_stage_tmem(2) <= 512,
                "TMEM budget");
  const int NB = swiglu ? 2 : 1, r = w->r;
  const int cols = act->M <= 16 ? 16 : act->M <= 32 ? 32 : act->M <= 64 ? 64 : 128;
  const int blocks = split.blocks, ranks = split.ranks, steps = w->K_pad / 256;
  const int stage = few_stage_bytes(NB, cols);
  const int part = few_part_bytes(NB, cols);
  const int slots = (steps + ranks - 1) / ranks + (r + 31) / 32;
  int stages = (kFewMaxSmem - 1024 - part) / stage;
  if (stages > slots) stages = slots;  // one, where a CTA has a single K step and no branch
  if (stages > kFewMaxStages) stages = kFewMaxStages;
  int tmem = 32;
  while (tmem < NB * cols + stages * few_stage_tmem(NB)) tmem *= 2;
  CUtensorMap tmW, tmX, tmU, tmL2;
  std::memset(&tmU, 0, sizeof(tmU));
  std::memcpy(&tmW, &w->tmap[3][0], sizeof(CUtensorMap));
  std::memcpy(&tmL2, &w->tmap[4][0], sizeof(CUtensorMap));
  if (svdq_status s = make_tmap(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, act->codes, act->K_pad / 2, act->M_pad,
                                act->K_pad / 2, 128, cols, CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  if (r > 0) {
    if (svdq_status s = make_tmap(&tmU, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, act->U, r, 2 * static_cast<uint64_t>(act->M_pad),
                                  static_cast<uint64_t>(r) * 2, r < 32 ? r : 32, cols, lr_swizzle(r));
        s != SVDQ_OK)
      return s;
  }
  svdq::mx::FewGemmArgs g{};
  g.sfw = static_cast<const uint8_t*>(w->scales);
  g.sfx = static_cast<const uint8_t*>(act->scales);
  g.bias = reinterpret_cast<const __nv_bfloat16*>(bias);
  g.Y = Y;
  g.ldy = ldy;
  g.wait_ns = g_wait_ns.load();
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
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  set_programmatic(attr[1]);
  cfg.gridDim = dim3(blocks * ranks, 1, 1);
  cfg.blockDim = dim3(svdq::mx::kFewThreads, 1, 1);
  const int smem = stages * stage + part + 1024;
  cfg.dynamicSmemBytes = static_cast<size_t>(smem < kFewMinSmem ? kFewMinSmem : smem);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, NB == 2 ? svdq::mx::few_gemm_kernel<2> : svdq::mx::few_gemm_kernel<1>,
                                           tmW, tmX, tmU, tmL2, g);
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of mx::few_gemm_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("mx::few_gemm_kernel");
}

svdq_status mx_fill_weight(uint8_t* b, int N, int K, int r, int swiglu, svdq_mx_weight* out) {
  svdq_mx_weight w{};
  w.N = N;
  w.K = K;
  w.r = r;
  w.swiglu_interleaved = swiglu ? 1 : 0;
  w.n_tile = mx_n_tile(N, swiglu);
  w.N_pad = mx_n_pad(N, swiglu);
  w.K_pad = mx_k_pad(K);
  const MxWeightLayout l = mx_weight_layout(w.N_pad, w.K_pad, r);
  w.codes = b + l.codes;
  w.scales = b + l.scales;
  w.inv_lambda = reinterpret_cast<float*>(b + l.inv_lambda);
  w.L1s_t = b + l.l1t;
  w.L2_t = b + l.l2t;
  static_assert(sizeof(w.tmap) >= 5 * sizeof(CUtensorMap), "tmap storage");
  CUtensorMap tmB, tmL2, tmL1, tmB64, tmL264;
  std::memset(&tmL264, 0, sizeof(tmL264));
  std::memset(&tmL2, 0, sizeof(tmL2));
  std::memset(&tmL1, 0, sizeof(tmL1));
  if (svdq_status s = make_tmap(&tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, w.K_pad / 2, w.N_pad, w.K_pad / 2, 128,
                                w.n_tile / 2, CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  // the same in boxes of 64 rows: the few-row product's blocks of 128 tile columns
  if (svdq_status s = make_tmap(&tmB64, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, w.K_pad / 2, w.N_pad, w.K_pad / 2, 128, 64,
                                CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  if (r > 0) {
    if (svdq_status s = make_tmap(&tmL264, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w.L2_t, r, w.N_pad,
                                  static_cast<uint64_t>(r) * 2, r < 32 ? r : 32, 64, lr_swizzle(r));
        s != SVDQ_OK)
      return s;
    if (svdq_status s = make_tmap(&tmL2, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w.L2_t, r, w.N_pad,
                                  static_cast<uint64_t>(r) * 2, r < 32 ? r : 32, w.n_tile / 2, lr_swizzle(r));
        s != SVDQ_OK)
      return s;
    if (svdq_status s = make_tmap(&tmL1, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w.L1s_t, w.K_pad, r,
                                  static_cast<uint64_t>(w.K_pad) * 2, 64, r, CU_TENSOR_MAP_SWIZZLE_128B);
        s != SVDQ_OK)
      return s;
  }
  std::memcpy(&w.tmap[0][0], &tmB, sizeof(CUtensorMap));
  std::memcpy(&w.tmap[1][0], &tmL2, sizeof(CUtensorMap));
  std::memcpy(&w.tmap[2][0], &tmL1, sizeof(CUtensorMap));
  std::memcpy(&w.tmap[3][0], &tmB64, sizeof(CUtensorMap));
  std::memcpy(&w.tmap[4][0], &tmL264, sizeof(CUtensorMap));
  *out = w;
  return SVDQ_OK;
}

}  // namespace

extern "C" {

size_t svdq_mx_weight_bytes(int N, int K, int r, int swiglu) {
  if (!mx_n_ok(N, swiglu) || !mx_k_ok(K) || !valid_r(r)) return 0;
  return mx_weight_layout(mx_n_pad(N, swiglu), mx_k_pad(K), r).total;
}

size_t svdq_mx_act_bytes(int M, int K, int r) {
  if (M < 1 || M >= (1 << 24) || !mx_k_ok(K) || !valid_r(r)) return 0;
  return mx_act_layout(M, K, r).total;
}

svdq_status svdq_mx_act_bind(int M, int K, int r, void* dst, size_t dst_bytes, svdq_mx_act* out) {
  if (out == nullptr || dst == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  const size_t need = svdq_mx_act_bytes(M, K, r);
  if (need == 0) return fail(SVDQ_ERR_UNSUPPORTED, "MXFP4 act shape M=%d K=%d r=%d unsupported", M, K, r);
  if (dst_bytes < need) return fail(SVDQ_ERR_INVALID_ARG, "MXFP4 act buffer %zu bytes < %zu", dst_bytes, need);
  if (reinterpret_cast<uintptr_t>(dst) % kAlign) return fail(SVDQ_ERR_UNSUPPORTED, "act buffer not 256-byte aligned");
  const MxActLayout l = mx_act_layout(M, K, r);
  uint8_t* b = static_cast<uint8_t*>(dst);
  svdq_mx_act a{};
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

svdq_status svdq_mx_pack_weight(const float* R_nk, const uint16_t* L1s_kr, const uint16_t* L2_rn,
                                const float* inv_lambda, int N, int K, int r, int swiglu, void* dst, size_t dst_bytes,
                                svdq_mx_weight* out, svdq_stream_t stream) {
  if (out == nullptr || R_nk == nullptr || dst == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (r > 0 && (L1s_kr == nullptr || L2_rn == nullptr)) return fail(SVDQ_ERR_INVALID_ARG, "null L1s / L2 with r > 0");
  const size_t need = svdq_mx_weight_bytes(N, K, r, swiglu);
  if (need == 0) return fail(SVDQ_ERR_UNSUPPORTED, "MXFP4 weight shape N=%d K=%d r=%d unsupported", N, K, r);
  if (!aligned16(R_nk) || (r > 0 && (!aligned16(L1s_kr) || !aligned16(L2_rn))) ||
      (reinterpret_cast<uintptr_t>(inv_lambda) & 3u))
    return fail(SVDQ_ERR_UNSUPPORTED, "inputs must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(dst) % kAlign) return fail(SVDQ_ERR_UNSUPPORTED, "dst not 256-byte aligned");
  if (dst_bytes < need) return fail(SVDQ_ERR_INVALID_ARG, "MXFP4 weight buffer %zu bytes < %zu", dst_bytes, need);
  int dev, sms;
  if (svdq_status s = mx_ready(&dev, &sms); s != SVDQ_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  svdq_mx_weight w{};
  if (svdq_status s = mx_fill_weight(static_cast<uint8_t*>(dst), N, K, r, swiglu, &w); s != SVDQ_OK) return s;
  SVDQ_CUDA(cudaMemsetAsync(dst, 0, need, st));  // padded rows and columns
  svdq::mx::fill_inv_lambda_kernel<<<grid_for(w.K_pad, 256, sms), 256, 0, st>>>(inv_lambda, K, w.K_pad, w.inv_lambda);
  if (svdq_status s = check_launch("mx::fill_inv_lambda_kernel"); s != SVDQ_OK) return s;
  svdq::mx::pack_quant_kernel<<<grid_for(static_cast<size_t>(N) * w.K_pad / 8, 256, sms), 256, 0, st>>>(
      R_nk, N, K, w.K_pad, w.n_tile, w.swiglu_interleaved, static_cast<uint8_t*>(w.codes),
      static_cast<uint8_t*>(w.scales));
  if (svdq_status s = check_launch("mx::pack_quant_kernel"); s != SVDQ_OK) return s;
  if (r > 0) {
    svdq::mx::transpose_l1_kernel<<<grid_for(static_cast<size_t>(w.K_pad) * r, 256, sms), 256, 0, st>>>(
        reinterpret_cast<const __nv_bfloat16*>(L1s_kr), K, w.K_pad, r, static_cast<__nv_bfloat16*>(w.L1s_t));
    if (svdq_status s = check_launch("mx::transpose_l1_kernel"); s != SVDQ_OK) return s;
    svdq::mx::pack_l2_kernel<<<grid_for(static_cast<size_t>(N) * r, 256, sms), 256, 0, st>>>(
        reinterpret_cast<const __nv_bfloat16*>(L2_rn), N, r, w.n_tile, w.swiglu_interleaved,
        static_cast<__nv_bfloat16*>(w.L2_t));
    if (svdq_status s = check_launch("mx::pack_l2_kernel"); s != SVDQ_OK) return s;
  }
  *out = w;
  return SVDQ_OK;
}

svdq_status svdq_mx_weight_bind(int N, int K, int r, int swiglu, void* blob, size_t blob_bytes, svdq_mx_weight* out) {
  if (out == nullptr || blob == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  const size_t need = svdq_mx_weight_bytes(N, K, r, swiglu);
  if (need == 0) return fail(SVDQ_ERR_UNSUPPORTED, "MXFP4 weight shape N=%d K=%d r=%d unsupported", N, K, r);
  if (reinterpret_cast<uintptr_t>(blob) % kAlign) return fail(SVDQ_ERR_UNSUPPORTED, "blob not 256-byte aligned");
  if (blob_bytes < need) return fail(SVDQ_ERR_INVALID_ARG, "MXFP4 weight blob %zu bytes < %zu", blob_bytes, need);
  if (svdq_status s = mx_ready(nullptr, nullptr); s != SVDQ_OK) return s;
  return mx_fill_weight(static_cast<uint8_t*>(blob), N, K, r, swiglu, out);
}

svdq_status svdq_mx_quantize_act(const uint16_t* X, long long ldx, const svdq_mx_weight* w, const svdq_mx_act* act,
                                 svdq_stream_t stream) {
  if (X == nullptr || w == nullptr || act == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (act->K != w->K || act->r != w->r)
    return fail(SVDQ_ERR_INVALID_ARG, "act (K=%d r=%d) does not match weight (K=%d r=%d)", act->K, act->r, w->K, w->r);
  if (svdq_status s = check_mx_weight(w); s != SVDQ_OK) return s;
  if (svdq_status s = check_mx_act(act); s != SVDQ_OK) return s;
  if (!aligned16(X)) return fail(SVDQ_ERR_UNSUPPORTED, "X must be 16-byte aligned");
  if (ldx < act->K || ldx % 8 != 0 || ldx >= (1ll << 38))
    return fail(SVDQ_ERR_UNSUPPORTED, "row stride %lld of X: a multiple of 8 and at least K=%d", ldx, act->K);
  int dev, sms;
  if (svdq_status s = mx_ready(&dev, &sms); s != SVDQ_OK) return s;
  const int r = w->r;
  if (mx_few_quant_rows(act->M, act->K_pad, r)) {
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
    // rows per cluster: the fewest that keep all clusters on the SMs at once (K = 12288, r = 32: one row
    // per cluster 7.8 us, eight 15.8 us)
    f.rows = 1;
    while (f.rows < 8 && (act->M + f.rows - 1) / f.rows * svdq::mx::kFewQuantCluster > sms) f.rows *= 2;
    const int x_smem = r > 0 ? f.rows * (act->K_pad / svdq::mx::kFewQuantCluster) * 2 : 0;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = svdq::mx::kFewQuantCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    set_programmatic(attr[1]);
    cfg.gridDim = dim3((act->M + f.rows - 1) / f.rows * svdq::mx::kFewQuantCluster, 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.dynamicSmemBytes = static_cast<size_t>(x_smem);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg,
                                             r == 0    ? svdq::mx::few_quant_kernel<0>
                                             : r == 16 ? svdq::mx::few_quant_kernel<16>
                                             : r == 32 ? svdq::mx::few_quant_kernel<32>
                                                       : svdq::mx::few_quant_kernel<64>,
                                             f);
    if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of mx::few_quant_kernel failed: %s", cudaGetErrorString(e));
    return check_launch("mx::few_quant_kernel");
  }
  CUtensorMap tmX, tmL1;
  std::memcpy(&tmL1, &w->tmap[2][0], sizeof(CUtensorMap));
  if (svdq_status s = make_tmap(&tmX, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, X, act->K, act->M,
                                static_cast<uint64_t>(ldx) * 2, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  // K split over a cluster as for the NVFP4 kernel 1 (the same kernel body and resources)
  const int m_tiles = act->M_pad / 128;
  int csize = 1;
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    const int* mc = g_dev[dev].k1_clusters[r == 0 ? 0 : r == 16 ? 1 : r == 32 ? 2 : 3];
    for (int c = 2; c <= 4; ++c)
      if (m_tiles <= mc[c - 1] && act->K_pad % (64 * c) == 0) csize = c;
  }
  svdq::mx::ActArgs a;
  a.inv_lambda = w->inv_lambda;
  a.codes = static_cast<uint8_t*>(act->codes);
  a.sf = static_cast<uint8_t*>(act->scales);
  a.U = static_cast<__nv_bfloat16*>(act->U);
  a.wait_ns = g_wait_ns.load();
  a.M = act->M;
  a.K = act->K_pad;
  a.M_pad = act->M_pad;
  a.k_per_cta = act->K_pad / csize;

  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = csize;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  set_programmatic(attr[1]);
  cfg.gridDim = dim3(m_tiles * csize, 1, 1);
  cfg.blockDim = dim3(svdq::kQ1Threads, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaSuccess;
  switch (r) {
    case 0:
      cfg.dynamicSmemBytes = svdq::Q1Layout<0>::kSmem;
      e = cudaLaunchKernelEx(&cfg, svdq::quant_act_kernel<0, svdq::mx::Act>, tmX, tmL1, a);
      break;
    case 16:
      cfg.dynamicSmemBytes = svdq::Q1Layout<16>::kSmem;
      e = cudaLaunchKernelEx(&cfg, svdq::quant_act_kernel<16, svdq::mx::Act>, tmX, tmL1, a);
      break;
    case 32:
      cfg.dynamicSmemBytes = svdq::Q1Layout<32>::kSmem;
      e = cudaLaunchKernelEx(&cfg, svdq::quant_act_kernel<32, svdq::mx::Act>, tmX, tmL1, a);
      break;
    default:
      cfg.dynamicSmemBytes = svdq::Q1Layout<64>::kSmem;
      e = cudaLaunchKernelEx(&cfg, svdq::quant_act_kernel<64, svdq::mx::Act>, tmX, tmL1, a);
      break;
  }
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of the MXFP4 quant_act_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("quant_act_kernel (MXFP4)");
}

}  // extern "C"

namespace {

svdq_status check_mx_gemm(const svdq_mx_act* act, const svdq_mx_weight* w, const uint16_t* bias, svdq_epilogue epi,
                          const void* Y, long long ldy, svdq_out_dtype out_dtype) {
  if (act == nullptr || w == nullptr || Y == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (act->K != w->K || act->r != w->r) return fail(SVDQ_ERR_INVALID_ARG, "act does not match weight");
  if (svdq_status s = check_mx_weight(w); s != SVDQ_OK) return s;
  if (svdq_status s = check_mx_act(act); s != SVDQ_OK) return s;
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

// svdq_mx_gemm on checked arguments.
svdq_status mx_gemm(const svdq_mx_act* act, const svdq_mx_weight* w, const uint16_t* bias, svdq_epilogue epi, void* Y,
                    long long ldy, svdq_out_dtype out_dtype, svdq_stream_t stream) {
  const bool has_bias = (epi & 1) != 0, swiglu = (epi & 2) != 0;
  const int n_out = swiglu ? w->N / 2 : w->N, esize = out_dtype == SVDQ_OUT_F32 ? 4 : 2;
  int dev, sms;
  if (svdq_status s = mx_ready(&dev, &sms); s != SVDQ_OK) return s;

  if (const FewSplit split = mx_few_split(w, swiglu, dev); mx_few_product_rows(act->M, w, swiglu, split, sms))
    return mx_few_gemm(act, w, bias, has_bias, swiglu, Y, ldy, esize, split, stream);
  const int r = w->r, n_tile = w->n_tile;
  CUtensorMap tmA, tmU, tmB, tmL2, tmY;
  std::memset(&tmU, 0, sizeof(tmU));
  if (svdq_status s = make_tmap(&tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, act->codes, act->K_pad / 2, act->M_pad,
                                act->K_pad / 2, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B);
      s != SVDQ_OK)
    return s;
  if (r > 0) {
    if (svdq_status s = make_tmap(&tmU, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, act->U, r, 2 * static_cast<uint64_t>(act->M_pad),
                                  static_cast<uint64_t>(r) * 2, r < 32 ? r : 32, 128, lr_swizzle(r));
        s != SVDQ_OK)
      return s;
  }
  std::memcpy(&tmB, &w->tmap[0][0], sizeof(CUtensorMap));
  std::memcpy(&tmL2, &w->tmap[1][0], sizeof(CUtensorMap));
  // columns past n_out and rows past M are clipped by the store
  if (svdq_status s = make_tmap(&tmY, esize == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, Y,
                                n_out, act->M, static_cast<uint64_t>(ldy) * esize, 32, 32,
                                esize == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
      s != SVDQ_OK)
    return s;

  svdq::mx::GemmArgs g{};
  g.sfa = static_cast<const uint8_t*>(act->scales);
  g.sfb = static_cast<const uint8_t*>(w->scales);
  g.bias = reinterpret_cast<const __nv_bfloat16*>(bias);
  g.wait_ns = g_wait_ns.load();
  g.M = act->M;
  g.M_pad = act->M_pad;
  g.N = w->N;
  g.K = w->K_pad;
  g.r = r;
  g.m_tiles = act->M_pad / 128;
  g.m_pairs = (g.m_tiles + 1) / 2;
  g.k_iters = w->K_pad / 256;
  g.out_f32 = esize == 4 ? 1 : 0;
  g.epi = static_cast<int>(epi);
  g.n_tile = n_tile;
  // 128-wide tiles where all of them run at once: more SMs share the work of a small layer (us at 128 / the
  // packed width: 512x3072x3072 8.8 / 11.3, 1024x1024x768 5.2 / 7.5; with two rounds of them, 300x3072x9216,
  // 14.7 / 12.3). SwiGLU's column pairs need the packed tile.
  int tile = n_tile, max_pairs = 0;
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    const int* most = g_mx[dev].max_pairs;
    if (!swiglu && static_cast<long long>(g.m_pairs) * ((w->N + 127) / 128) <= most[2]) tile = 128;
    max_pairs = most[tile == 384 ? 0 : tile == 256 ? 1 : 2];
  }
  g.n_tiles = swiglu ? w->N_pad / 256 : (w->N + tile - 1) / tile;
  g.num_tiles = g.m_pairs * g.n_tiles;
  if (tile != n_tile) {  // boxes of 64 rows
    std::memcpy(&tmB, &w->tmap[3][0], sizeof(CUtensorMap));
    std::memcpy(&tmL2, &w->tmap[4][0], sizeof(CUtensorMap));
  }
  const int pairs = g.num_tiles < max_pairs ? g.num_tiles : max_pairs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (tile == 384)
    e = launch_pair_gemm(svdq::pair_gemm_kernel<svdq::mx::Gemm, 384, kMxStages384>, 2 * pairs,
                         MxLayout<384, kMxStages384>::kSmem, st, tmA, tmB, tmU, tmL2, tmY, g);
  else if (tile == 256)
    e = launch_pair_gemm(svdq::pair_gemm_kernel<svdq::mx::Gemm, 256, kMxStages256>, 2 * pairs,
                         MxLayout<256, kMxStages256>::kSmem, st, tmA, tmB, tmU, tmL2, tmY, g);
  else
    e = launch_pair_gemm(svdq::pair_gemm_kernel<svdq::mx::Gemm, 128, kMxStages128>, 2 * pairs,
                         MxLayout<128, kMxStages128>::kSmem, st, tmA, tmB, tmU, tmL2, tmY, g);
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of pair_gemm_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("pair_gemm_kernel (MXFP4)");
}

}  // namespace

extern "C" {

svdq_status svdq_mx_gemm(const svdq_mx_act* act, const svdq_mx_weight* w, const uint16_t* bias, svdq_epilogue epi,
                         void* Y, long long ldy, svdq_out_dtype out_dtype, svdq_stream_t stream) {
  if (svdq_status s = check_mx_gemm(act, w, bias, epi, Y, ldy, out_dtype); s != SVDQ_OK) return s;
  return mx_gemm(act, w, bias, epi, Y, ldy, out_dtype, stream);
}

svdq_status svdq_mx_linear(const uint16_t* X, long long ldx, const svdq_mx_weight* w, const svdq_mx_act* act,
                           const uint16_t* bias, svdq_epilogue epi, void* Y, long long ldy, svdq_out_dtype out_dtype,
                           svdq_stream_t stream) {
  if (svdq_status s = check_mx_gemm(act, w, bias, epi, Y, ldy, out_dtype); s != SVDQ_OK) return s;
  if (svdq_status s = svdq_mx_quantize_act(X, ldx, w, act, stream); s != SVDQ_OK) return s;
  return mx_gemm(act, w, bias, epi, Y, ldy, out_dtype, stream);
}

svdq_status svdq_mx_export_weight(const svdq_mx_weight* w, uint8_t* codes, uint8_t* scales, svdq_stream_t stream) {
  if (w == nullptr || codes == nullptr || scales == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_mx_weight(w); s != SVDQ_OK) return s;
  if (reinterpret_cast<uintptr_t>(codes) & 3u) return fail(SVDQ_ERR_UNSUPPORTED, "codes must be 4-byte aligned");
  int dev, sms;
  if (svdq_status s = mx_ready(&dev, &sms); s != SVDQ_OK) return s;
  svdq::mx::export_kernel<<<grid_for(static_cast<size_t>(w->N) * (w->K / 8), 256, sms), 256, 0,
                            static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(w->codes), static_cast<const uint8_t*>(w->scales), w->N, w->K, w->K_pad, w->n_tile,
      w->swiglu_interleaved, codes, scales);
  return check_launch("mx::export_kernel");
}

svdq_status svdq_mx_export_act(const svdq_mx_act* act, uint8_t* codes, uint8_t* scales, svdq_stream_t stream) {
  if (act == nullptr || codes == nullptr || scales == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_mx_act(act); s != SVDQ_OK) return s;
  if (reinterpret_cast<uintptr_t>(codes) & 3u) return fail(SVDQ_ERR_UNSUPPORTED, "codes must be 4-byte aligned");
  int dev, sms;
  if (svdq_status s = mx_ready(&dev, &sms); s != SVDQ_OK) return s;
  svdq::mx::export_kernel<<<grid_for(static_cast<size_t>(act->M) * (act->K / 8), 256, sms), 256, 0,
                            static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(act->codes), static_cast<const uint8_t*>(act->scales), act->M, act->K, act->K_pad, 0,
      0, codes, scales);
  return check_launch("mx::export_kernel");
}

svdq_status svdq_mx_dequantize_act(const svdq_mx_act* act, void* out, long long ld, svdq_out_dtype out_dtype,
                                   svdq_stream_t stream) {
  if (act == nullptr || out == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_mx_act(act); s != SVDQ_OK) return s;
  if (out_dtype != SVDQ_OUT_BF16 && out_dtype != SVDQ_OUT_F32) return fail(SVDQ_ERR_INVALID_ARG, "bad out dtype");
  if (!aligned16(out)) return fail(SVDQ_ERR_UNSUPPORTED, "out must be 16-byte aligned");
  if (ld < act->K || ld % 8 != 0)
    return fail(SVDQ_ERR_UNSUPPORTED, "row stride %lld of out: a multiple of 8 and at least K=%d", ld, act->K);
  int dev, sms;
  if (svdq_status s = mx_ready(&dev, &sms); s != SVDQ_OK) return s;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  set_programmatic(attr[0]);
  cfg.gridDim = dim3((act->M + svdq::mx::kDeqRows - 1) / svdq::mx::kDeqRows, (act->K / 8 + 255) / 256, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto* kern = out_dtype == SVDQ_OUT_F32 ? svdq::mx::dequantize_act_kernel<true> : svdq::mx::dequantize_act_kernel<false>;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<const uint8_t*>(act->codes),
                                           static_cast<const uint8_t*>(act->scales), act->M, act->K, act->K_pad, out, ld);
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of mx::dequantize_act_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("mx::dequantize_act_kernel");
}

}  // extern "C"

// ================================================================== block norms
namespace {

constexpr int kNormMaxD = 32768;

bool bad_norm(const svdq_norm& n) {
  return n.kind < SVDQ_NORM_NONE || n.kind > SVDQ_NORM_LAYER || (n.f32 != 0 && n.f32 != 1) ||
         (n.kind != SVDQ_NORM_NONE && !(n.eps >= 0.0f));
}
bool misaligned(const void* p, int f32) { return (reinterpret_cast<uintptr_t>(p) & (f32 ? 3u : 1u)) != 0; }

// The bytes of an activation: `samples` blocks, ss apart, of `rows` rows of `row` bytes, ls apart.
struct Span {
  uintptr_t lo, hi;
  uintptr_t row, ls, block, ss;
  bool even;  // one run of rows, ls apart throughout
  Span(const void* p, const svdq_block_norm_args* a, long long ld, long long sample, int f32) {
    const uintptr_t e = f32 ? 4 : 2;
    even = a->offsets != nullptr || sample == 0 || a->M <= a->rows_per_sample;
    const long long rows = even ? a->M : a->rows_per_sample, samples = even ? 1 : (a->M + rows - 1) / rows;
    row = a->D * e;
    ls = ld * e;
    block = (rows - 1) * ls + row;
    ss = even ? block : sample * e;
    lo = reinterpret_cast<uintptr_t>(p);
    hi = lo + (samples - 1) * ss + block;
  }
  // Whether two may share a byte: not if their ranges are apart, or if one lies in columns (or in a slice
  // of a sample) that the other leaves out throughout.
  bool overlaps(const Span& o) const {
    if (hi <= o.lo || o.hi <= lo) return false;
    const auto beside = [](uintptr_t p, uintptr_t n, uintptr_t q, uintptr_t m, uintptr_t period) {
      const uintptr_t d = q >= p ? (q - p) % period : (period - (p - q) % period) % period;
      return d >= n && d + m <= period;
    };
    if (ls == o.ls && (even || ss % ls == 0) && (o.even || o.ss % ls == 0) && beside(lo, row, o.lo, o.row, ls))
      return false;
    return !(ss == o.ss && ss > block && beside(lo, block, o.lo, o.block, ss));
  }
};

svdq_status check_norm_args(const svdq_block_norm_args* a, bool quant) {
  if (a == nullptr || a->x == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (a->M < 0 || a->M >= (1 << 24) || a->D < 1) return fail(SVDQ_ERR_INVALID_ARG, "block norm of %d rows of %d", a->M, a->D);
  if (a->D > kNormMaxD) return fail(SVDQ_ERR_UNSUPPORTED, "block norm rows of %d values (at most %d)", a->D, kNormMaxD);
  const int flags[] = {a->x_f32, a->y_f32, a->h_f32, a->mod_f32};
  for (int f : flags)
    if (f != 0 && f != 1) return fail(SVDQ_ERR_INVALID_ARG, "a type flag is neither 0 nor 1");
  if (a->samples < 1 || (a->offsets == nullptr && a->rows_per_sample < 1))
    return fail(SVDQ_ERR_INVALID_ARG, "block norm of %d samples of %d rows", a->samples, a->rows_per_sample);
  if (a->offsets == nullptr && a->M > 0 && (a->M - 1) / a->rows_per_sample >= a->samples)
    return fail(SVDQ_ERR_INVALID_ARG, "%d rows are more than %d samples of %d", a->M, a->samples, a->rows_per_sample);
  if (bad_norm(a->post) || bad_norm(a->norm)) return fail(SVDQ_ERR_INVALID_ARG, "bad norm kind, eps or type flag");
  const bool wants_h = quant || a->h != nullptr;
  if (wants_h != (a->norm.kind != SVDQ_NORM_NONE))
    return fail(SVDQ_ERR_INVALID_ARG, wants_h ? "h without a norm" : "a norm without h");
  if (!wants_h && (a->scale != nullptr || a->shift != nullptr))
    return fail(SVDQ_ERR_INVALID_ARG, "scale and shift without h");
  if (a->y == nullptr && (a->x_out != nullptr || a->gate != nullptr || a->post.kind != SVDQ_NORM_NONE))
    return fail(SVDQ_ERR_INVALID_ARG, "x_out, gate or a post norm without y");
  if (!wants_h && a->x_out == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "no output");
  const struct { const void* p; long long ld, ss; } acts[] = {
      {a->x, a->ldx, a->sx}, {a->y, a->ldy, a->sy}, {a->x_out, a->ld_out, a->s_out}, {a->h, a->ldh, a->sh}};
  for (const auto& t : acts) {
    if (t.p == nullptr) continue;
    if (t.ld < a->D || t.ld >= (1ll << 38))
      return fail(SVDQ_ERR_INVALID_ARG, "row stride %lld for rows of %d", t.ld, a->D);
    if (t.ss != 0 && (a->offsets != nullptr || t.ss < (a->rows_per_sample - 1) * t.ld + a->D || t.ss >= (1ll << 38)))
      return fail(SVDQ_ERR_INVALID_ARG, "sample stride %lld", t.ss);
  }
  const long long mods[] = {a->gate ? a->ld_gate : 0, a->scale ? a->ld_scale : 0, a->shift ? a->ld_shift : 0};
  for (long long ld : mods)
    if (ld < 0 || ld >= (1ll << 38)) return fail(SVDQ_ERR_INVALID_ARG, "sample stride %lld", ld);
  if (misaligned(a->x, a->x_f32) || misaligned(a->y, a->y_f32) || misaligned(a->x_out, a->x_f32) ||
      misaligned(a->h, a->h_f32) || misaligned(a->gate, a->mod_f32) || misaligned(a->scale, a->mod_f32) ||
      misaligned(a->shift, a->mod_f32) || misaligned(a->post.weight, a->post.f32) ||
      misaligned(a->post.bias, a->post.f32) || misaligned(a->norm.weight, a->norm.f32) ||
      misaligned(a->norm.bias, a->norm.f32) || misaligned(a->offsets, 1))
    return fail(SVDQ_ERR_UNSUPPORTED, "a pointer is not aligned to its element");
  if (a->M > 0) {
    // rows are read once, by the threads that write x_out's: x_out may be x, nothing else may overlap
    const Span x(a->x, a, a->ldx, a->sx, a->x_f32);
    if (a->x_out != nullptr) {
      const Span o(a->x_out, a, a->ld_out, a->s_out, a->x_f32);
      if (o.overlaps(x) && !(a->x_out == a->x && a->ld_out == a->ldx && o.ss == x.ss))
        return fail(SVDQ_ERR_INVALID_ARG, "x_out overlaps x without being x");
      if (o.overlaps(Span(a->y, a, a->ldy, a->sy, a->y_f32))) return fail(SVDQ_ERR_INVALID_ARG, "x_out overlaps y");
    }
    if (a->h != nullptr) {
      const Span h(a->h, a, a->ldh, a->sh, a->h_f32);
      if (h.overlaps(x) || (a->y != nullptr && h.overlaps(Span(a->y, a, a->ldy, a->sy, a->y_f32))) ||
          (a->x_out != nullptr && h.overlaps(Span(a->x_out, a, a->ld_out, a->s_out, a->x_f32))))
        return fail(SVDQ_ERR_INVALID_ARG, "h overlaps x, y or x_out");
    }
  }
  return SVDQ_OK;
}

// Every row and vector starts on a 16-byte boundary and holds whole groups of 8: the 16-byte path.
bool norm_vectorised(const svdq_block_norm_args* a) {
  if (a->D % 8 != 0) return false;
  const struct { const void* p; long long ld; int f32; } rows[] = {
      {a->x, a->sx, a->x_f32},          {a->y, a->sy, a->y_f32},           {a->x_out, a->s_out, a->x_f32},
      {a->h, a->sh, a->h_f32},          {a->x, a->ldx, a->x_f32},         {a->y, a->ldy, a->y_f32},          {a->x_out, a->ld_out, a->x_f32},
      {a->h, a->ldh, a->h_f32},         {a->gate, a->ld_gate, a->mod_f32}, {a->scale, a->ld_scale, a->mod_f32},
      {a->shift, a->ld_shift, a->mod_f32}, {a->post.weight, 0, 0},         {a->post.bias, 0, 0},
      {a->norm.weight, 0, 0},           {a->norm.bias, 0, 0}};
  for (const auto& v : rows)
    if (v.p != nullptr && (!aligned16(v.p) || (v.ld * (v.f32 ? 4 : 2)) % 16 != 0)) return false;
  return true;
}

svdq::norm::Norm to_norm(const svdq_norm& n) {
  svdq::norm::Norm o{};
  o.kind = n.kind;
  o.eps = n.eps;
  o.w = {n.weight, 0, n.f32};
  o.b = {n.bias, 0, n.f32};
  return o;
}

// The instantiations of the 16-byte kernel: C chunks of 8 per thread and R rows at a time; x's type, y's
// (or none), a quantized output or not.
using NormKernel = void (*)(svdq::norm::Args, int, int, int, unsigned long long);
constexpr int norm_batch(int chunks) { return chunks == 1 ? 4 : chunks == 2 ? 2 : 1; }
template <bool XF32, int Y, bool QUANT>
NormKernel norm_kernel(int chunks, bool share) {
  using namespace svdq::norm;
  if (!share)
    return chunks <= 2   ? block_norm_kernel<2, norm_batch(2), XF32, Y, QUANT, false>
           : chunks <= 6 ? block_norm_kernel<6, norm_batch(6), XF32, Y, QUANT, false>
                         : block_norm_kernel<8, norm_batch(8), XF32, Y, QUANT, false>;
  switch (chunks) {
    case 1: return block_norm_kernel<1, norm_batch(1), XF32, Y, QUANT, true>;
    case 2: return block_norm_kernel<2, norm_batch(2), XF32, Y, QUANT, true>;
    case 4: return block_norm_kernel<4, norm_batch(4), XF32, Y, QUANT, true>;
    default: return block_norm_kernel<6, norm_batch(6), XF32, Y, QUANT, true>;  // eight leave no room for factors
  }
}
template <bool XF32, bool QUANT>
NormKernel norm_kernel(int chunks, bool share, int y) {
  using namespace svdq::norm;
  return y == kNoY    ? norm_kernel<XF32, kNoY, QUANT>(chunks, share)
         : y == kF32Y ? norm_kernel<XF32, kF32Y, QUANT>(chunks, share)
                      : norm_kernel<XF32, kBf16Y, QUANT>(chunks, share);
}
NormKernel norm_kernel(int chunks, bool share, bool x_f32, int y, bool quant) {
  if (quant) return x_f32 ? norm_kernel<true, true>(chunks, share, y) : norm_kernel<false, true>(chunks, share, y);
  return x_f32 ? norm_kernel<true, false>(chunks, share, y) : norm_kernel<false, false>(chunks, share, y);
}
// Quantized forms whose shared factors leave no room for the smoothing reciprocals: rows of bf16 x and y in
// (8192, 12288], rows of x alone in (12288, 16384].
NormKernel norm_kernel_far_lambdas(bool x_f32, int y) {
  using namespace svdq::norm;
  if (y != kNoY) return block_norm_kernel<6, norm_batch(6), false, kBf16Y, true, true, false>;
  return x_f32 ? block_norm_kernel<4, norm_batch(4), true, kNoY, true, true, false>
               : block_norm_kernel<4, norm_batch(4), false, kNoY, true, true, false>;
}
cudaError_t launch_norm_any(const cudaLaunchConfig_t& cfg, int chunks, const svdq::norm::Args& k, int G) {
  switch (chunks) {
    case 1: return cudaLaunchKernelEx(&cfg, svdq::norm::block_norm_any_kernel<1>, k, G);
    case 2: return cudaLaunchKernelEx(&cfg, svdq::norm::block_norm_any_kernel<2>, k, G);
    case 4: return cudaLaunchKernelEx(&cfg, svdq::norm::block_norm_any_kernel<4>, k, G);
    case 6: return cudaLaunchKernelEx(&cfg, svdq::norm::block_norm_any_kernel<6>, k, G);
    default: return cudaLaunchKernelEx(&cfg, svdq::norm::block_norm_any_kernel<8>, k, G);
  }
}

constexpr int kNormSmem = 212 * 1024;  // the most a block's rings take
// fp32 x and y wider than this (six chunks for each of 512 threads) do not fit them: the element-wise kernel's
// rows, and refused with a quantized output. All other rows up to kNormMaxD fit.
constexpr int kNormMaxF32Pair = 6 * 512 * 8;
static_assert(kNormMaxF32Pair * 8 <= kNormSmem && kNormMaxD * 6 <= kNormSmem, "rows that fit");
struct NormState {
  bool ready = false;
};
NormState g_norm[64];

svdq_status norm_setup() {
  for (int chunks : {1, 2, 4, 6, 8})
    for (int v = 0; v < 24; ++v)
      SVDQ_CUDA(cudaFuncSetAttribute(norm_kernel(chunks, v >= 12, v & 1, (v >> 1) % 3, (v / 6) & 1),
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem));
  for (int v = 0; v < 3; ++v)
    SVDQ_CUDA(cudaFuncSetAttribute(norm_kernel_far_lambdas(v == 1, v == 2 ? svdq::norm::kBf16Y : svdq::norm::kNoY),
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kNormSmem));
  return SVDQ_OK;
}
svdq_status norm_ready(int* sm_out) {
  int dev = 0;
  if (svdq_status s = device_ready(&dev, sm_out); s != SVDQ_OK) return s;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  if (!g_norm[dev].ready) {
    if (svdq_status s = norm_setup(); s != SVDQ_OK) return s;
    g_norm[dev].ready = true;
  }
  return SVDQ_OK;
}

svdq_status run_norm(const svdq_block_norm_args* a, const svdq_mx_weight* w, const svdq_mx_act* act, bool vec,
                     int sms, svdq_stream_t stream) {
  svdq::norm::Args k{};
  k.x = a->x;
  k.y = a->y;
  k.x_out = a->x_out;
  k.h = a->h;
  k.ldx = a->ldx;
  k.ldy = a->ldy;
  k.ld_out = a->ld_out;
  k.ldh = a->ldh;
  const auto adj = [&](long long ss, long long ld) { return ss == 0 ? 0 : ss - a->rows_per_sample * ld; };
  k.adj_x = adj(a->sx, a->ldx);
  k.adj_y = adj(a->sy, a->ldy);
  k.adj_out = adj(a->s_out, a->ld_out);
  k.adj_h = adj(a->sh, a->ldh);
  k.x_f32 = a->x_f32;
  k.y_f32 = a->y_f32;
  k.h_f32 = a->h_f32;
  k.M = a->M;
  k.D = a->D;
  k.rows = act ? act->M_pad : a->M;
  k.samples = a->samples;
  k.rows_per_sample = a->offsets ? 0 : a->rows_per_sample;
  k.per_sample = a->offsets || a->rows_per_sample == 1 ? 0 : ~0ull / a->rows_per_sample + 1;
  k.offsets = a->offsets;
  k.skip = a->skip_scale;
  k.res = a->res_scale;
  k.gate = {a->gate, a->ld_gate, a->mod_f32};
  k.scale = {a->scale, a->ld_scale, a->mod_f32};
  k.shift = {a->shift, a->ld_shift, a->mod_f32};
  k.post = to_norm(a->post);
  k.pre = to_norm(a->norm);
  if (act) {
    k.inv_lambda = w->inv_lambda;
    k.codes = static_cast<uint8_t*>(act->codes);
    k.sf = static_cast<uint8_t*>(act->scales);
    k.K_pad = act->K_pad;
  }
  const int eights = ((act ? act->K_pad : a->D) + 7) / 8;
  const auto whole = [](int c) { return c <= 2 ? c : c <= 4 ? 4 : c <= 6 ? 6 : 8; };
  // warps per row for at most `most` chunks of 8 values per thread
  const auto row_warps = [&](int most) {
    const int w = (eights + 32 * most - 1) / (32 * most);
    return svdq::norm::kMaxWarps / (w < svdq::norm::kMaxWarps ? svdq::norm::kMaxWarps / w : 1);  // leaves no warp over
  };
  int W = row_warps(6), chunks = whole((eights + 32 * W - 1) / (32 * W));
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  set_programmatic(attr[0]);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int elem_bytes = (a->x_f32 ? 4 : 2) + (a->y == nullptr ? 0 : a->y_f32 ? 4 : 2);
  cudaError_t e;
  if (vec) {
    const auto stage_bytes = [&] { return norm_batch(chunks) * chunks * 256 * W * elem_bytes; };
    const auto factor_bytes = [&] { return chunks * 256 * W * (a->y ? 12 : 8); };
    // Factors of a run's sample in shared memory where a run gives every group two batches and the SMs have
    // more than two rows each; else (or where they do not fit beside a batch) two, six or eight chunks per
    // thread and vectors read per row, which with few rows is sooner done: 24 and 296 rows of 3072, gate, post-norm,
    // residual and norm 6.4 and 6.9 us against 7.2 with shared factors, quantized 7.5 against 9.0 (24 rows),
    // a norm alone 3.7 against 4.9; at 400 rows 7.6 / 7.3 and 4.5 / 5.1, at 600 rows 10.4 / 7.4 and 5.7 / 5.2.
    const int per_run = a->offsets ? a->M / a->samples : a->rows_per_sample;
    const bool share = a->M > 2 * sms && per_run >= 2 * (svdq::norm::kMaxWarps / W) * norm_batch(chunks) &&
                       stage_bytes() + factor_bytes() <= kNormSmem;
    // a quantized output's smoothing reciprocals, where the shared factors leave room for them
    int lambda_bytes = act && share ? chunks * 256 * W * 4 : 0;
    const bool far_lambdas = act && share && stage_bytes() + factor_bytes() + lambda_bytes > kNormSmem;
    if (far_lambdas) lambda_bytes = 0;
    if (!share) {
      W = row_warps(2);
      const int need = (eights + 32 * W - 1) / (32 * W);
      chunks = need <= 2 ? 2 : need <= 6 ? 6 : 8;
    }
    if (stage_bytes() <= kNormSmem) {  // but for fp32 x and y wider than kNormMaxF32Pair
      // Rows in flight per SM: as many groups as fit a block, but no more than about 80 KB of batches; a
      // second stage where that leaves room for one. Measured on B200 over two samples of 16896 rows of
      // 3072, all bf16 (12 KB of x and y): 6 groups 137 us, 8 groups 157 us, 4 groups 171 us, 6 groups with
      // two stages 138 us; without y (6 KB) over 4608 rows: 8 groups 13.2 us, 6 groups 15.2 us, 8 groups with
      // two stages 13.9 us; 4000 rows of 8192 without y (2 groups, 32 KB): one stage 33.8 us, two 32.1 us.
      // More groups, up to 128 KB, for a quantized output, which is bound by its instructions (16896 rows of
      // 3072 with y: 6 groups 91 us, 8 groups 79 us), and where the call's bytes about fit the L2, so that the
      // rounds of rows count, and rows fill the groups (with y, bf16, from HBM: 1000 rows 11.0 -> 9.8 us, 4608
      // 27.8 -> 25.5, 6000 32.8 / 32.8; x fp32: 3000 29.2 -> 27.3, 4608 37.5 / 37.6, 8448 60.5 / 66.6; bf16 from
      // L2, 600 rows 7.5 / 8.3).
      // Two sets of factors where they cost no group.
      const long long bytes = 1ll * a->M * a->D * (elem_bytes + (a->x_out == nullptr ? 0 : a->x_f32 ? 4 : 2) +
                                                   (a->h == nullptr ? 0 : a->h_f32 ? 4 : 2));
      const bool more = act || (bytes <= 160ll * 1000 * 1000 && a->M > 6 * sms);
      const int in_flight = (more ? 128 : 80) * 1024, R = norm_batch(chunks), batches = (k.rows + R - 1) / R;
      int groups = svdq::norm::kMaxWarps / W, fixed = share ? factor_bytes() + lambda_bytes : 0;
      while (groups > 1 && (groups * stage_bytes() > in_flight || groups * stage_bytes() + fixed > kNormSmem)) --groups;
      if (!share)
        while (groups > 1 && (groups - 1) * sms >= batches) --groups;  // few rows: over all SMs
      const int sets = share && groups * stage_bytes() + fixed + factor_bytes() <= kNormSmem ? 2 : 1;
      if (sets == 2) fixed += factor_bytes();
      const int stages =
          2 * groups * stage_bytes() <= 80 * 1024 && 2 * groups * stage_bytes() + fixed <= kNormSmem ? 2 : 1;
      const int blocks = (batches + groups - 1) / groups;
      cfg.gridDim = dim3(blocks < sms ? blocks : sms, 1, 1);
      cfg.blockDim = dim3(groups * 32 * W, 1, 1);
      cfg.dynamicSmemBytes = static_cast<size_t>(groups) * stages * stage_bytes() + fixed;
      const int y = a->y == nullptr ? svdq::norm::kNoY : 1 + a->y_f32;
      e = cudaLaunchKernelEx(&cfg,
                             far_lambdas ? norm_kernel_far_lambdas(a->x_f32, y)
                                         : norm_kernel(chunks, share, a->x_f32, y, act != nullptr),
                             k, 32 * W, stages, sets, g_wait_ns.load());
      if (e != cudaSuccess)
        return fail(SVDQ_ERR_CUDA, "launch of norm::block_norm_kernel failed: %s", cudaGetErrorString(e));
      return check_launch("norm::block_norm_kernel");
    }
  }
  W = row_warps(1);
  chunks = whole((eights + 32 * W - 1) / (32 * W));
  const int groups = W >= 4 ? 1 : 4 / W;
  cfg.gridDim = dim3(grid_for(k.rows, groups, sms), 1, 1);
  cfg.blockDim = dim3(groups * 32 * W, 1, 1);
  e = launch_norm_any(cfg, chunks, k, 32 * W);
  if (e != cudaSuccess) return fail(SVDQ_ERR_CUDA, "launch of norm::block_norm_kernel failed: %s", cudaGetErrorString(e));
  return check_launch("norm::block_norm_kernel");
}

}  // namespace

extern "C" {

svdq_status svdq_block_norm(const svdq_block_norm_args* a, svdq_stream_t stream) {
  if (svdq_status s = check_norm_args(a, false); s != SVDQ_OK) return s;
  int sms;
  if (svdq_status s = norm_ready(&sms); s != SVDQ_OK) return s;
  if (a->M == 0) return SVDQ_OK;
  return run_norm(a, nullptr, nullptr, norm_vectorised(a), sms, stream);
}

svdq_status svdq_block_norm_quantize_mx(const svdq_block_norm_args* a, const svdq_mx_weight* w, const svdq_mx_act* act,
                                        svdq_stream_t stream) {
  if (w == nullptr || act == nullptr) return fail(SVDQ_ERR_INVALID_ARG, "null pointer");
  if (svdq_status s = check_norm_args(a, true); s != SVDQ_OK) return s;
  if (svdq_status s = check_mx_weight(w); s != SVDQ_OK) return s;
  if (svdq_status s = check_mx_act(act); s != SVDQ_OK) return s;
  if (act->M != a->M || act->K != a->D || w->K != a->D)
    return fail(SVDQ_ERR_INVALID_ARG, "act (M=%d K=%d) and weight (K=%d) do not match %d rows of %d", act->M, act->K,
                w->K, a->M, a->D);
  if (act->r != 0 || w->r != 0)
    return fail(SVDQ_ERR_UNSUPPORTED, "a branch of rank %d projects h: use svdq_block_norm and svdq_mx_quantize_act",
                w->r ? w->r : act->r);
  if (!norm_vectorised(a)) return fail(SVDQ_ERR_UNSUPPORTED, "a quantized output needs 16-byte aligned rows and vectors");
  if (a->y != nullptr && a->x_f32 && a->y_f32 && a->D > kNormMaxF32Pair)
    return fail(SVDQ_ERR_UNSUPPORTED, "fp32 rows of x and y of %d values (at most %d with a quantized output)", a->D,
                kNormMaxF32Pair);
  int sms;
  if (svdq_status s = norm_ready(&sms); s != SVDQ_OK) return s;
  return run_norm(a, w, act, true, sms, stream);
}

}  // extern "C"
