// moe_api.cu -- host side of gmm_moe: argument checks, workspace layout and launches.
#include <algorithm>
#include <atomic>

#include "api_common.h"
#include "moe.cuh"
#include "tma_host.h"

using namespace scem;

namespace {

gmm_status check_moe(const gmm_moe_problem* p) {
  if (!p) return GMM_ERR_INVALID_ARG;
  if (p->T < 0 || p->D < 1 || p->F < 1 || p->E < 1 || p->m < 1 || p->m > kMaxTopM)
    return GMM_ERR_INVALID_ARG;
  if (p->dtype != GMM_F32 && p->dtype != GMM_BF16 && p->dtype != GMM_F16)
    return GMM_ERR_INVALID_ARG;
  if (p->act != GMM_ACT_SILU && p->act != GMM_ACT_GELU) return GMM_ERR_INVALID_ARG;
  if (p->ldx < p->D || p->ldy < p->D) return GMM_ERR_INVALID_ARG;
  if (p->dtype == GMM_F32) return GMM_ERR_UNSUPPORTED;
  if (p->T > kMoeMaxT || p->E > kMoeMaxE) return GMM_ERR_UNSUPPORTED;
  if (p->D % 8 != 0 || p->F % 8 != 0 || p->ldx % 8 != 0) return GMM_ERR_UNSUPPORTED;
  if (p->D > (1 << 20) || p->F > (1 << 20) || p->ldx >= ((int64_t)1 << 39) ||  // (a tensor map's row
      p->ldy > ((int64_t)1 << 40))                                              // stride: 2^40 bytes)
    return GMM_ERR_UNSUPPORTED;
  if ((int64_t)p->E * 2 * p->F >= ((int64_t)1 << 31) || (int64_t)p->E * p->D >= ((int64_t)1 << 31))
    return GMM_ERR_UNSUPPORTED;
  return GMM_OK;
}

// Workspace: status word, then h: T * m rows of F hi halves, and as many of lo halves.
constexpr size_t kMoeH = 256;

size_t moe_bytes(const gmm_moe_problem* p) {
  return kMoeH + 2 * align_up((size_t)p->T * p->m * p->F * 2, 256);
}

// A launch that may start while the kernel before it in the stream ends: both kernels wait
// (griddepcontrol) before they touch what it wrote.
template <typename Kern, typename... Args>
bool launch(Kern kern, unsigned grid, int cluster, int smem, cudaStream_t st, Args... args) {
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return false;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kMoeThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

constexpr int kMoeSmem = 227 * 1024;

// Shared memory for the stages behind the fixed parts.
int ring_bytes(int fixed) { return kMoeSmem - fixed - 1024; }

constexpr int kMostFixed = moe_fixed(kMoeMaxE, kMoeMaxSlots);
static_assert(moe_stages(kMoeSmem - 1024 - kMostFixed - kMoeMaxT * kMoeTile * 4, true, 16,
                         kMoeTile) > 0 &&
                  moe_stages(kMoeSmem - 1024 - kMostFixed - kMoeSwap, false, 64, kMoeTile) > 0,
              "a ring at the most tokens");

// How many clusters of C of the down kernel's CTAs (one per SM) are resident at once: they do not
// pack the GPCs (148, 74, 45, 33, 26, 22, 15, 15 for C = 1..8 on 148 SMs).  Asked once per device.
template <typename T>
int down_clusters(int device, int C) {
  static std::atomic<int> known[64][9];
  const bool keep = device >= 0 && device < 64;
  if (keep)
    if (int n = known[device][C].load()) return n;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C);
  cfg.blockDim = dim3(kMoeThreads);
  cfg.dynamicSmemBytes = kMoeSmem;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaFuncSetAttribute(moe_down_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kMoeSmem) != cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, moe_down_kernel<T>, &cfg) != cudaSuccess || n < 1)
    return 0;
  if (keep) known[device][C] = n;
  return n;
}

// Rows of y per cluster (a multiple of 8 up to 128) and CTAs per cluster (which share out the
// experts): the least time of a CTA, whose step costs by its rows but not below those of about
// 56, by its tokens, and by how much less than 56 KB of weights its ring holds, among the shapes
// whose clusters are all resident at once (one more would take a second turn: 58 us instead of 42
// for 32 tokens).  No odd clusters: 43 of the 45 resident clusters of 3 take 228 us where 37 take
// 183 and 22 of 6 take 172 (32 tokens, 8 of 128 experts of 2048 x 768).  The model is fitted to
// few shapes: for 256 tokens of 16 experts it took one that needed 133 us where clusters of 4 with
// 72 rows needed 119.
template <typename T>
bool down_shape(const gmm_moe_problem* p, int sms, int* C, int* rows) {
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return false;
  const int experts = std::min(p->E, p->T * p->m), fixed = moe_fixed(p->E, p->T * p->m);
  *C = 1;
  *rows = kMoeTile;
  double best = 1e30;
  const double tokens = std::min(32.0, (double)p->T * p->m / experts);
  for (int c = 1; c <= 8 && c <= experts; c += c == 1 ? 1 : 2) {
    const int fit = c == 1 ? sms : down_clusters<T>(device, c);
    if (fit < 1) return false;
    for (int r = 8; r <= kMoeTile; r += 8) {
      if ((p->D + r - 1) / r > fit) continue;
      const int stages =
          moe_stages(ring_bytes(fixed + p->T * r * 4), true, tokens > 16 ? 32 : 16, r);
      const double cost = ((experts + c - 1) / c) * (std::max(r, 56) + 8 + 2 * tokens) *
                              std::max(1.0, 56.0 * 1024 / (128 * r * std::max(stages, 1))) +
                          0.01 * c;
      if (cost < best) best = cost, *C = c, *rows = r;
    }
  }
  return true;
}

template <typename T>
gmm_status moe_launch(const gmm_moe_problem* p, MoeArgs a, const void* X, const void* W_up,
                      const void* W_down, cudaStream_t st) {
  int sms = 0;
  gmm_status s = api_device_sms(&sms);
  if (s != GMM_OK) return s;
  int C = 1;
  if (!down_shape<T>(p, sms, &C, &a.block_rows)) return api_launched(0), GMM_ERR_CUDA;
  CUtensorMap up64, up16, down, x1, h1;
  const uint64_t D = p->D, F = p->F, E = p->E, slots = (uint64_t)p->T * p->m;
  if (!make_tmap_16b_sw128(&up64, W_up, D, E * 2 * F, D * 2, 64) ||
      !make_tmap_16b_sw128(&up16, W_up, D, E * 2 * F, D * 2, 16) ||
      !make_tmap_16b_sw128(&down, W_down, F, E * D, F * 2, a.block_rows) ||
      !make_tmap_16b_sw128(&x1, X, D, p->T, (uint64_t)p->ldx * 2, 1) ||
      !make_tmap_16b_sw128(&h1, a.h_hi, F, 2 * slots, F * 2, 1))
    return GMM_ERR_CUDA;
  a.wait_ns = api_wait_budget();
  const int fixed = moe_fixed(p->E, p->T * p->m), up_fixed = fixed + kMoeSwap;
  a.ring_bytes = ring_bytes(up_fixed);
  if (!launch(moe_up_kernel<T>, sms, 1, up_fixed + 1024 + a.ring_bytes, st, a, up64, up16,
              x1))
    return api_launched(0), GMM_ERR_CUDA;
  if ((s = api_launched(1)) != GMM_OK) return s;
  const int blocks = (p->D + a.block_rows - 1) / a.block_rows;
  const int down_fixed = fixed + p->T * a.block_rows * 4;
  a.ring_bytes = ring_bytes(down_fixed);
  if (!launch(moe_down_kernel<T>, blocks * C, C, down_fixed + 1024 + a.ring_bytes, st, a, C, down,
              h1))
    return api_launched(0), GMM_ERR_CUDA;
  return api_launched(1);
}

}  // namespace

extern "C" {

gmm_status gmm_moe_workspace_size(const gmm_moe_problem* p, size_t* bytes) {
  gmm_status s = check_moe(p);
  if (s != GMM_OK) return s;
  if (!bytes) return GMM_ERR_INVALID_ARG;
  *bytes = moe_bytes(p);
  return GMM_OK;
}

gmm_status gmm_moe(const gmm_moe_problem* p, const void* X, const int32_t* idx, const float* resp,
                   const void* W_up, const void* W_down, void* Y, void* ws, size_t ws_bytes,
                   void* stream) {
  gmm_status s = check_moe(p);
  if (s != GMM_OK) return s;
  if (p->T == 0) return GMM_OK;
  if (!X || !idx || !resp || !W_up || !W_down || !Y) return GMM_ERR_INVALID_ARG;
  if ((uintptr_t)X % 16 != 0 || (uintptr_t)W_up % 16 != 0 || (uintptr_t)W_down % 16 != 0 ||
      (uintptr_t)Y % 2 != 0)
    return GMM_ERR_UNSUPPORTED;
  if (!ws || (uintptr_t)ws % 256 != 0 || ws_bytes < moe_bytes(p)) return GMM_ERR_WORKSPACE;
  char* hi = (char*)ws + kMoeH;
  char* lo = hi + (size_t)p->T * p->m * p->F * 2;
  MoeArgs a = {Y,    idx,  resp,   hi,     lo, p->T, p->m, p->E,
               p->D, p->F, p->ldy, p->act, 0,  0,    0,    (unsigned int*)ws};
  cudaStream_t st = (cudaStream_t)stream;
  if (p->dtype == GMM_BF16) return moe_launch<__nv_bfloat16>(p, a, X, W_up, W_down, st);
  return moe_launch<__half>(p, a, X, W_up, W_down, st);
}

}  // extern "C"
