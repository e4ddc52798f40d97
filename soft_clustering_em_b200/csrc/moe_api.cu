// moe_api.cu -- host side of gmm_moe: argument checks, workspace layout and launches.
#include <algorithm>

#include "api_common.h"
#include "moe.cuh"

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
  if (p->D > (1 << 20) || p->F > (1 << 20) || p->ldx > ((int64_t)1 << 40) ||
      p->ldy > ((int64_t)1 << 40))
    return GMM_ERR_UNSUPPORTED;
  return GMM_OK;
}

// Workspace: status word, then h as hi and lo halves, T * m rows of F each.
struct MoeLayout {
  size_t hi, lo, total;
};

MoeLayout moe_layout(const gmm_moe_problem* p) {
  MoeLayout L;
  const size_t h = align_up((size_t)p->T * p->m * p->F * 2, 256);
  L.hi = 256;
  L.lo = L.hi + h;
  L.total = L.lo + h;
  return L;
}

template <typename T>
gmm_status moe_launch(const gmm_moe_problem* p, MoeArgs a, cudaStream_t st) {
  int sms = 0;
  gmm_status s = api_device_sms(&sms);
  if (s != GMM_OK) return s;
  moe_up_kernel<T><<<2 * sms, kMoeThreads, 0, st>>>(a);
  if ((s = api_launched(1)) != GMM_OK) return s;
  a.row_blocks = (p->D + kMoeRows - 1) / kMoeRows;
  const size_t smem = (size_t)p->T * kMoeRows * kMoeWarps * 4;
  auto kern = moe_down_kernel<T>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
      cudaSuccess)
    return api_launched(0), GMM_ERR_CUDA;
  kern<<<a.row_blocks, kMoeThreads, smem, st>>>(a, 1);
  return api_launched(1);
}

}  // namespace

extern "C" {

gmm_status gmm_moe_workspace_size(const gmm_moe_problem* p, size_t* bytes) {
  gmm_status s = check_moe(p);
  if (s != GMM_OK) return s;
  if (!bytes) return GMM_ERR_INVALID_ARG;
  *bytes = moe_layout(p).total;
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
  const MoeLayout L = moe_layout(p);
  if (!ws || (uintptr_t)ws % 256 != 0 || ws_bytes < L.total) return GMM_ERR_WORKSPACE;
  char* b = (char*)ws;
  MoeArgs a = {X,      W_up, W_down, Y,    idx,    resp,   b + L.hi, b + L.lo, p->T,
               p->m,   p->E, p->D,   p->F, p->ldx, p->ldy, p->act,   0,        (unsigned int*)ws};
  cudaStream_t st = (cudaStream_t)stream;
  if (p->dtype == GMM_BF16) return moe_launch<__nv_bfloat16>(p, a, st);
  return moe_launch<__half>(p, a, st);
}

}  // extern "C"
