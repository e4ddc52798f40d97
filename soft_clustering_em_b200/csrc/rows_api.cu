// rows_api.cu -- host side of gmm_logprobs, gmm_logprobs_backward and gmm_route:
// argument checks and launches.
#include <math.h>

#include <algorithm>

#include "api_common.h"
#include "rows.cuh"

using namespace scem;

namespace {

constexpr int32_t kMaxRowClasses = 1 << 24;
constexpr int kShortRow = 1024;  // classes a warp holds in registers

size_t row_elem(int32_t t) { return t == GMM_F32 ? 4 : 2; }

gmm_status check_rows(const gmm_rows* r, const void* Z) {
  if (!r) return GMM_ERR_INVALID_ARG;
  if (r->N < 0 || r->K < 1 || r->ld < r->K) return GMM_ERR_INVALID_ARG;
  if (r->dtype != GMM_F32 && r->dtype != GMM_BF16 && r->dtype != GMM_F16)
    return GMM_ERR_INVALID_ARG;
  if (!(r->scale > 0.f) || !isfinite(r->scale)) return GMM_ERR_INVALID_ARG;
  if (!isfinite(r->scale * kLog2e)) return GMM_ERR_UNSUPPORTED;
  if (r->K > kMaxRowClasses) return GMM_ERR_UNSUPPORTED;
  if (r->N > ((int64_t)1 << 40) || r->ld > ((int64_t)1 << 40) ||
      (double)r->N * (double)r->ld > 1e18)
    return GMM_ERR_UNSUPPORTED;
  if (r->N == 0) return GMM_OK;
  if (!Z) return GMM_ERR_INVALID_ARG;
  if ((uintptr_t)Z % row_elem(r->dtype) != 0) return GMM_ERR_UNSUPPORTED;
  return GMM_OK;
}

template <typename T, int kLanes, int kEl>
void short_launch(const RowArgs& a, bool vec, cudaStream_t st) {
  const int64_t rows = 8 * (32 / kLanes);
  const unsigned grid = (unsigned)std::min<int64_t>((a.N + rows - 1) / rows, 1 << 24);
  if (vec)
    row_short_kernel<T, kLanes, kEl, true><<<grid, 256, 0, st>>>(a);
  else
    row_short_kernel<T, kLanes, kEl, false><<<grid, 256, 0, st>>>(a);
}

// CTAs per long row, 1, 2, 4 or 8: the fewest microseconds by a model of what was measured.  A
// call takes `rounds` turns of the resident CTAs.  A turn is a slice at 27 or 40 GB/s a CTA, or at
// its share of the memory bandwidth, and a fixed part: the joining of sums and alternatives,
// dearer across a cluster, and dearer the fuller the SMs are.  (64 rows of 131,072 bf16 with
// 20 alternatives: 20.4 us on one CTA each, 17.0 on four; 592 rows of 4,096: 10.5 on one, 77
// on four.)
int row_cluster(int64_t N, double row_bytes, int m, int slots) {
  int best = 1;
  double best_us = 1e30;
  for (int C = 1; C <= 8; C *= 2) {
    if (C > 1 && row_bytes / C < 4096) break;
    const int64_t rounds = (N * C + slots - 1) / slots;
    const double active = (double)std::min<int64_t>(N * C, slots);
    const double full = active / slots;
    const double rate = std::min(m > 0 ? 27e3 : 40e3, 6.5e6 / active);  // bytes per us
    const double join = C == 1 ? (m > 0 ? 6.0 + 0.18 * m : 3.0) * (0.7 + 0.3 * full)
                               : (m > 0 ? 11.0 + 0.2 * m : 7.0) * (0.4 + 0.6 * full);
    const double us = rounds * (row_bytes / C / rate + join);
    if (us < best_us) best = C, best_us = us;
  }
  return best;
}

template <typename T>
gmm_status rows_launch(const RowArgs& a, cudaStream_t st) {
  int sms = 0;
  gmm_status s = api_device_sms(&sms);
  if (s != GMM_OK) return s;
  if (a.K <= kShortRow) {
    const bool vec = (uintptr_t)a.Z % 16 == 0 && (a.ld * sizeof(T)) % 16 == 0;
    if (a.K <= 256 && a.N <= 16 * sms)
      short_launch<T, 32, 8>(a, vec, st);
    else if (a.K <= 64)
      short_launch<T, 8, 8>(a, vec, st);
    else if (a.K <= 128)
      short_launch<T, 8, 16>(a, vec, st);
    else if (a.K <= 256)
      short_launch<T, 8, 32>(a, vec, st);
    else if (a.K <= 512)
      short_launch<T, 16, 32>(a, vec, st);
    else
      short_launch<T, 32, 32>(a, vec, st);
    return api_launched(1);
  }
  constexpr int smem = kRowWarps * kRowStages * kRowStep * 16;
  auto kern = a.m > 0 ? row_long_kernel<T, true> : row_long_kernel<T, false>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return api_launched(0), GMM_ERR_CUDA;
  int C = row_cluster(a.N, (double)a.K * sizeof(T), a.m, kRowCtas * sms);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(a.N * C, kRowCtas * sms / C * C));
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = C > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kern, a, C) != cudaSuccess) return api_launched(0), GMM_ERR_CUDA;
  return api_launched(1);
}

gmm_status rows_dispatch(const gmm_rows* r, const RowArgs& a, void* stream) {
  cudaStream_t st = (cudaStream_t)stream;
  if (r->dtype == GMM_F32) return rows_launch<float>(a, st);
  if (r->dtype == GMM_BF16) return rows_launch<__nv_bfloat16>(a, st);
  return rows_launch<__half>(a, st);
}

template <typename T>
gmm_status grad_launch(RowGradArgs a, cudaStream_t st) {
  if (a.K <= 2048) {
    int sms = 0;
    gmm_status s = api_device_sms(&sms);
    if (s != GMM_OK) return s;
    a.slices = 1;
    a.blocks = (unsigned)std::min<int64_t>((a.N + 7) / 8, 1 << 24);
    row_grad_kernel<T, 32><<<a.blocks + std::min(a.blocks, 4u * sms), 256, 0, st>>>(a);
  } else {
    const int per = 4 * 4 * 256 * Vec16<T>::n;  // four batches of a CTA
    a.slices = (a.K + per - 1) / per;
    a.blocks = (unsigned)std::min<int64_t>(a.N * a.slices, 1 << 24);
    row_grad_kernel<T, 256><<<a.blocks, 256, 0, st>>>(a);
  }
  return api_launched(1);
}

}  // namespace

extern "C" {

gmm_status gmm_logprobs(const gmm_rows* r, const void* Z, const int32_t* ids, int32_t m,
                        float* logp, float* entropy, float* lse, int32_t* top_idx,
                        float* top_logp, uint32_t* dev_flags, void* stream) {
  gmm_status s = check_rows(r, Z);
  if (s != GMM_OK) return s;
  if (m < 0 || m > kMaxAlt) return GMM_ERR_INVALID_ARG;
  if (r->N == 0) return GMM_OK;
  if ((ids != nullptr) != (logp != nullptr)) return GMM_ERR_INVALID_ARG;
  if (m > 0 && (!top_idx || !top_logp)) return GMM_ERR_INVALID_ARG;
  if (m == 0 && !logp && !entropy && !lse) return GMM_ERR_INVALID_ARG;
  RowArgs a = {Z,   r->N, r->ld, r->K,    r->scale, ids, m, logp, entropy,
               lse, top_idx, top_logp, 0, dev_flags};
  return rows_dispatch(r, a, stream);
}

gmm_status gmm_route(const gmm_rows* r, const void* Z, int32_t m, int32_t renorm, int32_t* idx,
                     float* resp, uint32_t* dev_flags, void* stream) {
  gmm_status s = check_rows(r, Z);
  if (s != GMM_OK) return s;
  if (m < 1 || m > kMaxTopM || m > r->K) return GMM_ERR_INVALID_ARG;
  if (r->N == 0) return GMM_OK;
  if (!idx || !resp) return GMM_ERR_INVALID_ARG;
  RowArgs a = {Z,       r->N,    r->ld, r->K, r->scale,       nullptr,  m, nullptr, nullptr,
               nullptr, idx, resp,  renorm ? 2 : 1, dev_flags};
  return rows_dispatch(r, a, stream);
}

gmm_status gmm_logprobs_backward(const gmm_rows* r, const void* Z, const int32_t* ids,
                                 const float* lse, const float* entropy, const float* dlogp,
                                 const float* dentropy, const float* dlse, int32_t m,
                                 const int32_t* top_idx, const float* dtop, void* dZ, int64_t ldd,
                                 uint32_t* dev_flags, void* stream) {
  gmm_status s = check_rows(r, Z);
  if (s != GMM_OK) return s;
  if (m < 0 || m > kMaxAlt || ldd < r->K) return GMM_ERR_INVALID_ARG;
  if (ldd > ((int64_t)1 << 40) || (double)r->N * (double)ldd > 1e18) return GMM_ERR_UNSUPPORTED;
  if (r->N == 0) return GMM_OK;
  if (!lse || !dZ) return GMM_ERR_INVALID_ARG;
  if (dlogp && !ids) return GMM_ERR_INVALID_ARG;
  if (dentropy && !entropy) return GMM_ERR_INVALID_ARG;
  if (m > 0 && (!top_idx || !dtop)) return GMM_ERR_INVALID_ARG;
  if (!dlogp && !dentropy && !dlse && m == 0) return GMM_ERR_INVALID_ARG;
  if (dZ == Z && ldd != r->ld) return GMM_ERR_INVALID_ARG;
  if ((uintptr_t)dZ % row_elem(r->dtype) != 0) return GMM_ERR_UNSUPPORTED;
  RowGradArgs a = {Z,   dZ,      r->N,  r->ld,    ldd,  r->K, 1,  0, r->scale,
                   ids, lse,     entropy, dlogp, dentropy, dlse, m,    top_idx, dtop, dev_flags};
  cudaStream_t st = (cudaStream_t)stream;
  if (r->dtype == GMM_F32) return grad_launch<float>(a, st);
  if (r->dtype == GMM_BF16) return grad_launch<__nv_bfloat16>(a, st);
  return grad_launch<__half>(a, st);
}

}  // extern "C"
