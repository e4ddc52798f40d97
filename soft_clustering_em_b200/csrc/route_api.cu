// route_api.cu -- host side of gmm_route_loss and gmm_route_backward: argument checks and
// launches.
#include <float.h>
#include <math.h>

#include <algorithm>

#include "api_common.h"
#include "route.cuh"

using namespace scem;

namespace {

constexpr int32_t kMostSegments = 1 << 20;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

size_t elem(int32_t t) { return t == GMM_F32 ? 4 : 2; }

gmm_status check_route(const gmm_rows* r, int32_t m, int32_t S) {
  if (!r) return GMM_ERR_INVALID_ARG;
  if (r->N < 0 || r->K < 1 || r->ld < r->K || m < 1 || m > kMaxTopM || S < 0)
    return GMM_ERR_INVALID_ARG;
  if (r->dtype != GMM_F32 && r->dtype != GMM_BF16 && r->dtype != GMM_F16)
    return GMM_ERR_INVALID_ARG;
  if (!(r->scale > 0.f) || !isfinite(r->scale)) return GMM_ERR_INVALID_ARG;
  if (!isfinite(r->scale * kLog2e) || r->K > kRouteMostK || S > kMostSegments ||
      r->N >= ((int64_t)1 << 31) / m || r->ld > kMaxStride ||
      (double)r->N * (double)r->ld > 1e18)
    return GMM_ERR_UNSUPPORTED;
  return GMM_OK;
}

// CTAs of the loss and the rows of each: at least 32 rows, or about a segment's where those are
// shorter (a CTA takes a segment after the other, 1 us each), and three CTAs on each of 148 SMs at
// most, or whole turns of those: a lane adds up at most 512 rows in float32 before the pieces' sums
// are joined in 64 bits.  (Like terms round one way: 2^28 rows of 12 logits of 0 in 444 pieces, 18,893
// additions a lane, gave a load that was off by 1e-4.)
struct LossPlan {
  int64_t chunks, rows;
};
constexpr int64_t kLossAdds = 512;
LossPlan loss_plan(int64_t N, int32_t S, int K) {
  LossPlan p;
  p.chunks = std::max<int64_t>((N + 31) / 32, std::min<int64_t>(N, S));
  p.chunks = std::max<int64_t>(1, std::min<int64_t>(p.chunks, 444));
  const int64_t most = kLossAdds * kRouteWarps * (K <= 128 ? 4 : K <= 256 ? 2 : 1);
  p.chunks *= std::max<int64_t>(1, (N + p.chunks * most - 1) / (p.chunks * most));
  p.rows = std::max<int64_t>(1, (N + p.chunks - 1) / p.chunks);
  return p;
}

size_t loss_bytes(const gmm_rows* r, int32_t S) {
  return (size_t)(loss_plan(r->N, S, r->K).chunks + std::max(S, 1)) * route_slot(r->K) * 4;
}

// How rows of K classes are taken (route_vec).
template <typename T>
int route_mode(bool aligned, int K) {
  return !aligned ? 0 : K % Vec16<T>::n != 0 ? 1 : 2;
}

// Whether the rows are few enough for one launch, a cluster of CTAs per segment, in `*direct`: 6
// turns of its warps at most (8, should one of several segments have all).  CTAs: as many as that
// takes, and one for each two turns of an average segment, up to 8 and to what is resident at
// once.  (fp32, by one launch and by two: 512 rows of 64 4.6 and 7.0 us, 1,536 6.9 and 7.4, in 5
// segments 5.1 and 8.8; 512 of 256 6.8 and 8.0, but 1,024 of those in 8 turns 9.3 and 8.1.)
template <typename T, int kLanes, int kEl>
gmm_status load_launch(const RouteArgs& a, float* part, const RouteLossOut& o, int mode,
                       bool* direct, cudaStream_t st) {
  constexpr int kTurn = kRouteWarps * (32 / kLanes);
  int ctas = 1, most = a.S == 1 ? 6 : 8;
  while (ctas < 8 && (int64_t)2 * ctas * a.S <= 148 * 2 &&
         ((int64_t)most * ctas * kTurn < a.N || (int64_t)2 * ctas * kTurn * a.S < a.N))
    ctas *= 2;
  *direct = a.N <= (int64_t)most * ctas * kTurn;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(*direct ? (int64_t)ctas * a.S : (a.N + a.rows - 1) / a.rows));
  cfg.blockDim = dim3(kRouteThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = *direct && ctas > 1 ? 2 : 1;
  auto kern = *direct ? mode == 0   ? route_load_kernel<T, kLanes, kEl, 0, true>
                        : mode == 1 ? route_load_kernel<T, kLanes, kEl, 1, true>
                                    : route_load_kernel<T, kLanes, kEl, 2, true>
              : mode == 0 ? route_load_kernel<T, kLanes, kEl, 0, false>
              : mode == 1 ? route_load_kernel<T, kLanes, kEl, 1, false>
                          : route_load_kernel<T, kLanes, kEl, 2, false>;
  if (cudaLaunchKernelEx(&cfg, kern, a, part, o) != cudaSuccess)
    return api_launched(0), GMM_ERR_CUDA;
  return api_launched(1);
}

// Lanes and places per row.  Here up to 16 places, so that three CTAs are resident: 262,144 rows of
// 256 fp32 take 54 us with 16 lanes of 16, 62 with 8 of 32.
template <typename T>
gmm_status load_dispatch(const RouteArgs& a, float* part, const RouteLossOut& o, bool* direct,
                         cudaStream_t st) {
  const int mode = route_mode<T>((uintptr_t)a.Z % 16 == 0 && a.ld * sizeof(T) % 16 == 0, a.K);
  if (a.K <= 64) return load_launch<T, 8, 8>(a, part, o, mode, direct, st);
  if (a.K <= 128) return load_launch<T, 8, 16>(a, part, o, mode, direct, st);
  if (a.K <= 256) return load_launch<T, 16, 16>(a, part, o, mode, direct, st);
  if (a.K <= 512) return load_launch<T, 32, 16>(a, part, o, mode, direct, st);
  return load_launch<T, 32, 32>(a, part, o, mode, direct, st);
}

// The least float32 whose product with scale is not -inf.
float least_logit(float scale) {
  float x = std::max(-FLT_MAX, -FLT_MAX / scale);  // (off by a step at most)
  if (x > -FLT_MAX) x = nextafterf(x, -INFINITY);
  while (isinf(x * scale)) x = nextafterf(x, 0.f);
  return x;
}

template <typename T, int kLanes, int kEl>
gmm_status grad_launch(RouteGradArgs g, int mode, cudaStream_t st) {
  int sms = 0;
  gmm_status s = api_device_sms(&sms);
  if (s != GMM_OK) return s;
  constexpr int kRows = 32 / kLanes;
  const int64_t warps = std::min<int64_t>((g.r.N + kRows - 1) / kRows,
                                          (int64_t)sms * kRouteWarps * route_ctas(kEl));
  g.r.rows = ((g.r.N + warps - 1) / warps + kRows - 1) / kRows * kRows;
  const unsigned grid =
      (unsigned)((g.r.N + g.r.rows * kRouteWarps - 1) / (g.r.rows * kRouteWarps));
  auto kern = mode == 0   ? route_grad_kernel<T, kLanes, kEl, 0>
              : mode == 1 ? route_grad_kernel<T, kLanes, kEl, 1>
                          : route_grad_kernel<T, kLanes, kEl, 2>;
  return api_launch_next(kern, dim3(grid), kRouteThreads, 0, st, g);
}

// Here few lanes, so that a warp has four rows to share its reductions and the rows' fixed part:
// 65,536 rows of 256 fp32 take 31 us with 8 lanes of 32, 38 with 16 of 16.
template <typename T>
gmm_status grad_dispatch(const RouteGradArgs& g, cudaStream_t st) {
  const int mode = route_mode<T>((uintptr_t)g.r.Z % 16 == 0 && g.r.ld * sizeof(T) % 16 == 0 &&
                                     (uintptr_t)g.dZ % 16 == 0 && g.ldd * sizeof(T) % 16 == 0,
                                 g.r.K);
  if (g.r.K <= 64) return grad_launch<T, 8, 8>(g, mode, st);
  if (g.r.K <= 128) return grad_launch<T, 8, 16>(g, mode, st);
  if (g.r.K <= 256) return grad_launch<T, 8, 32>(g, mode, st);
  if (g.r.K <= 512) return grad_launch<T, 16, 32>(g, mode, st);
  return grad_launch<T, 32, 32>(g, mode, st);
}

}  // namespace

extern "C" {

gmm_status gmm_route_loss_workspace_size(const gmm_rows* r, int32_t S, size_t* bytes) {
  gmm_status s = check_route(r, 1, S);
  if (s != GMM_OK) return s;
  if (!bytes) return GMM_ERR_INVALID_ARG;
  *bytes = loss_bytes(r, S);
  return GMM_OK;
}

gmm_status gmm_route_loss(const gmm_rows* r, const void* Z, const int32_t* idx, int32_t m,
                          const uint8_t* mask, const int32_t* offsets, int32_t S, float* balance,
                          float* z, float* load, int32_t* counts, int32_t* rows,
                          uint32_t* dev_flags, void* ws, size_t ws_bytes, void* stream) {
  gmm_status s = check_route(r, m, S);
  if (s != GMM_OK) return s;
  if (!offsets && S != 1) return GMM_ERR_INVALID_ARG;
  if (S == 0) return GMM_OK;
  if (!balance && !z && !load && !counts && !rows) return GMM_ERR_INVALID_ARG;
  if (r->N > 0 && (!Z || !idx)) return GMM_ERR_INVALID_ARG;
  if ((uintptr_t)Z % elem(r->dtype) != 0) return GMM_ERR_UNSUPPORTED;
  if (!ws || (uintptr_t)ws % 256 != 0 || ws_bytes < loss_bytes(r, S)) return GMM_ERR_WORKSPACE;
  const LossPlan plan = loss_plan(r->N, S, r->K);
  const RouteArgs a = {Z,    r->N,    r->ld, r->K,      r->scale, idx, m,
                       mask, offsets, S,     plan.rows, dev_flags};
  cudaStream_t st = (cudaStream_t)stream;
  const RouteLossOut o = {balance, z, load, counts, rows};
  if (r->N > 0) {
    bool direct = false;
    s = r->dtype == GMM_F32    ? load_dispatch<float>(a, (float*)ws, o, &direct, st)
        : r->dtype == GMM_BF16 ? load_dispatch<__nv_bfloat16>(a, (float*)ws, o, &direct, st)
                               : load_dispatch<__half>(a, (float*)ws, o, &direct, st);
    if (s != GMM_OK || direct) return s;
  }
  // a cluster per segment: 32 experts to a CTA, up to 8 CTAs, of 1,024 threads, while all segments'
  // are resident at once (64 segments of 7,152 rows of 244: 35 us in clusters of 8, 12 in twos)
  const int ctas = std::max(1, std::min({kReduceCtas, (r->K + 31) / 32, 148 / S}));
  const int threads = (int64_t)S * ctas > 296 ? 256 : 1024;
  int cols = 32;
  while (cols * ctas < r->K && cols < threads) cols *= 2;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)S * ctas);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  auto kern = threads == 256 ? route_reduce_kernel<256> : route_reduce_kernel<1024>;
  if (cudaLaunchKernelEx(&cfg, kern, a, (const float*)ws, o, cols) != cudaSuccess)
    return api_launched(0), GMM_ERR_CUDA;
  return api_launched(1);
}

gmm_status gmm_route_backward(const gmm_rows* r, const void* Z, const int32_t* idx, int32_t m,
                              const float* dresp, int32_t renorm, const int32_t* counts,
                              const int32_t* rows, const float* dbalance, const float* dz,
                              const uint8_t* mask, const int32_t* offsets, int32_t S, void* dZ,
                              int64_t ldd, uint32_t* dev_flags, void* stream) {
  gmm_status s = check_route(r, m, S);
  if (s != GMM_OK) return s;
  if (ldd < r->K) return GMM_ERR_INVALID_ARG;
  if (ldd > kMaxStride || (double)r->N * (double)ldd > 1e18) return GMM_ERR_UNSUPPORTED;
  const bool losses = dbalance || dz;
  if (losses && !offsets && S != 1) return GMM_ERR_INVALID_ARG;
  if (losses && offsets && S < 1) return GMM_ERR_INVALID_ARG;
  if (r->N == 0) return GMM_OK;
  if (!dresp && !losses) return GMM_ERR_INVALID_ARG;
  if (!Z || !dZ || (dresp && !idx) || (dbalance && !counts) || (losses && !rows))
    return GMM_ERR_INVALID_ARG;
  if (dZ == Z && ldd != r->ld) return GMM_ERR_INVALID_ARG;
  if ((uintptr_t)Z % elem(r->dtype) != 0 || (uintptr_t)dZ % elem(r->dtype) != 0)
    return GMM_ERR_UNSUPPORTED;
  const RouteArgs a = {Z,    r->N,    r->ld, r->K, r->scale, idx, m,
                       mask, offsets, S,     0,    dev_flags};
  const RouteGradArgs g = {a,  dresp, renorm != 0, counts, rows, dbalance,
                           dz, dZ,    ldd,         least_logit(r->scale)};
  cudaStream_t st = (cudaStream_t)stream;
  if (r->dtype == GMM_F32) return grad_dispatch<float>(g, st);
  if (r->dtype == GMM_BF16) return grad_dispatch<__nv_bfloat16>(g, st);
  return grad_dispatch<__half>(g, st);
}

}  // extern "C"
