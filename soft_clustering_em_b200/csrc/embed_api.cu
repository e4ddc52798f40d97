// embed_api.cu -- host side of gmm_embed and gmm_embed_backward: argument checks, workspace
// layout and launches.
#include <math.h>

#include <algorithm>

#include "api_common.h"
#include "embed.cuh"

using namespace scem;

namespace {

constexpr int32_t kMaxEmbedK = 1 << 24;
constexpr int32_t kMaxEmbedD = 1 << 20;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

size_t elem(int32_t t) { return t == GMM_F32 ? 4 : 2; }
bool is_type(int32_t t) { return t == GMM_F32 || t == GMM_BF16 || t == GMM_F16; }

gmm_status check_embed(const gmm_embed_problem* p) {
  if (!p) return GMM_ERR_INVALID_ARG;
  if (p->N < 0 || p->m < 1 || p->m > kMaxTopM || p->K < 1 || p->D < 1 || !is_type(p->dtype) ||
      !isfinite(p->scale))
    return GMM_ERR_INVALID_ARG;
  if (p->ldw < p->D || p->ldy < p->D) return GMM_ERR_INVALID_ARG;
  if (p->K > kMaxEmbedK || p->D > kMaxEmbedD || p->ldw > kMaxStride || p->ldy > kMaxStride ||
      p->N >= ((int64_t)1 << 31) / p->m || (double)p->N * (double)p->D > 1e12 ||
      (double)p->N * (double)p->ldy > 1e18 || (double)p->K * (double)p->ldw > 1e18)
    return GMM_ERR_UNSUPPORTED;
  return GMM_OK;
}

// Whether rows of a tensor start on 16 bytes.
bool aligned_rows(const void* base, int64_t ld, size_t size) {
  return (uintptr_t)base % 16 == 0 && ld * size % 16 == 0;
}

template <typename T, bool kVec>
gmm_status embed_launch(EmbedArgs a, cudaStream_t st) {
  constexpr int V = Unit<T, kVec>::n;
  int sms = 0;
  gmm_status s = api_device_sms(&sms);
  if (s != GMM_OK) return s;
  a.units = (a.D + V - 1) / V;
  a.magic = a.units > 1 ? (uint32_t)((((uint64_t)1 << 32) + a.units - 1) / a.units) : 0;
  const int64_t all = a.N * a.units;
  // one unit per thread while that leaves SMs without work
  if (all <= (int64_t)sms * 2 * kEmbedThreads) {
    embed_kernel<T, kVec, 1><<<(unsigned)((all + 255) / 256), kEmbedThreads, 0, st>>>(a);
  } else {
    embed_kernel<T, kVec, 4><<<(unsigned)((all + 1023) / 1024), kEmbedThreads, 0, st>>>(a);
  }
  return api_launched(1);
}

template <typename T>
gmm_status embed_vec(const EmbedArgs& a, cudaStream_t st) {
  return aligned_rows(a.W, a.ldw, sizeof(T)) && aligned_rows(a.Y, a.ldy, sizeof(T))
             ? embed_launch<T, true>(a, st)
             : embed_launch<T, false>(a, st);
}

// ---------------------------------------------------------------- the gradient
// Digits of the sort: as few as hold the classes 0 .. K (K: none).
struct SortPlan {
  int passes, bits;
  uint32_t tiles, per_warp;
};

SortPlan sort_plan(uint32_t M, int K) {
  int bits = 1;
  while (bits < 31 && (K >> bits) != 0) bits++;
  SortPlan s;
  s.passes = (bits + kSortBits - 1) / kSortBits;
  s.bits = (bits + s.passes - 1) / s.passes;
  s.tiles = std::max(1u, std::min<uint32_t>(kSortTiles, (M + kSortThreads - 1) / kSortThreads));
  const uint32_t warps = s.tiles * kSortWarps;
  s.per_warp = std::max(32u, (M / warps + (M % warps != 0) + 31) / 32 * 32);
  return s;
}

// Choices per chunk.  More, and fewer runs are cut; fewer, and there are more CTAs.
uint32_t grad_chunk(uint32_t M) {
  uint32_t c = 16;
  while (c < 128 && M / c > 8192) c *= 2;
  return c;
}

// Workspace: two buffers of sorted classes and their places, counts, seen classes, cut sums.
struct GradLayout {
  size_t key[2], src[2], counts, seen, part, total;
  uint32_t chunk, chunks;
  int width;
};

GradLayout grad_layout(const gmm_embed_problem* p) {
  GradLayout L;
  const uint32_t M = (uint32_t)(p->N * p->m);
  const SortPlan s = sort_plan(M, p->K);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  for (int i = 0; i < 2; i++) {
    L.key[i] = take((size_t)M * 4);
    L.src[i] = take((size_t)M * 4);
  }
  L.counts = take(((size_t)s.tiles << s.bits) * 4);
  L.seen = take(p->K);
  L.chunk = grad_chunk(M);
  L.chunks = M / L.chunk + (M % L.chunk != 0);
  L.width = (p->D + 7) / 8 * 8;
  L.part = take((size_t)L.chunks * 2 * L.width * 4);
  L.total = off;
  return L;
}

struct GradCall {
  const gmm_embed_problem* p;
  const void *dY, *W;
  const int32_t* idx;
  const float* resp;
  void* dW;
  int64_t ldd;
  bool add;
  float* dresp;
  uint32_t* flags;
  char* ws;
  cudaStream_t st;
};

template <typename T, bool kVec>
gmm_status dot_launch(const GradCall& g) {
  const gmm_embed_problem* p = g.p;
  constexpr int V = Unit<T, kVec>::n;
  EmbedDotArgs a = {g.W,  g.dY, g.idx, g.dresp, p->N, p->ldw, p->ldy,
                    p->m, p->K, p->D,  (p->D + V - 1) / V, p->scale, g.flags};
  int sms = 0;
  gmm_status s = api_device_sms(&sms);
  if (s != GMM_OK) return s;
  auto go = [&](auto kern, int lanes) {
    const int rows = kEmbedThreads / lanes;
    const int64_t blocks = std::min<int64_t>((p->N + rows - 1) / rows, (int64_t)sms * 64);
    return api_launch_next(kern, dim3((unsigned)blocks), kEmbedThreads, 0, g.st, a);
  };
  if (a.units <= 16) {
    if (p->m == 1) return go(embed_dot_kernel<T, kVec, 8, 1>, 8);
    if (p->m == 2) return go(embed_dot_kernel<T, kVec, 8, 2>, 8);
    return go(embed_dot_kernel<T, kVec, 8, kMaxTopM>, 8);
  }
  if (p->m == 1) return go(embed_dot_kernel<T, kVec, 32, 1>, 32);
  if (p->m == 2) return go(embed_dot_kernel<T, kVec, 32, 2>, 32);
  return go(embed_dot_kernel<T, kVec, 32, kMaxTopM>, 32);
}

template <typename T, typename TO, bool kVec>
gmm_status grad_launch(const GradCall& g) {
  const gmm_embed_problem* p = g.p;
  const GradLayout L = grad_layout(p);
  const uint32_t M = (uint32_t)(p->N * p->m);
  const SortPlan plan = sort_plan(M, p->K);
  constexpr int V = Unit<T, kVec>::n;
  EmbedGradArgs a = {};
  a.dY = g.dY;
  a.resp = g.resp;
  a.seen = g.add ? nullptr : (const uint8_t*)(g.ws + L.seen);
  a.dW = g.dW;
  a.part = (float*)(g.ws + L.part);
  a.ldy = p->ldy;
  a.ldd = g.ldd;
  a.by_m = (((uint64_t)1 << 34) + p->m - 1) / p->m;
  a.M = M;
  a.chunk = L.chunk;
  a.chunks = L.chunks;
  a.K = p->K;
  a.D = p->D;
  a.units = (p->D + V - 1) / V;
  a.lanes = 8;
  while (a.lanes < kEmbedThreads && a.lanes < a.units) a.lanes *= 2;
  a.width = L.width;
  a.scale = p->scale;
  a.m = p->m;

  gmm_status s;
  if (cudaFuncSetAttribute(sort_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSortWarps * (4 << kSortBits)) != cudaSuccess)
    return api_launched(0), GMM_ERR_CUDA;
  for (int i = 0; i < plan.passes; i++) {
    SortArgs o = {};
    o.idx = i == 0 ? g.idx : nullptr;
    o.key = a.key;
    o.src = a.src;
    o.key_out = (uint32_t*)(g.ws + L.key[i & 1]);
    o.src_out = (uint32_t*)(g.ws + L.src[i & 1]);
    o.counts = (uint32_t*)(g.ws + L.counts);
    o.seen = i == 0 && !g.add ? (uint8_t*)(g.ws + L.seen) : nullptr;
    o.M = M;
    o.per_warp = plan.per_warp;
    o.K = p->K;
    o.bits = plan.bits;
    o.shift = i * plan.bits;
    o.flags = g.flags;
    if ((s = api_launch_next(sort_count_kernel, dim3(plan.tiles), kSortThreads, 0, g.st, o)) != GMM_OK)
      return s;
    if ((s = api_launch_next(sort_place_kernel, dim3(plan.tiles), kSortThreads,
                         kSortWarps * ((size_t)4 << plan.bits), g.st, o)) != GMM_OK)
      return s;
    a.key = o.key_out;
    a.src = o.src_out;
  }
  if (M > 0) {
    const unsigned groups = kEmbedThreads / a.lanes;
    const dim3 grid((a.chunks + groups - 1) / groups, (a.units + a.lanes - 1) / a.lanes);
    if ((s = api_launch_next(embed_sum_kernel<T, TO, kVec>, grid, kEmbedThreads, 0, g.st, a)) !=
        GMM_OK)
      return s;
  }
  const unsigned fill = g.add ? 0 : (unsigned)((p->K + kFillRows - 1) / kFillRows);
  if (a.chunks + fill > 0 &&
      (s = api_launch_next(embed_finish_kernel<T, TO, kVec>, dim3(a.chunks + fill), kEmbedThreads, 0,
                       g.st, a, a.chunks)) != GMM_OK)
    return s;
  return GMM_OK;
}

template <typename T>
gmm_status grad_types(const GradCall& g, bool wide) {
  const gmm_embed_problem* p = g.p;
  gmm_status s = GMM_OK;
  if (g.dresp && p->N > 0) {
    s = aligned_rows(g.W, p->ldw, sizeof(T)) && aligned_rows(g.dY, p->ldy, sizeof(T))
            ? dot_launch<T, true>(g)
            : dot_launch<T, false>(g);
    if (s != GMM_OK) return s;
  }
  if (!g.dW) return GMM_OK;
  const bool vec = aligned_rows(g.dY, p->ldy, sizeof(T)) &&
                   aligned_rows(g.dW, g.ldd, wide ? sizeof(float) : sizeof(T));
  if (wide) return vec ? grad_launch<T, float, true>(g) : grad_launch<T, float, false>(g);
  return vec ? grad_launch<T, T, true>(g) : grad_launch<T, T, false>(g);
}

}  // namespace

extern "C" {

gmm_status gmm_embed(const gmm_embed_problem* p, const void* W, const int32_t* idx,
                     const float* resp, void* Y, uint32_t* dev_flags, void* stream) {
  gmm_status s = check_embed(p);
  if (s != GMM_OK) return s;
  if (p->N == 0) return GMM_OK;
  if (!W || !idx || !Y) return GMM_ERR_INVALID_ARG;
  if ((uintptr_t)W % elem(p->dtype) != 0 || (uintptr_t)Y % elem(p->dtype) != 0)
    return GMM_ERR_UNSUPPORTED;
  const EmbedArgs a = {W,    idx,  resp, Y,        p->N, p->ldw, p->ldy,
                       p->m, p->K, p->D, p->scale, 0,    0,      dev_flags};
  cudaStream_t st = (cudaStream_t)stream;
  if (p->dtype == GMM_F32) return embed_vec<float>(a, st);
  if (p->dtype == GMM_BF16) return embed_vec<__nv_bfloat16>(a, st);
  return embed_vec<__half>(a, st);
}

gmm_status gmm_embed_workspace_size(const gmm_embed_problem* p, size_t* bytes) {
  gmm_status s = check_embed(p);
  if (s != GMM_OK) return s;
  if (!bytes) return GMM_ERR_INVALID_ARG;
  *bytes = grad_layout(p).total;
  return GMM_OK;
}

gmm_status gmm_embed_backward(const gmm_embed_problem* p, const void* dY, const int32_t* idx,
                              const float* resp, const void* W, void* dW, int32_t dw_dtype,
                              int64_t ldd, int32_t accumulate, float* dresp, uint32_t* dev_flags,
                              void* ws, size_t ws_bytes, void* stream) {
  gmm_status s = check_embed(p);
  if (s != GMM_OK) return s;
  if (!dW && !dresp) return GMM_ERR_INVALID_ARG;
  if (dresp && p->N > 0 && !W) return GMM_ERR_INVALID_ARG;
  if (p->N > 0 && (!dY || !idx)) return GMM_ERR_INVALID_ARG;
  const size_t size = elem(p->dtype);
  if (dW) {
    if ((dw_dtype != GMM_F32 && dw_dtype != p->dtype) || ldd < p->D) return GMM_ERR_INVALID_ARG;
    if (ldd > kMaxStride || (double)p->K * (double)ldd > 1e18 ||
        (uintptr_t)dW % elem(dw_dtype) != 0)
      return GMM_ERR_UNSUPPORTED;
  }
  if ((uintptr_t)dY % size != 0 || (dresp && (uintptr_t)W % size != 0))
    return GMM_ERR_UNSUPPORTED;
  if (dW && (!ws || (uintptr_t)ws % 256 != 0 || ws_bytes < grad_layout(p).total))
    return GMM_ERR_WORKSPACE;
  const GradCall g = {p,     dY,        W,         idx,       resp,
                      dW,    ldd,       accumulate != 0, dresp, dev_flags,
                      (char*)ws, (cudaStream_t)stream};
  const bool wide = dW && dw_dtype == GMM_F32 && p->dtype != GMM_F32;
  if (p->dtype == GMM_F32) return grad_types<float>(g, false);
  if (p->dtype == GMM_BF16) return grad_types<__nv_bfloat16>(g, wide);
  return grad_types<__half>(g, wide);
}

}  // extern "C"
