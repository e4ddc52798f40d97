// embed_api.cu -- host side of gmm_embed and gmm_embed_backward: argument checks, workspace
// layout and launches.
#include <math.h>

#include <algorithm>
#include <atomic>

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
// How rows of D elements are taken (Unit).
template <typename T>
int unit_mode(bool aligned, int D) {
  return !aligned ? 0 : D % Vec16<T>::n != 0 ? 1 : 2;
}

template <typename T, int kMode>
gmm_status embed_launch(EmbedArgs a, cudaStream_t st) {
  constexpr int V = Unit<T, kMode>::n;
  int sms = 0;
  gmm_status s = api_device_sms(&sms);
  if (s != GMM_OK) return s;
  a.units = (a.D + V - 1) / V;
  const bool few = a.N * a.units <= (int64_t)sms * 2 * kEmbedThreads;
  // Lanes of a row: of the shapes with up to `most` units per lane, the one that wastes the fewest
  // places; of those, the fewest lanes.  One unit per lane while more would leave SMs without work.
  int per = 1;
  auto shape = [&](int most) {
    int64_t least = INT64_MAX;
    for (int bits = 8; bits >= 0; bits--) {
      const int64_t lanes = (int64_t)1 << bits, each = (a.units + lanes - 1) / lanes;
      if (each > most && bits < 6) break;
      if (each * lanes <= least) {
        least = each * lanes;
        a.lane_bits = bits;
        per = (int)std::min<int64_t>(each, most);
      }
    }
  };
  auto go = [&](auto kern) {
    const int rows = kEmbedThreads >> a.lane_bits, width = per << a.lane_bits;
    const dim3 grid((unsigned)((a.N + rows - 1) / rows), (a.units + width - 1) / width);
    return api_launch_next(kern, grid, kEmbedThreads, 0, st, a);
  };
  shape(few ? 1 : a.m <= 2 ? 4 : a.m <= 4 ? 2 : 1);
  if (a.m == 1)
    return per == 1   ? go(embed_kernel<T, kMode, 1, 1>)
           : per == 2 ? go(embed_kernel<T, kMode, 1, 2>)
           : per == 3 ? go(embed_kernel<T, kMode, 1, 3>)
                      : go(embed_kernel<T, kMode, 1, 4>);
  if (a.m == 2)
    return per == 1   ? go(embed_kernel<T, kMode, 2, 1>)
           : per == 2 ? go(embed_kernel<T, kMode, 2, 2>)
           : per == 3 ? go(embed_kernel<T, kMode, 2, 3>)
                      : go(embed_kernel<T, kMode, 2, 4>);
  if (a.m <= 4)
    return per == 1 ? go(embed_kernel<T, kMode, 4, 1>) : go(embed_kernel<T, kMode, 4, 2>);
  return go(embed_kernel<T, kMode, kMaxTopM, 1>);
}

template <typename T>
gmm_status embed_vec(const EmbedArgs& a, cudaStream_t st) {
  const bool aligned = aligned_rows(a.W, a.ldw, sizeof(T)) && aligned_rows(a.Y, a.ldy, sizeof(T));
  const int mode = unit_mode<T>(aligned, a.D);
  return mode == 0   ? embed_launch<T, 0>(a, st)
         : mode == 1 ? embed_launch<T, 1>(a, st)
                     : embed_launch<T, 2>(a, st);
}

// ---------------------------------------------------------------- the gradient
// Digits of the sort: as few as hold the classes 0 .. K (K: none); tiles and a warp's choices for
// two kernels per digit.
struct SortPlan {
  int passes, bits;
  uint32_t tiles, per_warp;
};

uint32_t part_of(uint32_t M, uint32_t warps) {  // a warp's choices: whole rounds of 32
  return std::max(32u, (M / warps + (M % warps != 0) + 31) / 32 * 32);
}

SortPlan sort_plan(uint32_t M, int K) {
  int bits = 1;
  while (bits < 31 && (K >> bits) != 0) bits++;
  SortPlan s;
  s.passes = (bits + kSortBits - 1) / kSortBits;
  s.bits = (bits + s.passes - 1) / s.passes;
  s.tiles = std::max(1u, std::min<uint32_t>(kSortTiles, (M + kSortThreads - 1) / kSortThreads));
  s.per_warp = part_of(M, s.tiles * kSortWarps);
  return s;
}

size_t cluster_smem(int bits) { return ((size_t)(kClusterWarps + 1) << bits) * 4; }

// CTAs of the sorting cluster: 16 where the device has room for one, else 8.  Asked once per
// device.
bool cluster_size(int* C) {
  static std::atomic<int> known[64];
  int device = 0;
  if (cudaGetDevice(&device) != cudaSuccess) return false;
  const bool keep = device >= 0 && device < 64;
  if (keep && (*C = known[device].load()) != 0) return true;
  const int smem = (int)cluster_smem(kSortBits);
  if (cudaFuncSetAttribute(sort_cluster_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           smem) != cudaSuccess ||
      cudaFuncSetAttribute(sort_cluster_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                           1) != cudaSuccess)
    return false;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 16;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(kClusterThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  *C = cudaOccupancyMaxActiveClusters(&n, sort_cluster_kernel, &cfg) == cudaSuccess && n > 0 ? 16
                                                                                             : 8;
  cudaGetLastError();  // (a size that is not supported is no error of the call)
  if (keep) known[device] = *C;
  return true;
}

// Lanes of a group of the sums, for rows of so many units.
int grad_lanes(int units) {
  int lanes = 8;
  while (lanes < kEmbedThreads && lanes < units) lanes *= 2;
  return lanes;
}

// Choices per chunk: as few as leave no more CTAs than are resident at once (3 on each of 148
// SMs), or whole turns of those, between 16 and 128.  (131,072 x 2,048 bf16 from 16,384 choices:
// 122 us in chunks of 16, 2.3 turns of the CTAs, 116 in chunks of 40.)
uint32_t grad_chunk(const gmm_embed_problem* p, uint32_t M) {
  const int units = (int)((p->D * elem(p->dtype) + 15) / 16), lanes = grad_lanes(units);
  const uint64_t slices = (units + lanes - 1) / lanes, groups = kEmbedThreads / lanes;
  const uint64_t most = std::max<uint64_t>(1, 3 * 148 * groups / slices);
  const uint64_t turns = (M + most * kGradChunk - 1) / (most * kGradChunk);
  const uint64_t chunk = turns == 0 ? 0 : (M + most * turns - 1) / (most * turns);
  return (uint32_t)std::min<uint64_t>(kGradChunk, std::max<uint64_t>(16, (chunk + 7) / 8 * 8));
}

// Workspace: two buffers of sorted choices, counts, named classes, cut sums, Beside's word.
struct GradLayout {
  size_t list[2], counts, seen, part, beside, total;
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
  for (int i = 0; i < 2; i++) L.list[i] = take((size_t)M * sizeof(Choice));
  L.counts = take(((size_t)s.tiles << s.bits) * 4);
  L.seen = take(p->K);
  L.chunk = grad_chunk(p, M);
  L.chunks = M / L.chunk + (M % L.chunk != 0);
  L.width = (p->D + 7) / 8 * 8;
  L.part = take((size_t)L.chunks * 2 * L.width * 4);
  L.beside = take(8);
  L.total = off;
  return L;
}

std::atomic<unsigned long long> grad_calls{0x9e3779b97f4a7c15ull};  // (no other content's number)

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
  Beside beside;  // (no word: what would go on beside the sort waits for what is before it)
};

// The choices sorted by class, in *list.
// `seen`: K bytes for which classes are named, or null.
gmm_status sort_launch(const GradCall& g, const GradLayout& L, uint32_t M, uint8_t* seen,
                       const Choice** list) {
  const SortPlan plan = sort_plan(M, g.p->K);
  Choice* lists[2] = {(Choice*)(g.ws + L.list[0]), (Choice*)(g.ws + L.list[1])};
  *list = lists[(plan.passes - 1) & 1];
  if (M <= kSortCluster) {
    int most = 0, C = 1;  // 1,024 choices, one round of its warps, per CTA
    if (!cluster_size(&most)) return api_launched(0), GMM_ERR_CUDA;
    while (C < most && (uint32_t)C * kClusterThreads < M) C *= 2;
    const SortAllArgs a = {g.idx,       {lists[0], lists[1]}, seen,
                           M,           part_of(M, C * kClusterWarps),
                           g.p->K,      plan.passes,          plan.bits,
                           g.flags,     g.beside};
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(kClusterThreads);
    cfg.dynamicSmemBytes = cluster_smem(plan.bits);
    cfg.stream = g.st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (cudaLaunchKernelEx(&cfg, sort_cluster_kernel, a) != cudaSuccess)
      return api_launched(0), GMM_ERR_CUDA;
    return api_launched(1);
  }
  if (cudaFuncSetAttribute(sort_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kSortWarps * (4 << kSortBits)) != cudaSuccess)
    return api_launched(0), GMM_ERR_CUDA;
  for (int i = 0; i < plan.passes; i++) {
    SortArgs o = {};
    o.idx = i == 0 ? g.idx : nullptr;
    o.in = lists[(i + 1) & 1];
    o.out = lists[i & 1];
    o.counts = (uint32_t*)(g.ws + L.counts);
    o.seen = i == 0 ? seen : nullptr;
    o.M = M;
    o.per_warp = plan.per_warp;
    o.K = g.p->K;
    o.bits = plan.bits;
    o.shift = i * plan.bits;
    o.flags = g.flags;
    if (i == 0) o.beside = g.beside;
    gmm_status s;
    if ((s = api_launch_next(sort_count_kernel, dim3(plan.tiles), kSortThreads, 0, g.st, o)) !=
        GMM_OK)
      return s;
    if ((s = api_launch_next(sort_place_kernel, dim3(plan.tiles), kSortThreads,
                             kSortWarps * ((size_t)4 << plan.bits), g.st, o)) != GMM_OK)
      return s;
  }
  return GMM_OK;
}

template <typename T, int kMode>
gmm_status dot_launch(const GradCall& g) {
  const gmm_embed_problem* p = g.p;
  constexpr int V = Unit<T, kMode>::n;
  EmbedDotArgs a = {g.W,  g.dY, g.idx, g.dresp, p->N, p->ldw, p->ldy,
                    p->m, p->K, p->D,  (p->D + V - 1) / V, p->scale, g.flags, g.beside};
  int sms = 0;
  gmm_status s = api_device_sms(&sms);
  if (s != GMM_OK) return s;
  auto go = [&](auto kern, int lanes) {
    const int rows = kEmbedThreads / lanes;
    const int64_t blocks = std::min<int64_t>((p->N + rows - 1) / rows, sms * kBesideCtas);
    return api_launch_next(kern, dim3((unsigned)blocks), kEmbedThreads, 0, g.st, a);
  };
  auto lanes = [&](auto one, auto two, auto four, auto most, int n) {
    return p->m == 1 ? go(one, n) : p->m == 2 ? go(two, n) : p->m <= 4 ? go(four, n) : go(most, n);
  };
  if (a.units <= 64)  // 8 lanes of up to 8 units: 4 rows per warp
    return lanes(embed_dot_kernel<T, kMode, 8, 1>, embed_dot_kernel<T, kMode, 8, 2>,
                 embed_dot_kernel<T, kMode, 8, 4>, embed_dot_kernel<T, kMode, 8, kMaxTopM>, 8);
  if (p->N >= (int64_t)sms * kBesideCtas)
    return lanes(embed_dot_kernel<T, kMode, 32, 1>, embed_dot_kernel<T, kMode, 32, 2>,
                 embed_dot_kernel<T, kMode, 32, 4>, embed_dot_kernel<T, kMode, 32, kMaxTopM>, 32);
  // few rows: a CTA for each (8 rows of 5,987 fp16 that start anywhere: 177 us with a warp each)
  return lanes(embed_dot_kernel<T, kMode, 256, 1>, embed_dot_kernel<T, kMode, 256, 2>,
               embed_dot_kernel<T, kMode, 256, 4>, embed_dot_kernel<T, kMode, 256, kMaxTopM>, 256);
}

template <typename T>
gmm_status dot_vec(const GradCall& g) {
  if (!g.dresp || g.p->N == 0) return GMM_OK;
  const bool aligned =
      aligned_rows(g.W, g.p->ldw, sizeof(T)) && aligned_rows(g.dY, g.p->ldy, sizeof(T));
  const int mode = unit_mode<T>(aligned, g.p->D);
  return mode == 0   ? dot_launch<T, 0>(g)
         : mode == 1 ? dot_launch<T, 1>(g)
                     : dot_launch<T, 2>(g);
}

gmm_status fill_launch(const GradCall& g, size_t size, uint64_t rows) {
  int sms = 0;
  gmm_status s = api_device_sms(&sms);
  if (s != GMM_OK) return s;
  const uint64_t D = g.p->D;
  const bool one = g.ldd == g.p->D;  // one long row
  FillArgs a = {(char*)g.dW, one ? 1 : rows, (one ? rows * D : D) * size, (uint64_t)g.ldd * size,
                0, g.beside};
  a.parts = (a.row_bytes + kFillPiece - 1) / kFillPiece;
  const uint64_t blocks = (a.rows * a.parts + kEmbedThreads / 32 - 1) / (kEmbedThreads / 32);
  return api_launch_next(embed_fill_kernel,
                         dim3((unsigned)std::min<uint64_t>(blocks, sms * kBesideCtas)),
                         kEmbedThreads, 0, g.st, a);
}

// Rows that get their zeros beside the sort: what goes through while it runs (6 GB in a ms, from
// 12 us on 1 us more for every 8,192 choices).
uint64_t beside_rows(const gmm_embed_problem* p, uint32_t M, size_t size) {
  const uint64_t rows = (uint64_t)(6e6 * (12.0 + M / 8192.0) / ((double)p->D * size));
  return std::min<uint64_t>(p->K, std::max<uint64_t>(rows, 1));
}

// Up to kFew choices, in one launch (and the weights' gradient in one before it).
template <typename T, typename TO, int kMode>
gmm_status few_launch(const GradCall& g, EmbedGradArgs a) {
  const gmm_embed_problem* p = g.p;
  gmm_status s = dot_vec<T>(g);
  if (s != GMM_OK) return s;
  const int groups = kEmbedThreads / a.lanes;
  a.sum_blocks = (a.M + groups - 1) / groups;
  const uint64_t bytes = (uint64_t)p->D * sizeof(TO);
  a.fill_rows = (int)std::max<uint64_t>(8, std::min<uint64_t>(kFewRows, 131072 / bytes / 8 * 8));
  const unsigned fill = g.add ? 0 : (unsigned)((p->K + a.fill_rows - 1) / a.fill_rows);
  const EmbedFewArgs f = {a, g.idx, g.flags};
  return api_launch_next(embed_few_kernel<T, TO, kMode>,
                         dim3(a.sum_blocks + fill, (a.units + a.lanes - 1) / a.lanes),
                         kEmbedThreads, 0, g.st, f);
}

// Stream order: the sort; beside it the weights' gradient and rows of zeros; then the sums.
template <typename T, typename TO, int kMode>
gmm_status grad_launch(GradCall g) {
  const gmm_embed_problem* p = g.p;
  const GradLayout L = grad_layout(p);
  const uint32_t M = (uint32_t)(p->N * p->m);
  constexpr int V = Unit<T, kMode>::n;
  EmbedGradArgs a = {};
  gmm_status s;
  a.dY = g.dY;
  a.resp = g.resp;
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
  a.lanes = grad_lanes(a.units);
  a.width = L.width;
  a.scale = p->scale;
  a.m = p->m;
  a.add = g.add;
  if (M == 0) return g.add ? GMM_OK : fill_launch(g, sizeof(TO), p->K);
  if (M <= kFew) return few_launch<T, TO, kMode>(g, a);
  g.beside = {(unsigned long long*)(g.ws + L.beside), ++grad_calls};
  a.beside = g.beside.word;
  const uint64_t beside = g.add ? p->K : beside_rows(p, M, sizeof(TO));
  uint8_t* seen = beside < (uint64_t)p->K ? (uint8_t*)(g.ws + L.seen) : nullptr;
  if ((s = sort_launch(g, L, M, seen, &a.list)) != GMM_OK) return s;
  if ((s = dot_vec<T>(g)) != GMM_OK) return s;
  if (!g.add && (s = fill_launch(g, sizeof(TO), beside)) != GMM_OK) return s;
  const unsigned groups = kEmbedThreads / a.lanes;
  a.sum_blocks = (a.chunks + groups - 1) / groups;
  // the other rows' zeros: blocks of about 128 KB, one per SM ahead of the sums' so that the memory
  // is busy while those wait for it
  const uint64_t left = p->K - beside, bytes = (uint64_t)p->D * sizeof(TO);
  a.seen = seen;
  a.fill_from = (int)beside;
  a.fill_rows = (int)std::max<uint64_t>(8, std::min<uint64_t>(4096, (131072 / bytes + 7) / 8 * 8));
  const uint32_t fill = (uint32_t)((left + a.fill_rows - 1) / a.fill_rows);
  a.fill_first = std::min(fill, 148u);
  const dim3 grid(a.sum_blocks + fill, (a.units + a.lanes - 1) / a.lanes);
  if ((s = api_launch_next(embed_sum_kernel<T, TO, kMode>, grid, kEmbedThreads,
                           (size_t)groups * a.chunk * 12, g.st, a)) != GMM_OK)
    return s;
  constexpr int kWarps = kEmbedThreads / 32;
  return api_launch_next(embed_join_kernel<T, TO, kMode>,
                         dim3((a.chunks + kWarps - 1) / kWarps, (a.units + 31) / 32),
                         kEmbedThreads, 0, g.st, a);
}

template <typename T, typename TO>
gmm_status grad_vec(const GradCall& g) {
  const bool aligned = aligned_rows(g.dY, g.p->ldy, sizeof(T)) &&
                       aligned_rows(g.dW, g.ldd, sizeof(TO));
  const int mode = unit_mode<T>(aligned, g.p->D);
  return mode == 0   ? grad_launch<T, TO, 0>(g)
         : mode == 1 ? grad_launch<T, TO, 1>(g)
                     : grad_launch<T, TO, 2>(g);
}

template <typename T>
gmm_status grad_types(const GradCall& g, bool wide) {
  if (!g.dW) return dot_vec<T>(g);
  return wide ? grad_vec<T, float>(g) : grad_vec<T, T>(g);
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
                       p->m, p->K, p->D, p->scale, 0,    0,    dev_flags};
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
  if (!dW && !dresp && p->N > 0) return GMM_ERR_INVALID_ARG;
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
                      (char*)ws, (cudaStream_t)stream, {}};
  const bool wide = dW && dw_dtype == GMM_F32 && p->dtype != GMM_F32;
  if (p->dtype == GMM_F32) return grad_types<float>(g, false);
  if (p->dtype == GMM_BF16) return grad_types<__nv_bfloat16>(g, wide);
  return grad_types<__half>(g, wide);
}

}  // extern "C"
