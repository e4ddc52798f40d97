// embed.cuh -- rows of a table chosen by an assignment, and the gradient by sorted classes:
// kernels of gmm_embed and gmm_embed_backward.
//
//   Y_n = scale sum_j r_nj W[idx_nj]              (r = 1 without weights)
//   dW_k = scale sum_{(n,j): idx_nj = k} r_nj dY_n
//   dr_nj = scale <dY_n, W[idx_nj]>
// Sums are held in float32 and rounded once.  Everything is bound by memory: the named rows
// and the output go through once.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "vec16.cuh"

namespace scem {

constexpr int kEmbedThreads = 256;

struct EmbedArgs {
  const void* W;
  const int32_t* idx;  // N x m
  const float* resp;   // N x m, may be null
  void* Y;
  int64_t N, ldw, ldy;
  int m, K, D;
  float scale;
  int units;       // of kEl elements per row
  uint32_t magic;  // ceil(2^32 / units)
  uint32_t* flags;
};

// A unit of a row: 16 bytes of T (kVec, rows start on 16 bytes), or one element.
template <typename T, bool kVec>
struct Unit {
  static constexpr int n = kVec ? Vec16<T>::n : 1;
  using Raw = typename std::conditional<kVec, uint4, T>::type;
  static __device__ __forceinline__ Raw zero() {
    if constexpr (kVec) return make_uint4(0, 0, 0, 0);
    else return T(0.f);
  }
  // unit u of a row of D elements; what is behind the row is 0
  static __device__ __forceinline__ Raw load(const T* row, int u, int D) {
    if constexpr (kVec) {
      if (u * n + n <= D) return load16(row + u * n);
      union {
        uint4 r;
        T x[n];
      } part;
      part.r = zero();
#pragma unroll
      for (int e = 0; e < n; e++)
        if (u * n + e < D) part.x[e] = row[u * n + e];
      return part.r;
    } else {
      return row[u];
    }
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&x)[n]) {
    if constexpr (kVec) Vec16<T>::unpack(r, x);
    else x[0] = to_f32(r);
  }
  static __device__ __forceinline__ void store(T* row, int u, int D, const float (&x)[n]) {
    if constexpr (kVec) {
      const uint4 r = Vec16<T>::pack(x);
      if (u * n + n <= D) {
        *reinterpret_cast<uint4*>(row + u * n) = r;
        return;
      }
#pragma unroll
      for (int e = 0; e < n; e++)
        if (u * n + e < D) from_f32(row + u * n + e, x[e]);
    } else {
      from_f32(row + u, x[0]);
    }
  }
};

// ------------------------------------------------------------------ lookup
// A thread takes kPer units of the N x units outputs, 256 apart, so that kPer choices and then
// kPer units are on their way at once.
template <typename T, bool kVec, int kPer>
__global__ void __launch_bounds__(kEmbedThreads) embed_kernel(EmbedArgs a) {
  using U = Unit<T, kVec>;
  const int64_t first = (int64_t)blockIdx.x * (kPer * kEmbedThreads);
  const int64_t row0 = first <= 0xffffffffll ? (int64_t)((uint32_t)first / (uint32_t)a.units)
                                             : first / a.units;
  const uint32_t unit0 = (uint32_t)(first - row0 * a.units) + threadIdx.x;
  int64_t row[kPer];
  int unit[kPer];
#pragma unroll
  for (int p = 0; p < kPer; p++) {
    const uint32_t i = unit0 + p * kEmbedThreads;
    // (exact: below 1,025 units i is below 2^12, and rows of more are passed at most once)
    const uint32_t q = a.units > kPer * kEmbedThreads ? i >= (uint32_t)a.units
                       : a.units == 1                 ? i
                                                      : __umulhi(i, a.magic);
    row[p] = row0 + q;
    unit[p] = (int)(i - q * a.units);
  }
  auto legal = [&](int k) {
    if ((unsigned)k < (unsigned)a.K) return true;
    if (k != -1 && a.flags) atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
    return false;
  };
  if (a.m == 1) {
    int k[kPer];
    typename U::Raw r[kPer];
    float w[kPer];
#pragma unroll
    for (int p = 0; p < kPer; p++) k[p] = row[p] < a.N ? a.idx[row[p]] : -1;
#pragma unroll
    for (int p = 0; p < kPer; p++) w[p] = a.resp && row[p] < a.N ? a.resp[row[p]] : 1.f;
#pragma unroll
    for (int p = 0; p < kPer; p++) {
      const bool ok = legal(k[p]);
      r[p] = ok ? U::load((const T*)a.W + k[p] * a.ldw, unit[p], a.D) : U::zero();
      if (!ok) w[p] = 0.f;
    }
#pragma unroll
    for (int p = 0; p < kPer; p++) {
      if (row[p] >= a.N) continue;
      float x[U::n];
      U::unpack(r[p], x);
#pragma unroll
      for (int e = 0; e < U::n; e++) x[e] = x[e] * w[p] * a.scale;
      U::store((T*)a.Y + row[p] * a.ldy, unit[p], a.D, x);
    }
    return;
  }
#pragma unroll 1
  for (int p = 0; p < kPer; p++) {
    if (row[p] >= a.N) return;
    float y[U::n] = {};
#pragma unroll 1
    for (int j0 = 0; j0 < a.m; j0 += 4) {
      typename U::Raw r[4];
      float w[4];
      const int64_t at = row[p] * a.m + j0;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const int k = j0 + j < a.m ? a.idx[at + j] : -1;
        const bool ok = legal(k);
        w[j] = !ok ? 0.f : a.resp ? a.resp[at + j] : 1.f;
        r[j] = ok ? U::load((const T*)a.W + k * a.ldw, unit[p], a.D) : U::zero();
      }
#pragma unroll
      for (int j = 0; j < 4; j++) {
        float x[U::n];
        U::unpack(r[j], x);
#pragma unroll
        for (int e = 0; e < U::n; e++) y[e] = fmaf(w[j], x[e], y[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < U::n; e++) y[e] *= a.scale;
    U::store((T*)a.Y + row[p] * a.ldy, unit[p], a.D, y);
  }
}

// ------------------------------------------------------------------ choices sorted by class
// A stable sort of the M = N m choices by class, least significant digit first, one to three
// digits of up to kSortBits bits.  A choice of no class gets class K and ends up behind all
// others.  Per digit two kernels: each CTA counts the digits of its contiguous tile, then (all
// counts known) places its entries.  Warps take contiguous parts of a tile, 32 entries at a
// time; equal digits are ranked by a match across the warp.
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBits = 10;
constexpr int kSortTiles = 148;  // most tiles

struct SortArgs {
  const int32_t* idx;       // the first digit: the choices themselves
  const uint32_t *key, *src;  // later digits: what the one before wrote
  uint32_t *key_out, *src_out;
  uint32_t* counts;         // tiles x bins
  uint8_t* seen;            // K bytes, may be null: which classes are named
  uint32_t M;
  uint32_t per_warp;        // entries, a multiple of 32
  int K, shift, bits;
  uint32_t* flags;
};

__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, uint32_t i) {
  if (!a.idx) return a.key[i];
  const int k = a.idx[i];
  return (unsigned)k < (unsigned)a.K ? (uint32_t)k : (uint32_t)a.K;
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a) {
  __shared__ uint32_t hist[1 << kSortBits];
  const int bins = 1 << a.bits;
  grid_dependents_launch();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) hist[b] = 0;
  grid_dependency_wait();
  if (a.seen)  // (set by the kernel after this one)
    for (int k = blockIdx.x * kSortThreads + threadIdx.x; k < a.K; k += gridDim.x * kSortThreads)
      a.seen[k] = 0;
  __syncthreads();
  const uint64_t begin = (uint64_t)blockIdx.x * kSortWarps * a.per_warp;
  const uint64_t end = min(begin + (uint64_t)kSortWarps * a.per_warp, (uint64_t)a.M);
  for (uint64_t i = begin + threadIdx.x; i < end; i += kSortThreads) {
    const uint32_t k = sort_key(a, (uint32_t)i);
    if (a.idx && k == (uint32_t)a.K && a.idx[i] != -1 && a.flags)
      atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
    atomicAdd(&hist[(k >> a.shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads)
    a.counts[blockIdx.x * bins + b] = hist[b];
}

__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortArgs a) {
  extern __shared__ uint32_t place[];  // [warp][bin]: where the warp's next entry of bin goes
  __shared__ uint32_t sums[kSortWarps];
  const int bins = 1 << a.bits, t = threadIdx.x, lane = t & 31, w = t >> 5;
  grid_dependents_launch();
  for (int i = t; i < kSortWarps * bins; i += kSortThreads) place[i] = 0;
  __syncthreads();
  grid_dependency_wait();
  const uint64_t begin = ((uint64_t)blockIdx.x * kSortWarps + w) * a.per_warp;
  const uint64_t end = min(begin + a.per_warp, (uint64_t)a.M);
  uint32_t* mine = place + w * bins;
  for (uint64_t i0 = begin; i0 < end; i0 += 32) {
    const uint64_t i = i0 + lane;
    if (i < end) atomicAdd(&mine[(sort_key(a, (uint32_t)i) >> a.shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  // Bins in order over the threads: entries of lower bins, then of the same bin in earlier
  // tiles, then in earlier warps.
  uint32_t carry = 0;
  for (int b0 = 0; b0 < bins; b0 += kSortThreads) {
    const int b = b0 + t;
    uint32_t before = 0, all = 0;
    if (b < bins) {
#pragma unroll 8
      for (int tile = 0; tile < (int)gridDim.x; tile++) {
        const uint32_t c = a.counts[tile * bins + b];
        all += c;
        before += tile < (int)blockIdx.x ? c : 0u;
      }
    }
    uint32_t scan = all;  // inclusive over the CTA
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) sums[w] = scan;
    __syncthreads();
    uint32_t lower = carry, total = 0;
    for (int q = 0; q < kSortWarps; q++) {
      if (q < w) lower += sums[q];
      total += sums[q];
    }
    carry += total;
    if (b < bins) {
      uint32_t at = lower + scan - all + before;
      for (int q = 0; q < kSortWarps; q++) {
        const uint32_t c = place[q * bins + b];
        place[q * bins + b] = at;
        at += c;
      }
    }
    __syncthreads();
  }
  for (uint64_t i0 = begin; i0 < end; i0 += 32) {
    const uint64_t i = i0 + lane;
    const bool live = i < end;
    const uint32_t k = live ? sort_key(a, (uint32_t)i) : 0u;
    const uint32_t bin = (k >> a.shift) & (bins - 1);
    const uint32_t equal = __match_any_sync(0xffffffffu, live ? bin : 0xffffffffu);
    const uint32_t rank = __popc(equal & ((1u << lane) - 1u));
    uint32_t at = 0;
    if (live) at = mine[bin] + rank;
    __syncwarp();
    if (live && rank == 0) mine[bin] = at + __popc(equal);
    __syncwarp();
    if (live) {
      a.key_out[at] = k;
      a.src_out[at] = a.idx ? (uint32_t)i : a.src[i];
      if (a.seen && k < (uint32_t)a.K) a.seen[k] = 1;
    }
  }
}

// ------------------------------------------------------------------ sums by class
// The sorted choices in chunks.  A group of `lanes` threads takes a chunk and `lanes` units of the
// rows, and adds up runs of equal class.  A run inside the chunk is a row of dW; one that the
// chunk's border cuts leaves its sum (at most two per chunk: of the run that came in, and of the
// one that goes on), and a second kernel adds those up, in order.  A class that is named a
// million times is so many chunks, each its own group's.
struct EmbedGradArgs {
  const void* dY;
  const float* resp;       // may be null
  const uint32_t *key, *src;
  const uint8_t* seen;     // null: dW is added to
  void* dW;
  float* part;             // chunks x 2 x width
  int64_t ldy, ldd;
  uint64_t by_m;           // ceil(2^34 / m)
  uint32_t M, chunk, chunks;
  int K, D, units, lanes, width;
  float scale;
  int m;
};

template <typename T, typename TO, bool kVec>
__device__ __forceinline__ void write_grad(const EmbedGradArgs& a, uint32_t k, int u,
                                           const float (&sum)[Unit<T, kVec>::n]) {
  constexpr int n = Unit<T, kVec>::n;
  TO* row = (TO*)a.dW + (int64_t)k * a.ldd;
  float x[n];
#pragma unroll
  for (int e = 0; e < n; e++) x[e] = sum[e] * a.scale;
  if constexpr (std::is_same<T, TO>::value) {
    if (!a.seen) {
      float old[n];
      Unit<T, kVec>::unpack(Unit<T, kVec>::load(row, u, a.D), old);
#pragma unroll
      for (int e = 0; e < n; e++) x[e] += old[e];
    }
    Unit<T, kVec>::store(row, u, a.D, x);
  } else {  // a float32 gradient of narrower rows: 32 bytes per unit
#pragma unroll
    for (int e = 0; e < n; e += 4) {
      if (kVec && u * n + e + 4 <= a.D) {
        float4* p = reinterpret_cast<float4*>(row + u * n + e);
        float4 v = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        if (!a.seen) {
          const float4 o = *p;
          v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
        }
        *p = v;
      } else {
#pragma unroll
        for (int i = e; i < e + 4 && i < n; i++)
          if (u * n + i < a.D) row[u * n + i] = a.seen ? x[i] : x[i] + row[u * n + i];
      }
    }
  }
}

constexpr int kGradBatch = 8;

template <typename T, typename TO, bool kVec>
__global__ void __launch_bounds__(kEmbedThreads) embed_sum_kernel(EmbedGradArgs a) {
  using U = Unit<T, kVec>;
  grid_dependents_launch();
  grid_dependency_wait();
  const int l = threadIdx.x & (a.lanes - 1);
  const uint32_t c = blockIdx.x * (kEmbedThreads / a.lanes) + threadIdx.x / a.lanes;
  const int u = blockIdx.y * a.lanes + l;
  if (c >= a.chunks || u >= a.units) return;
  const uint32_t begin = c * a.chunk, end = min(begin + a.chunk, a.M);
  bool came_in = begin > 0 && a.key[begin - 1] == a.key[begin];
  float sum[U::n] = {};
  for (uint32_t i = begin; i < end; i += kGradBatch) {
    uint32_t k[kGradBatch + 1], s[kGradBatch];
    typename U::Raw r[kGradBatch];
    float w[kGradBatch];
#pragma unroll
    for (int b = 0; b < kGradBatch; b++) {
      k[b] = i + b < end ? a.key[i + b] : a.K;
      s[b] = i + b < end ? a.src[i + b] : 0u;
    }
    // (the entry behind the batch, in the next chunk or not)
    k[kGradBatch] = i + kGradBatch < a.M ? a.key[i + kGradBatch] : a.K;
#pragma unroll
    for (int b = 0; b < kGradBatch; b++) {
      const bool live = k[b] < (uint32_t)a.K;
      const int64_t n = a.m == 1 ? s[b] : (int64_t)((s[b] * a.by_m) >> 34);
      r[b] = live ? U::load((const T*)a.dY + n * a.ldy, u, a.D) : U::zero();
      w[b] = live && a.resp ? a.resp[s[b]] : 1.f;
    }
#pragma unroll
    for (int b = 0; b < kGradBatch; b++) {
      if (k[b] >= (uint32_t)a.K) continue;
      float x[U::n];
      U::unpack(r[b], x);
#pragma unroll
      for (int e = 0; e < U::n; e++) sum[e] = fmaf(w[b], x[e], sum[e]);
      const bool last = i + b + 1 == end;
      // (past `end` inside a batch k says none: look at the entry itself)
      const bool goes_on =
          last ? end < a.M && a.key[end] == k[b] : k[b + 1] == k[b];
      if (goes_on && !last) continue;
      if (came_in || goes_on) {
        float* p = a.part + ((int64_t)c * 2 + (came_in ? 0 : 1)) * a.width + u * U::n;
        if constexpr (kVec) {
#pragma unroll
          for (int e = 0; e < U::n; e += 4)
            *reinterpret_cast<float4*>(p + e) =
                make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
        } else {
          p[0] = sum[0];
        }
      } else {
        write_grad<T, TO, kVec>(a, k[b], u, sum);
      }
      came_in = false;
#pragma unroll
      for (int e = 0; e < U::n; e++) sum[e] = 0.f;
    }
  }
}

// Blocks [0, chunks): the sums of the run that begins in a chunk and goes on behind it, 32 units
// at a time by 8 warps, which share out the run's chunks.  Blocks behind those: rows of classes
// that nothing names get zeros.
constexpr int kFillRows = 64;

template <typename T, typename TO, bool kVec>
__global__ void __launch_bounds__(kEmbedThreads) embed_finish_kernel(EmbedGradArgs a,
                                                                     uint32_t joins) {
  using U = Unit<T, kVec>;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  constexpr int kWarps = kEmbedThreads / 32;
  grid_dependency_wait();
  if (blockIdx.x >= joins) {
    const int k0 = (int)(blockIdx.x - joins) * kFillRows;
    constexpr int V = kVec ? 16 / (int)sizeof(TO) : 1;
    const int units = (a.D + V - 1) / V;
    const int per = units >= 256 ? 256 : units > 16 ? 32 : 8;  // threads of a row
    const int l = threadIdx.x & (per - 1);
    for (int q = threadIdx.x / per; q < kFillRows && k0 + q < a.K; q += kEmbedThreads / per) {
      if (a.seen[k0 + q]) continue;
      TO* row = (TO*)a.dW + (int64_t)(k0 + q) * a.ldd;
      const float zero[V] = {};
      for (int u = l; u < units; u += per) Unit<TO, kVec>::store(row, u, a.D, zero);
    }
    return;
  }
  __shared__ float sh[kWarps][32 * U::n];
  const uint32_t c = blockIdx.x;
  const uint32_t begin = c * a.chunk, end = begin + a.chunk;
  if (end >= a.M) return;
  const uint32_t k = a.key[end - 1];
  if (k >= (uint32_t)a.K || a.key[end] != k) return;                   // nothing goes on
  if (a.key[begin] == k && begin > 0 && a.key[begin - 1] == k) return;  // it began before
  // the run's last chunk: the first whose last entry is of another class, or the last of all
  uint32_t lo = c + 1, hi = a.chunks - 1;
  while (lo < hi) {
    const uint32_t step = (hi - lo + 31) / 32, at = min(lo + step * lane, hi);
    const bool past = at == hi || a.key[(uint64_t)(at + 1) * a.chunk] != k;
    const int f = __ffs(__ballot_sync(0xffffffffu, past)) - 1;
    const uint32_t found = f < 0 ? hi : min(lo + step * f, hi);
    const uint32_t from = f == 0 ? lo : f < 0 ? lo + step * 31 + 1 : lo + step * (f - 1) + 1;
    hi = found;
    lo = min(from, hi);
  }
  const uint32_t last = lo;
  for (int u0 = 0; u0 < a.units; u0 += 32) {
    const int u = u0 + lane;
    float sum[U::n] = {};
    if (u < a.units) {
#pragma unroll 4
      for (uint32_t q = c + w; q <= last; q += kWarps) {
        const float* p = a.part + ((int64_t)q * 2 + (q == c ? 1 : 0)) * a.width + u * U::n;
#pragma unroll
        for (int e = 0; e < U::n; e++) sum[e] += p[e];
      }
    }
#pragma unroll
    for (int e = 0; e < U::n; e++) sh[w][lane * U::n + e] = sum[e];
    __syncthreads();
    if (w == 0 && u < a.units) {
      for (int q = 1; q < kWarps; q++) {
#pragma unroll
        for (int e = 0; e < U::n; e++) sum[e] += sh[q][lane * U::n + e];
      }
      write_grad<T, TO, kVec>(a, k, u, sum);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ gradient of the weights
// A group of 8 or 32 lanes per row n: <dY_n, W[idx_nj]> for its m choices, in a fixed order.
struct EmbedDotArgs {
  const void *W, *dY;
  const int32_t* idx;
  float* dresp;
  int64_t N, ldw, ldy;
  int m, K, D, units;
  float scale;
  uint32_t* flags;
};

template <typename T, bool kVec, int kLanes, int kMost>
__global__ void __launch_bounds__(kEmbedThreads) embed_dot_kernel(EmbedDotArgs a) {
  using U = Unit<T, kVec>;
  grid_dependents_launch();
  grid_dependency_wait();
  const int l = threadIdx.x % kLanes;
  const int64_t step = (int64_t)gridDim.x * (kEmbedThreads / kLanes);
  for (int64_t n0 = ((int64_t)blockIdx.x * kEmbedThreads + threadIdx.x) / 32 * (32 / kLanes);
       n0 < a.N; n0 += step) {  // (whole warps)
    const int64_t n = n0 + (threadIdx.x & 31) / kLanes;
    int k[kMost];
    float dot[kMost] = {};
#pragma unroll
    for (int j = 0; j < kMost; j++) {
      k[j] = n < a.N && j < a.m ? a.idx[n * a.m + j] : -1;
      if ((unsigned)k[j] >= (unsigned)a.K) {
        if (k[j] != -1 && a.flags) atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
        k[j] = -1;
      }
    }
    if (n < a.N) {
      for (int u = l; u < a.units; u += kLanes) {
        const typename U::Raw y = U::load((const T*)a.dY + n * a.ldy, u, a.D);
        typename U::Raw r[kMost];
#pragma unroll
        for (int j = 0; j < kMost; j++)
          r[j] = k[j] >= 0 ? U::load((const T*)a.W + k[j] * a.ldw, u, a.D) : U::zero();
        float yx[U::n];
        U::unpack(y, yx);
#pragma unroll
        for (int j = 0; j < kMost; j++) {
          float x[U::n];
          U::unpack(r[j], x);
#pragma unroll
          for (int e = 0; e < U::n; e++) dot[j] = fmaf(yx[e], x[e], dot[j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kMost; j++) {
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1)
        dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
      if (l == 0 && n < a.N && j < a.m) a.dresp[n * a.m + j] = k[j] < 0 ? 0.f : dot[j] * a.scale;
    }
  }
}

}  // namespace scem
