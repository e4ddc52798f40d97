// embed.cuh -- rows of a table chosen by an assignment, and the gradient by sorted classes:
// kernels of gmm_embed and gmm_embed_backward.
//
//   Y_n = scale sum_j r_nj W[idx_nj]              (r = 1 without weights)
//   dW_k = scale sum_{(n,j): idx_nj = k} r_nj dY_n
//   dr_nj = scale <dY_n, W[idx_nj]>
// Sums are held in float32 (of many chunks in 64 bits) and rounded once.  Everything is bound by
// memory: the named rows and the output go through once.  Measured figures are of one B200, calls
// back to back, beside the time of the bytes alone at the rate of a large copy (6,548 GB/s).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "sm100_prims.cuh"
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
  int units, lane_bits;
  uint32_t* flags;
};

// What a lane takes of a row at once, a unit.  kMode 1 and 2, rows that start on 16 bytes: 16
// bytes of T, the last unit perhaps a part (1) or whole as well (2: D is a multiple).  kMode 0,
// rows that start anywhere: four elements, as far apart as there are lanes, so that a warp's
// accesses lie together.
template <typename T, int kMode>
struct Unit {
  static constexpr bool kVec = kMode > 0;
  static constexpr int n = kVec ? Vec16<T>::n : 4;
  struct Elements {
    T x[n];
  };
  using Raw = typename std::conditional<kVec, uint4, Elements>::type;
  // The first element of lane l, of `lanes` that take units first, first + 1, ...
  static __device__ __forceinline__ int at(int first, int l, int lanes) {
    return kVec ? (first + l) * n : first * n + l;
  }
  static __device__ __forceinline__ Raw zero() {
    if constexpr (kVec) {
      return make_uint4(0, 0, 0, 0);
    } else {
      Raw r;
#pragma unroll
      for (int e = 0; e < n; e++) r.x[e] = T(0.f);
      return r;
    }
  }
  // The unit at element i of a row of D; what is behind the row is 0.
  static __device__ __forceinline__ Raw load(const T* row, int i, int lanes, int D) {
    if constexpr (!kVec) {
      Raw r;
      const T* p = row + i;
      if (i + (n - 1) * lanes < D) {
#pragma unroll
        for (int e = 0; e < n; e++, p += lanes) r.x[e] = *p;
      } else {
#pragma unroll
        for (int e = 0; e < n; e++, p += lanes) r.x[e] = i + e * lanes < D ? *p : T(0.f);
      }
      return r;
    } else {
      if (kMode == 2 || i + n <= D) return load16(row + i);
      union {
        uint4 r;
        T x[n];
      } part;
      part.r = zero();
#pragma unroll
      for (int e = 0; e < n; e++)
        if (i + e < D) part.x[e] = row[i + e];
      return part.r;
    }
  }
  static __device__ __forceinline__ void unpack(const Raw& r, float (&x)[n]) {
    if constexpr (kVec) {
      Vec16<T>::unpack(r, x);
    } else {
#pragma unroll
      for (int e = 0; e < n; e++) x[e] = to_f32(r.x[e]);
    }
  }
  // kStream: not read again soon by this kernel (the table stays in L2).
  template <bool kStream = false>
  static __device__ __forceinline__ void store(T* row, int i, int lanes, int D,
                                               const float (&x)[n]) {
    if constexpr (!kVec) {
      T* p = row + i;
      if (i + (n - 1) * lanes < D) {
#pragma unroll
        for (int e = 0; e < n; e++, p += lanes) from_f32(p, x[e]);
      } else {
#pragma unroll
        for (int e = 0; e < n; e++, p += lanes)
          if (i + e * lanes < D) from_f32(p, x[e]);
      }
    } else {
      if (kMode == 2 || i + n <= D) {
        if (kStream) __stcs(reinterpret_cast<uint4*>(row + i), Vec16<T>::pack(x));
        else *reinterpret_cast<uint4*>(row + i) = Vec16<T>::pack(x);
      } else {
#pragma unroll
        for (int e = 0; e < n; e++)
          if (i + e < D) from_f32(row + i + e, x[e]);
      }
    }
  }
};

// ------------------------------------------------------------------ lookup
// 2^lane_bits lanes per row; a lane takes kPer units of it, a row's lanes apart, so that a row's
// choices and addresses are formed once for kPer * kM units, all on their way at once.  Blocks y:
// where a row has more units than that.  kM: at least m.
//
// 1e6 rows of 96 fp32, two of 4,096 entries each: 79 to 89 us (61 us of bytes), at no one limit
// (2.7 of 4 instructions a clock, 65 % of the warps resident, 4.0 TB/s of mostly writes); with a
// thread per unit, indices and addresses formed for each, 117 to 209.  16,384 of 131,072 rows of
// 2,048 bf16: 13 us.  8 rows of those: 1.5 us.  Rows that start anywhere go element by element:
// 239,198 of 185 bf16 take 39 us (14 us of bytes).
template <typename T, int kMode, int kM, int kPer>
__global__ void __launch_bounds__(kEmbedThreads) embed_kernel(EmbedArgs a) {
  using U = Unit<T, kMode>;
  const int lanes = 1 << a.lane_bits, l = threadIdx.x & (lanes - 1);
  const int64_t row =
      (int64_t)blockIdx.x * (kEmbedThreads >> a.lane_bits) + (threadIdx.x >> a.lane_bits);
  auto at = [&](int p) { return U::at((int)(blockIdx.y * kPer + p) << a.lane_bits, l, lanes); };
  grid_dependency_wait();
  grid_dependents_launch();
  if (row >= a.N) return;
  int k[kM];
  float w[kM];
#pragma unroll
  for (int j = 0; j < kM; j++) {
    const bool live = kM == 1 || j < a.m;
    const int64_t c = kM == 1 ? row : row * a.m + j;
    k[j] = live ? a.idx[c] : -1;
    w[j] = live && a.resp ? a.resp[c] : 1.f;
  }
  typename U::Raw r[kPer][kM];
#pragma unroll
  for (int j = 0; j < kM; j++) {
    const bool ok = (unsigned)k[j] < (unsigned)a.K;
    if (!ok) {
      if (k[j] != -1 && a.flags) atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
      w[j] = 0.f;
    }
    w[j] *= a.scale;
    const T* from = (const T*)a.W + (ok ? k[j] : 0) * a.ldw;
#pragma unroll
    for (int p = 0; p < kPer; p++)
      r[p][j] = ok && at(p) < a.D ? U::load(from, at(p), lanes, a.D) : U::zero();
  }
  T* to = (T*)a.Y + row * a.ldy;
#pragma unroll
  for (int p = 0; p < kPer; p++) {
    if (at(p) >= a.D) return;
    F2 sum[U::n / 2];
#pragma unroll
    for (int j = 0; j < kM; j++) {
      float x[U::n];
      U::unpack(r[p][j], x);
#pragma unroll
      for (int e = 0; e < U::n; e += 2) {
        const F2 x2 = f2(x[e], x[e + 1]), w2 = f2(w[j], w[j]);
        sum[e / 2] = j == 0 ? f2_mul(x2, w2) : f2_fma(x2, w2, sum[e / 2]);
      }
    }
    float y[U::n];
#pragma unroll
    for (int e = 0; e < U::n; e += 2) f2_get(sum[e / 2], y[e], y[e + 1]);
    U::template store<true>(to, at(p), lanes, a.D, y);
  }
}

// ------------------------------------------------------------------ choices sorted by class
// A stable sort of the M = N m choices by class, least significant digit first, one to three
// digits of up to kSortBits bits.  A choice of no class gets class K and ends up behind all
// others.  Warps take contiguous parts of the choices, 32 at a time; equal digits are ranked by a
// match across the warp.
//
// Up to kSortCluster choices one cluster of CTAs does all of it, with its barriers between the
// steps, and leaves the other SMs to whatever else the gradient needs.  Beyond, two kernels per
// digit: each CTA counts the digits of its contiguous tile, then (all counts known) places its
// entries.  (With rows of 8 fp32 behind it, 131,072 choices of 4,096 classes take 34 us by the
// cluster and 35 by two kernels per digit, 16,384 18 and 22, 262,144 59 and 45.)  Bound by the
// latency of each step, and in the cluster by what 16 SMs can scatter.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortBits = 10;
constexpr int kSortTiles = 148;  // most tiles
constexpr int kClusterThreads = 1024;
constexpr int kClusterWarps = kClusterThreads / 32;
constexpr uint32_t kSortCluster = 1u << 17;

// What lets a kernel go on beside the sort before it in the stream.  Only a wait is sure to make
// visible what came before, and the sort has waited: its first kernel then stores a token of the call
// (release), and who reads it (acquire) sees all that the sort could see.  Who does not waits for the
// sort.  The sums take the word back, so that a replayed call does not find its own token.
struct Beside {
  unsigned long long *word, token;  // word: in the workspace, or null: nothing goes on beside
};
__device__ __forceinline__ void beside_allow(const Beside& b) {
  if (b.word && blockIdx.x == 0 && threadIdx.x == 0)
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(b.word), "l"(b.token) : "memory");
}
__device__ __forceinline__ void beside_wait(const Beside& b) {
  unsigned long long seen = 0;
  if (b.word)
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(seen) : "l"(b.word) : "memory");
  if (!b.word || seen != b.token) grid_dependency_wait();
}

// A choice on its way: its class and its place in idx.
using Choice = uint2;

struct SortArgs {
  const int32_t* idx;  // the first digit: the choices themselves
  const Choice* in;    // later digits: what the one before wrote
  Choice* out;
  uint32_t* counts;    // tiles x bins
  uint8_t* seen;       // K bytes with the first digit, or null: which classes are named
  uint32_t M;
  uint32_t per_warp;          // entries, a multiple of 32
  int K, shift, bits;
  uint32_t* flags;
  Beside beside;              // with the first digit
};

// Entries i0 + 32 b + lane of a warp's part, b < kSortBatch, all on their way at once; class K
// where there is none.
constexpr int kSortBatch = 8;
__device__ __forceinline__ void sort_fetch(const int32_t* idx, const Choice* in, uint64_t i0,
                                           uint64_t end, uint32_t K, uint32_t* flags,
                                           Choice (&c)[kSortBatch]) {
  i0 += threadIdx.x & 31;
#pragma unroll
  for (int b = 0; b < kSortBatch; b++) {
    const uint64_t i = i0 + 32 * b;
    c[b] = make_uint2(K, 0);
    if (i < end) c[b] = idx ? make_uint2((uint32_t)idx[i], (uint32_t)i) : __ldcg(in + i);
  }
  if (!idx) return;
#pragma unroll
  for (int b = 0; b < kSortBatch; b++) {
    if (c[b].x < K) continue;
    if (c[b].x != 0xffffffffu && i0 + 32 * b < end && flags)
      atomicOr(flags, GMM_DEVFLAG_BAD_INDEX);
    c[b].x = K;
  }
}

// K bytes of 0 (on 16 bytes, room up to the next 16), by threads of index t of n.
__device__ __forceinline__ void clear_seen(uint8_t* seen, int K, int t, int n) {
  uint4* v = reinterpret_cast<uint4*>(seen);
  for (int i = t; i < (K + 15) / 16; i += n) v[i] = make_uint4(0, 0, 0, 0);
}

// A class that is named.  (Looked at first: a frequent one would have a hundred thousand stores
// wait for one place in memory.)
__device__ __forceinline__ void mark_seen(uint8_t* seen, uint32_t k) {
  if (!seen[k]) seen[k] = 1;
}

// The warp's 32 entries to their places, in order: `next` holds where each bin's next entry goes.
__device__ __forceinline__ void sort_put(uint32_t* next, bool live, Choice c, uint32_t bin,
                                         Choice* out) {
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t equal = __match_any_sync(0xffffffffu, live ? bin : 0xffffffffu);
  const uint32_t rank = __popc(equal & ((1u << lane) - 1u));
  uint32_t at = 0;
  if (live) at = next[bin] + rank;
  __syncwarp();
  if (live && rank == 0) next[bin] = at + __popc(equal);
  __syncwarp();
  if (live) out[at] = c;
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(SortArgs a) {
  __shared__ uint32_t hist[1 << kSortBits];
  const int bins = 1 << a.bits;
  for (int b = threadIdx.x; b < bins; b += kSortThreads) hist[b] = 0;
  __syncthreads();
  grid_dependency_wait();
  beside_allow(a.beside);
  grid_dependents_launch();
  if (a.seen)
    clear_seen(a.seen, a.K, blockIdx.x * kSortThreads + threadIdx.x, gridDim.x * kSortThreads);
  const uint64_t begin = ((uint64_t)blockIdx.x * kSortWarps + threadIdx.x / 32) * a.per_warp;
  const uint64_t end = min(begin + a.per_warp, (uint64_t)a.M);
  for (uint64_t i0 = begin; i0 < end; i0 += 32 * kSortBatch) {
    Choice c[kSortBatch];
    sort_fetch(a.idx, a.in, i0, end, (uint32_t)a.K, a.flags, c);
#pragma unroll
    for (int b = 0; b < kSortBatch; b++)
      if (i0 + 32 * b + (threadIdx.x & 31) < end)
        atomicAdd(&hist[(c[b].x >> a.shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads)
    a.counts[blockIdx.x * bins + b] = hist[b];
}

__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(SortArgs a) {
  extern __shared__ uint32_t place[];  // [warp][bin]: where the warp's next entry of bin goes
  __shared__ uint32_t sums[kSortWarps], of_bin[2][kSortThreads];
  const int bins = 1 << a.bits, t = threadIdx.x, lane = t & 31, w = t >> 5;
  for (int i = t; i < kSortWarps * bins; i += kSortThreads) place[i] = 0;
  __syncthreads();
  grid_dependency_wait();
  grid_dependents_launch();
  const uint64_t begin = min(((uint64_t)blockIdx.x * kSortWarps + w) * a.per_warp, (uint64_t)a.M);
  const uint64_t end = min(begin + a.per_warp, (uint64_t)a.M);
  uint32_t* mine = place + w * bins;
  Choice c[kSortBatch];
  for (uint64_t i0 = begin; i0 < end; i0 += 32 * kSortBatch) {
    sort_fetch(a.idx, a.in, i0, end, (uint32_t)a.K, nullptr, c);
#pragma unroll
    for (int b = 0; b < kSortBatch; b++)
      if (i0 + 32 * b + lane < end) atomicAdd(&mine[(c[b].x >> a.shift) & (bins - 1)], 1u);
  }
  // Bins in order over the threads: entries of lower bins, then of the same bin in earlier
  // tiles, then in earlier warps.  With few bins several threads share a bin's tiles.
  const int cols = min(bins, kSortThreads), groups = kSortThreads / cols;
  const int col = t & (cols - 1), tiles = (int)gridDim.x;
  uint32_t carry = 0;
  for (int b0 = 0; b0 < bins; b0 += cols) {
    uint32_t before = 0, all = 0;
    constexpr int kAhead = 20;  // counts on their way at once
    for (int tile0 = t / cols; tile0 < tiles; tile0 += kAhead * groups) {
      uint32_t n[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; q++) {
        const int tile = tile0 + q * groups;
        n[q] = tile < tiles ? __ldcg(a.counts + tile * bins + b0 + col) : 0u;
      }
#pragma unroll
      for (int q = 0; q < kAhead; q++) {
        all += n[q];
        before += tile0 + q * groups < (int)blockIdx.x ? n[q] : 0u;
      }
    }
    of_bin[0][t] = all;
    of_bin[1][t] = before;
    __syncthreads();
    if (t < cols) {
      for (int g = 1; g < groups; g++) {
        all += of_bin[0][g * cols + t];
        before += of_bin[1][g * cols + t];
      }
    } else {
      all = 0;
    }
    uint32_t scan = all;  // inclusive over the CTA
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) sums[w] = scan;
    __syncthreads();
    static_assert(kSortWarps == 32, "a lane for each warp's sum");
    const uint32_t lower = carry + __reduce_add_sync(0xffffffffu, lane < w ? sums[lane] : 0u);
    carry += __reduce_add_sync(0xffffffffu, sums[lane]);
    if (t < cols) {
      uint32_t at = lower + scan - all + before;
#pragma unroll
      for (int q0 = 0; q0 < kSortWarps; q0 += 8) {
        uint32_t n[8];
#pragma unroll
        for (int q = 0; q < 8; q++) n[q] = place[(q0 + q) * bins + b0 + t];
#pragma unroll
        for (int q = 0; q < 8; q++) {
          place[(q0 + q) * bins + b0 + t] = at;
          at += n[q];
        }
      }
    }
    __syncthreads();
  }
  for (uint64_t i0 = begin; i0 < end; i0 += 32 * kSortBatch) {
    if (a.per_warp > 32 * kSortBatch)  // (else they are still here)
      sort_fetch(a.idx, a.in, i0, end, (uint32_t)a.K, nullptr, c);
#pragma unroll
    for (int b = 0; b < kSortBatch; b++) {
      if (i0 + 32 * b >= end) break;  // (the same for the warp)
      if (a.seen && c[b].x < (uint32_t)a.K) mark_seen(a.seen, c[b].x);
      sort_put(mine, i0 + 32 * b + lane < end, c[b], (c[b].x >> a.shift) & (bins - 1), a.out);
    }
  }
}

// All digits by one cluster: per warp and bin first the counts, then the places.  The counts of
// the CTAs meet in shared memory.
struct SortAllArgs {
  const int32_t* idx;
  Choice* list[2];  // digit i writes buffer i & 1
  uint8_t* seen;    // K bytes, or null: which classes are named
  uint32_t M, per_warp;
  int K, passes, bits;
  uint32_t* flags;
  Beside beside;
};

__global__ void __launch_bounds__(kClusterThreads, 1) sort_cluster_kernel(SortAllArgs a) {
  extern __shared__ uint32_t place[];  // [warp][bin], then the CTA's counts [bin]
  __shared__ uint32_t sums[kClusterWarps];
  const int bins = 1 << a.bits, t = threadIdx.x, lane = t & 31, w = t >> 5;
  const uint32_t rank = sm100::cluster_ctarank(), ctas = sm100::cluster_nctarank();
  uint32_t* mine = place + w * bins;
  uint32_t* total = place + kClusterWarps * bins;
  const uint64_t begin = min(((uint64_t)rank * kClusterWarps + w) * a.per_warp, (uint64_t)a.M);
  const uint64_t end = min(begin + a.per_warp, (uint64_t)a.M);
  grid_dependency_wait();
  beside_allow(a.beside);
  grid_dependents_launch();
  if (a.seen) clear_seen(a.seen, a.K, rank * kClusterThreads + t, ctas * kClusterThreads);
  for (int pass = 0; pass < a.passes; pass++) {
    const int shift = pass * a.bits;
    const int32_t* idx = pass == 0 ? a.idx : nullptr;
    const Choice* in = a.list[(pass + 1) & 1];
    Choice c[kSortBatch];
    for (int i = lane; i < bins; i += 32) mine[i] = 0;
    __syncwarp();
    for (uint64_t i0 = begin; i0 < end; i0 += 32 * kSortBatch) {
      sort_fetch(idx, in, i0, end, (uint32_t)a.K, a.flags, c);
#pragma unroll
      for (int b = 0; b < kSortBatch; b++)
        if (i0 + 32 * b + lane < end) atomicAdd(&mine[(c[b].x >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    for (int b = t; b < bins; b += kClusterThreads) {
      uint32_t n = 0;
#pragma unroll 8
      for (int q = 0; q < kClusterWarps; q++) n += place[q * bins + b];
      total[b] = n;
    }
    __syncwarp();
    sm100::cluster_sync();
    static_assert((1 << kSortBits) <= kClusterThreads, "a thread for each bin");
    uint32_t before = 0, all = 0;
    if (t < bins) {
#pragma unroll 8
      for (uint32_t r = 0; r < ctas; r++) {
        uint32_t n;
        asm volatile("ld.shared::cluster.u32 %0, [%1];"
                     : "=r"(n)
                     : "r"(sm100::map_to_rank(sm100::smem_u32(total + t), r))
                     : "memory");
        all += n;
        before += r < rank ? n : 0u;
      }
    }
    uint32_t scan = all;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) sums[w] = scan;
    __syncthreads();
    uint32_t lower = lane < w ? sums[lane] : 0u;
    lower = __reduce_add_sync(0xffffffffu, lower);
    if (t < bins) {
      uint32_t at = lower + scan - all + before;
      for (int q0 = 0; q0 < kClusterWarps; q0 += 8) {
        uint32_t n[8];
#pragma unroll
        for (int q = 0; q < 8; q++) n[q] = place[(q0 + q) * bins + t];
#pragma unroll
        for (int q = 0; q < 8; q++) {
          place[(q0 + q) * bins + t] = at;
          at += n[q];
        }
      }
    }
    __syncthreads();
    for (uint64_t i0 = begin; i0 < end; i0 += 32 * kSortBatch) {
      if (a.per_warp > 32 * kSortBatch)  // (else they are still here)
        sort_fetch(idx, in, i0, end, (uint32_t)a.K, nullptr, c);
#pragma unroll
      for (int b = 0; b < kSortBatch; b++) {
        if (i0 + 32 * b >= end) break;  // (the same for the warp)
        if (idx && a.seen && c[b].x < (uint32_t)a.K) mark_seen(a.seen, c[b].x);
        sort_put(mine, i0 + 32 * b + lane < end, c[b], (c[b].x >> shift) & (bins - 1),
                 a.list[pass & 1]);
      }
    }
    // what the others placed is visible, and nobody's counts are read any more
    __syncwarp();
    sm100::cluster_sync();
  }
}

// ------------------------------------------------------------------ rows of zeros
// Rows [0, rows) beside the sort, before it is known which are named; pieces of a row, one per
// warp.  Does not wait for the sort before it in the stream (Beside), only ends after it: nothing
// that is written here is read or written there.  (The rows behind, of classes that nothing names,
// get their zeros with the sums.)
constexpr int kFillPiece = 16384;  // bytes
// CTAs per SM of a kernel that goes on beside the sort and ends after it: all of them are resident
// at once, also beside the sort's (one that waits keeps its place).
constexpr int kBesideCtas = 4;
struct FillArgs {
  char* base;
  uint64_t rows, row_bytes, stride;  // bytes
  uint64_t parts;                    // pieces per row
  Beside beside;
};

// n bytes of 0, by a warp.
__device__ __forceinline__ void zero_bytes(char* p, uint64_t n) {
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t head = (uint32_t)min(n, (uint64_t)(-(uintptr_t)p & 15u));
  const uint64_t body = (n - head) / 16;
  if (lane < head) p[lane] = 0;
  uint4* v = reinterpret_cast<uint4*>(p + head);
#pragma unroll 4
  for (uint64_t u = lane; u < body; u += 32) v[u] = make_uint4(0, 0, 0, 0);
  if (lane < n - head - body * 16) p[head + body * 16 + lane] = 0;
}

__global__ void __launch_bounds__(kEmbedThreads) embed_fill_kernel(FillArgs a) {
  grid_dependents_launch();
  beside_wait(a.beside);
  const uint64_t pieces = a.rows * a.parts;
  for (uint64_t i = (uint64_t)blockIdx.x * (kEmbedThreads / 32) + threadIdx.x / 32; i < pieces;
       i += (uint64_t)gridDim.x * (kEmbedThreads / 32)) {
    const uint64_t row = a.rows == 1 ? 0 : a.parts == 1 ? i : i / a.parts;
    const uint64_t at = (i - row * a.parts) * kFillPiece;
    zero_bytes(a.base + row * a.stride + at, min((uint64_t)kFillPiece, a.row_bytes - at));
  }
  grid_dependency_wait();
}

// ------------------------------------------------------------------ sums by class
// The sorted choices in chunks.  A group of `lanes` threads takes a chunk and `lanes` units of the
// rows, and adds up runs of equal class.  A run inside the chunk is a row of dW; one that the
// chunk's border cuts leaves its sum (at most two per chunk: of the run that came in, and of the
// one that goes on), and a second kernel adds those up, in order.  A class that is named a
// million times is so many chunks, each its own group's.
//
// The gradient of 131,072 x 2,048 bf16 from 16,384 tokens takes 102 to 105 us (92 us of bytes): the
// sort with the first zeros beside it 20, the sums with the other zeros 73 at 6.3 TB/s, the cut
// runs 6.  All zeros beside the sort and the sums behind them: 116.  200,001 rows of 96 fp32 with
// two of 4,096 entries each, added to what is there, and the weights' gradient: 74 to 76 us (13
// us of bytes): sort 21, weights 22, sums 26, cut runs 6; bound by the sort's latency and by
// reading each row of dY three times, out of L2 all but once.  (The weights' gradient with the
// sums, dY read twice: 80; the sums over a group of lanes cost more than the reading.)
struct EmbedGradArgs {
  const void* dY;
  const float* resp;       // may be null
  const Choice* list;      // sorted
  void* dW;
  float* part;             // chunks x 2 x width
  int64_t ldy, ldd;
  uint64_t by_m;           // ceil(2^34 / m)
  uint32_t M, chunk, chunks;
  int K, D, units, lanes, width;
  float scale;
  int m, add;
  // zeros for rows from fill_from on that `seen` does not name: blocks of fill_rows rows, the first
  // fill_first of them before the sums' blocks, the others behind
  const uint8_t* seen;
  int fill_from, fill_rows;
  uint32_t fill_first, sum_blocks;
  unsigned long long* beside;  // Beside's word
};

// Adds to float32 memory without waiting for what is there.  (An element is added to once in a
// call, so this is old + x rounded once, whatever the order; subnormal values count as 0.)
__device__ __forceinline__ void red_add(float* p, float x) {
  asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(p), "f"(x) : "memory");
}
__device__ __forceinline__ void red_add4(float* p, float4 x) {
  asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(x.x),
               "f"(x.y), "f"(x.z), "f"(x.w)
               : "memory");
}

// scale * sum to, or added to, row k's unit at element i.
template <typename T, typename TO, int kMode>
__device__ __forceinline__ void write_grad(const EmbedGradArgs& a, uint32_t k, int i, int lanes,
                                           const float (&sum)[Unit<T, kMode>::n]) {
  constexpr int n = Unit<T, kMode>::n;
  TO* row = (TO*)a.dW + (int64_t)k * a.ldd;
  float x[n];
#pragma unroll
  for (int e = 0; e < n; e++) x[e] = sum[e] * a.scale;
  if constexpr (std::is_same<TO, float>::value) {  // (units of T: 16 or 32 bytes of dW)
    if constexpr (kMode == 0) {
#pragma unroll
      for (int e = 0; e < n; e++) {
        if (i + e * lanes >= a.D) continue;
        if (a.add) red_add(row + i + e * lanes, x[e]);
        else row[i + e * lanes] = x[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < n; e += 4) {
        const float4 v = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
        if (kMode == 2 || i + e + 4 <= a.D) {
          if (a.add) red_add4(row + i + e, v);
          else *reinterpret_cast<float4*>(row + i + e) = v;
        } else {
#pragma unroll
          for (int q = e; q < e + 4; q++) {
            if (i + q >= a.D) continue;
            if (a.add) red_add(row + i + q, x[q]);
            else row[i + q] = x[q];
          }
        }
      }
    }
  } else {
    if (a.add) {
      float old[n];
      Unit<T, kMode>::unpack(Unit<T, kMode>::load(row, i, lanes, a.D), old);
#pragma unroll
      for (int e = 0; e < n; e++) x[e] += old[e];
    }
    Unit<T, kMode>::store(row, i, lanes, a.D, x);
  }
}

constexpr int kGradBatch = 8;
constexpr int kGradChunk = 128;  // most choices per chunk

// Shared memory: what the CTA's choices say (class, row of dY, weight), read once.
template <typename T, typename TO, int kMode>
__global__ void __launch_bounds__(kEmbedThreads, 3) embed_sum_kernel(EmbedGradArgs a) {
  using U = Unit<T, kMode>;
  extern __shared__ uint32_t stage[];
  grid_dependency_wait();
  grid_dependents_launch();
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.beside = 0;
  uint32_t block = blockIdx.x - a.fill_first;
  if (block >= a.sum_blocks) {  // (the first ones wrap around)
    if (blockIdx.y != 0) return;
    block = blockIdx.x < a.fill_first ? blockIdx.x : blockIdx.x - a.sum_blocks;
    const int64_t k0 = a.fill_from + (int64_t)block * a.fill_rows;
    for (int q = threadIdx.x / 32; q < a.fill_rows && k0 + q < a.K; q += kEmbedThreads / 32)
      if (!a.seen[k0 + q])
        zero_bytes((char*)((TO*)a.dW + (k0 + q) * a.ldd), (uint64_t)a.D * sizeof(TO));
    return;
  }
  const int l = threadIdx.x & (a.lanes - 1);
  const uint32_t groups = kEmbedThreads / a.lanes, g = threadIdx.x / a.lanes;
  const uint32_t per = groups * a.chunk;  // of the CTA
  uint32_t* key = stage;
  uint32_t* row = stage + per;
  float* weight = reinterpret_cast<float*>(stage + 2 * per);
  const uint32_t first = block * per;
  for (uint32_t i = threadIdx.x; i < per; i += kEmbedThreads) {
    uint32_t k = (uint32_t)a.K, n = 0;
    float w = 0.f;
    if (first + i < a.M) {
      const Choice c = a.list[first + i];
      const uint32_t s = c.y;
      k = c.x;
      n = a.m == 1 ? s : (uint32_t)((s * a.by_m) >> 34);
      w = !a.resp ? 1.f : k < (uint32_t)a.K ? a.resp[s] : 0.f;
    }
    key[i] = k;
    row[i] = n;
    weight[i] = w;
  }
  const uint32_t c = block * groups + g, begin = c * a.chunk;
  const uint32_t none = 0xffffffffu;
  uint32_t before = none, after = none;
  if (c < a.chunks) {
    if (begin > 0) before = a.list[begin - 1].x;
    if (begin + a.chunk < a.M) after = a.list[begin + a.chunk].x;
  }
  __syncthreads();
  const int at = U::at(blockIdx.y * a.lanes, l, a.lanes);
  if (c >= a.chunks || at >= a.D) return;
  key += g * a.chunk;
  row += g * a.chunk;
  weight += g * a.chunk;
  bool came_in = before == key[0];
  float sum[U::n] = {};
  for (uint32_t i = 0; i < a.chunk; i += kGradBatch) {  // (a multiple of the batch)
    typename U::Raw r[kGradBatch];
#pragma unroll
    for (int b = 0; b < kGradBatch; b++)
      r[b] = key[i + b] < (uint32_t)a.K
                 ? U::load((const T*)a.dY + (int64_t)row[i + b] * a.ldy, at, a.lanes, a.D)
                 : U::zero();
#pragma unroll
    for (int b = 0; b < kGradBatch; b++) {
      const uint32_t k = key[i + b];
      if (k >= (uint32_t)a.K) return;  // the choices of no class are the last ones
      const float w = weight[i + b];
      float x[U::n];
      U::unpack(r[b], x);
#pragma unroll
      for (int e = 0; e < U::n; e++) sum[e] = fmaf(w, x[e], sum[e]);
      const bool last = i + b + 1 == a.chunk;
      const bool goes_on = (last ? after : key[i + b + 1]) == k;
      if (goes_on && !last) continue;
      if (came_in || goes_on) {
        float* p = a.part + ((int64_t)c * 2 + (came_in ? 0 : 1)) * a.width + at;
        if constexpr (U::kVec) {
#pragma unroll
          for (int e = 0; e < U::n; e += 4)
            *reinterpret_cast<float4*>(p + e) =
                make_float4(sum[e], sum[e + 1], sum[e + 2], sum[e + 3]);
        } else {
#pragma unroll
          for (int e = 0; e < U::n; e++)
            if (at + e * a.lanes < a.D) p[e * a.lanes] = sum[e];
        }
      } else {
        write_grad<T, TO, kMode>(a, k, at, a.lanes, sum);
      }
      came_in = false;
#pragma unroll
      for (int e = 0; e < U::n; e++) sum[e] = 0.f;
    }
  }
}

// The sums of runs that chunks' borders cut.  A warp looks at a chunk, for 32 units (blocks y):
// does a run begin in it and go on behind it?  It adds up a run of a few chunks by itself; longer
// ones are shared out over the CTA's threads.  (268,005 choices of 305 classes: 10 us, 24 before
// the long ones' loads were eight at a time.)
constexpr int kJoinShort = 8;  // chunks
constexpr int kJoinBatch = 8;  // chunks on their way at once

template <typename T, typename TO, int kMode>
__global__ void __launch_bounds__(kEmbedThreads) embed_join_kernel(EmbedGradArgs a) {
  using U = Unit<T, kMode>;
  constexpr int kWarps = kEmbedThreads / 32;
  __shared__ float sh[kEmbedThreads][U::n];
  __shared__ uint32_t long_chunk[kWarps], long_last[kWarps];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  grid_dependency_wait();
  grid_dependents_launch();
  const uint32_t c = blockIdx.x * kWarps + w;
  const uint64_t begin = (uint64_t)c * a.chunk, end = begin + a.chunk;
  int at = U::at(blockIdx.y * 32, lane, 32);
  auto part = [&](uint32_t q, bool tail, float (&x)[U::n]) {
    const float* p = a.part + ((int64_t)q * 2 + tail) * a.width + at;
    if constexpr (U::kVec) {
#pragma unroll
      for (int e = 0; e < U::n; e += 4) {
        const float4 v = *reinterpret_cast<const float4*>(p + e);
        x[e] = v.x, x[e + 1] = v.y, x[e + 2] = v.z, x[e + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < U::n; e++) x[e] = at + e * 32 < a.D ? p[e * 32] : 0.f;
    }
  };
  uint32_t k = (uint32_t)a.K, last = 0;
  bool mine = false;
  if (end < a.M) {
    k = a.list[end - 1].x;
    const uint32_t next = a.list[end].x, head = a.list[begin].x;
    const uint32_t before = begin > 0 ? a.list[begin - 1].x : 0xffffffffu;
    mine = k < (uint32_t)a.K && next == k && !(head == k && before == k);
  }
  if (mine) {
    // the run's last chunk: the first behind c whose own next entry is of another class
    uint32_t lo = c + 1, hi = a.chunks - 1;
    while (lo < hi) {
      const uint32_t step = (hi - lo + 31) / 32, probe = min(lo + step * lane, hi);
      const bool past = probe == hi || a.list[(uint64_t)(probe + 1) * a.chunk].x != k;
      const int f = __ffs(__ballot_sync(0xffffffffu, past)) - 1;
      const uint32_t found = f < 0 ? hi : min(lo + step * f, hi);
      const uint32_t from = f == 0 ? lo : f < 0 ? lo + step * 31 + 1 : lo + step * (f - 1) + 1;
      hi = found;
      lo = min(from, hi);
    }
    last = lo;
    if (last - c <= kJoinShort && at < a.D) {
      float sum[U::n], x[kJoinShort][U::n];
      part(c, true, sum);
#pragma unroll
      for (int q = 0; q < kJoinShort; q++)
        if (c + 1 + q <= last) part(c + 1 + q, false, x[q]);
#pragma unroll
      for (int q = 0; q < kJoinShort; q++) {
        if (c + 1 + q > last) continue;
#pragma unroll
        for (int e = 0; e < U::n; e++) sum[e] += x[q][e];
      }
      write_grad<T, TO, kMode>(a, k, at, 32, sum);
    }
  }
  const bool is_long = mine && last - c > kJoinShort;
  if (lane == 0) {
    long_chunk[w] = is_long ? c : 0xffffffffu;
    long_last[w] = last;
  }
  if (__syncthreads_or(is_long) == 0) return;
  // as many threads of a row as it has lanes; groups of those take every so many chunks
  const int first = blockIdx.y * 32 * U::n, rest = a.D - first;
  const int used = U::kVec ? (rest + U::n - 1) / U::n : rest;
  int lanes = 32;
  while (lanes / 2 >= used) lanes /= 2;
  const int ul = threadIdx.x & (lanes - 1), g = threadIdx.x / lanes, groups = kEmbedThreads / lanes;
  at = U::at(blockIdx.y * 32, ul, 32);
  for (int q = 0; q < kWarps; q++) {
    const uint32_t from = long_chunk[q], to = long_last[q];
    if (from == 0xffffffffu) continue;  // (the same for all threads)
    // (alike terms all round one way: 8 batches of chunks at most in float32)
    float sum[U::n] = {};
    double total[U::n] = {};
    if (at < a.D) {
      int batch = 0;
      for (uint32_t i0 = from + g; i0 <= to; i0 += kJoinBatch * groups) {
        float x[kJoinBatch][U::n];
#pragma unroll
        for (int b = 0; b < kJoinBatch; b++) {
          const uint32_t i = i0 + b * groups;
          if (i <= to) part(i, i == from, x[b]);
        }
#pragma unroll
        for (int b = 1; b < kJoinBatch; b++) {
          if (i0 + b * groups > to) continue;
#pragma unroll
          for (int e = 0; e < U::n; e++) x[0][e] += x[b][e];
        }
#pragma unroll
        for (int e = 0; e < U::n; e++) sum[e] += x[0][e];
        if (++batch % 8 == 0) {
#pragma unroll
          for (int e = 0; e < U::n; e++) {
            total[e] += (double)sum[e];
            sum[e] = 0.f;
          }
        }
      }
    }
#pragma unroll
    for (int e = 0; e < U::n; e++) sh[threadIdx.x][e] = sum[e] = (float)(total[e] + (double)sum[e]);
    for (int o = groups / 2; o > 0; o /= 2) {
      __syncthreads();
      if (g < o) {
#pragma unroll
        for (int e = 0; e < U::n; e++) {
          sum[e] += sh[threadIdx.x + o * lanes][e];
          sh[threadIdx.x][e] = sum[e];
        }
      }
    }
    if (g == 0 && at < a.D)
      write_grad<T, TO, kMode>(a, a.list[((uint64_t)from + 1) * a.chunk].x, at, 32, sum);
    __syncthreads();
  }
}

// ------------------------------------------------------------------ few choices
// Up to kFew choices go without a sort, in one launch: a group of lanes per choice looks through
// all of them (in shared memory), and where its choice is the first of its class adds up the
// class's rows, in order.  Blocks behind those: zeros for the classes that nothing names.  (Added
// to a table of 2,048: one token or 128 different ones take 2.7 to 2.9 us, 11 to 16 through the
// sort; 16 of one class 6.4, 128 of one class 33, as each batch waits for the one before.)
constexpr int kFew = 128;
constexpr int kFewRows = 4096;  // most rows of zeros per block

struct EmbedFewArgs {
  EmbedGradArgs g;
  const int32_t* idx;
  uint32_t* flags;
};

template <typename T, typename TO, int kMode>
__global__ void __launch_bounds__(kEmbedThreads, 2) embed_few_kernel(EmbedFewArgs f) {
  using U = Unit<T, kMode>;
  const EmbedGradArgs& a = f.g;
  __shared__ int32_t choice[kFew];
  __shared__ uint32_t match[kEmbedThreads / 8][kFew / 32];  // per group: where its class is named
  __shared__ uint8_t named[kFewRows];
  grid_dependency_wait();
  grid_dependents_launch();
  const int t = threadIdx.x, lane = t & 31, M = (int)a.M;
  for (int i = t; i < kFew; i += kEmbedThreads) {
    int k = i < M ? f.idx[i] : -1;
    if ((unsigned)k >= (unsigned)a.K) {
      if (k != -1 && f.flags) atomicOr(f.flags, GMM_DEVFLAG_BAD_INDEX);
      k = -1;
    }
    choice[i] = k;
  }
  if (blockIdx.x >= a.sum_blocks) {
    if (blockIdx.y != 0) return;
    const int64_t k0 = (int64_t)(blockIdx.x - a.sum_blocks) * a.fill_rows;
    for (int q = t; q < a.fill_rows; q += kEmbedThreads) named[q] = 0;
    __syncthreads();
    for (int i = t; i < M; i += kEmbedThreads) {
      const int64_t q = choice[i] - k0;
      if (choice[i] >= 0 && q >= 0 && q < a.fill_rows) named[q] = 1;
    }
    __syncthreads();
    for (int q = t / 32; q < a.fill_rows && k0 + q < a.K; q += kEmbedThreads / 32)
      if (!named[q]) zero_bytes((char*)((TO*)a.dW + (k0 + q) * a.ldd), (uint64_t)a.D * sizeof(TO));
    return;
  }
  __syncthreads();
  const int l = t & (a.lanes - 1), g = t / a.lanes, groups = kEmbedThreads / a.lanes;
  const int mine = blockIdx.x * groups + g;
  const int k = mine < M ? choice[mine] : -1;
  // every warp for its groups (several, or a part of one)
  for (int q = 0; q < 32; q += a.lanes < 32 ? a.lanes : 32) {
    const int kq = __shfl_sync(0xffffffffu, k, q);
    for (int w = 0; w < kFew / 32; w++) {
      const uint32_t found = __ballot_sync(0xffffffffu, kq >= 0 && choice[w * 32 + lane] == kq);
      if (lane == q) match[g][w] = found;
    }
  }
  __syncthreads();
  if (k < 0) return;
  for (int w = 0; w <= mine / 32; w++) {
    const uint32_t before = w < mine / 32 ? 0xffffffffu : (1u << (mine & 31)) - 1u;
    if (match[g][w] & before) return;  // an earlier choice has this class
  }
  const int at = U::at(blockIdx.y * a.lanes, l, a.lanes);
  if (at >= a.D) return;
  float sum[U::n] = {};
  int word = mine / 32;
  uint32_t bits = match[g][word];
  auto next = [&]() {
    while (bits == 0 && ++word < kFew / 32) bits = match[g][word];
    if (word >= kFew / 32) return -1;
    const int i = word * 32 + __ffs(bits) - 1;
    bits &= bits - 1;
    return i;
  };
  for (bool more = true; more;) {
    typename U::Raw r[kGradBatch];
    float w[kGradBatch];
#pragma unroll
    for (int b = 0; b < kGradBatch; b++) {
      const int i = more ? next() : -1;
      more = i >= 0;
      const int64_t n = i / a.m;
      r[b] = more ? U::load((const T*)a.dY + n * a.ldy, at, a.lanes, a.D) : U::zero();
      w[b] = !more ? 0.f : a.resp ? a.resp[i] : 1.f;
    }
#pragma unroll
    for (int b = 0; b < kGradBatch; b++) {
      float x[U::n];
      U::unpack(r[b], x);
#pragma unroll
      for (int e = 0; e < U::n; e++) sum[e] = fmaf(w[b], x[e], sum[e]);
    }
  }
  write_grad<T, TO, kMode>(a, (uint32_t)k, at, a.lanes, sum);
}

// ------------------------------------------------------------------ gradient of the weights
// A group of 8, 32 or (for few rows) all 256 lanes per row n: <dY_n, W[idx_nj]> for its m choices,
// in a fixed order.  (Like the rows of zeros it goes on beside the sort, and ends after it.)
// The instances for more than 4 choices spill 4 to 76 bytes per thread at the 64 registers that 4
// CTAs per SM leave, and sort_count_kernel 28 at 32.
struct EmbedDotArgs {
  const void *W, *dY;
  const int32_t* idx;
  float* dresp;
  int64_t N, ldw, ldy;
  int m, K, D, units;
  float scale;
  uint32_t* flags;
  Beside beside;
};

template <typename T, int kMode, int kLanes, int kMost>
__global__ void __launch_bounds__(kEmbedThreads, kBesideCtas) embed_dot_kernel(EmbedDotArgs a) {
  using U = Unit<T, kMode>;
  // units of a lane on their way at once
  constexpr int kAhead = kMost == 1 ? 4 : kMost == 2 ? 2 : 1;
  constexpr int kWarps = kLanes / 32;  // of a row, where it has more than one
  __shared__ float sh[kLanes > 32 ? kWarps : 1][kMost];
  grid_dependents_launch();
  beside_wait(a.beside);
  const int l = threadIdx.x % kLanes;
  const int64_t step = (int64_t)gridDim.x * (kEmbedThreads / kLanes);
  int64_t n = ((int64_t)blockIdx.x * kEmbedThreads + threadIdx.x) / kLanes;
  int next[kMost];  // the choices of the row after this one
  auto choices = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < kMost; j++) next[j] = row < a.N && j < a.m ? a.idx[row * a.m + j] : -1;
  };
  choices(n);
  // (whole warps go on, and the whole CTA, if it has one row)
  for (; __any_sync(0xffffffffu, n < a.N); n += step) {
    int k[kMost];
    float dot[kMost] = {};
#pragma unroll
    for (int j = 0; j < kMost; j++) {
      k[j] = next[j];
      if ((unsigned)k[j] >= (unsigned)a.K) {
        if (k[j] != -1 && a.flags) atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
        k[j] = -1;
      }
    }
    choices(n + step);
    if (n < a.N) {
      const T* dy = (const T*)a.dY + n * a.ldy;
      for (int u0 = 0; u0 < a.units; u0 += kAhead * kLanes) {
        typename U::Raw y[kAhead], r[kAhead][kMost];
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
          const int at = U::at(u0 + i * kLanes, l, kLanes);
          y[i] = at < a.D ? U::load(dy, at, kLanes, a.D) : U::zero();
#pragma unroll
          for (int j = 0; j < kMost; j++)
            r[i][j] = at < a.D && k[j] >= 0
                          ? U::load((const T*)a.W + k[j] * a.ldw, at, kLanes, a.D)
                          : U::zero();
        }
#pragma unroll
        for (int i = 0; i < kAhead; i++) {
          float yx[U::n];
          U::unpack(y[i], yx);
#pragma unroll
          for (int j = 0; j < kMost; j++) {
            float x[U::n];
            U::unpack(r[i][j], x);
#pragma unroll
            for (int e = 0; e < U::n; e++) dot[j] = fmaf(yx[e], x[e], dot[j]);
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kMost; j++) {
#pragma unroll
      for (int o = (kLanes < 32 ? kLanes : 32) / 2; o > 0; o >>= 1)
        dot[j] += __shfl_xor_sync(0xffffffffu, dot[j], o);
    }
    if constexpr (kLanes > 32) {
      if (l % 32 == 0) {
#pragma unroll
        for (int j = 0; j < kMost; j++) sh[l / 32][j] = dot[j];
      }
      __syncthreads();
      if (l == 0) {
#pragma unroll
        for (int j = 0; j < kMost; j++) {
#pragma unroll
          for (int w = 1; w < kWarps; w++) dot[j] += sh[w][j];
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kMost; j++)
      if (l == 0 && n < a.N && j < a.m) a.dresp[n * a.m + j] = k[j] < 0 ? 0.f : dot[j] * a.scale;
  }
  grid_dependency_wait();
}

}  // namespace scem
