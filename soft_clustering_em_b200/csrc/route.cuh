// route.cuh -- how a router loads its experts, and the router's gradient: kernels of
// gmm_route_loss and gmm_route_backward.
//
// p = softmax(scale x) over the K experts of a row.  Per segment of rows, over its L rows that
// count:
//   load_k = 1/L sum_n p_nk     counts_k = how often idx names k
//   balance = K sum_k (counts_k / (m L)) load_k        z = 1/L sum_n lse_n^2
// and for upstream gradients dbalance, dz (per segment) and dresp (of the weights that
// gmm_route gave, r = p of the chosen or q = p over the chosen's sum):
//   dx_k = scale [ p_k (g_k - sum_i p_i g_i + 2 dz/L lse - R) + sum_j [idx_j = k] a_j ],
//   g_k = dbalance K counts_k / (m L^2),
//   a_j = p_j dresp_j, R = sum_j a_j      or   a_j = q_j (dresp_j - sum_i q_i dresp_i), R = 0.
//
// A row sits in the registers of 8 to 32 lanes, as in row_short_kernel, and is read once.  Both are
// bound by memory for long rows, by the row's fixed part (reductions over its lanes, the chosen
// classes) for short ones.  Measured figures are of one B200, calls back to back, beside the time
// of the bytes alone at the rate of a large copy (6,548 GB/s).
#pragma once

#include "rows.cuh"

namespace scem {

constexpr int kRouteMostK = 1024;
constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / 32;
// CTAs per SM, for so many entries of a row per lane.
constexpr int route_ctas(int entries) { return entries <= 16 ? 3 : 2; }

struct RouteArgs {
  const void* Z;
  int64_t N, ld;
  int K;
  float scale;
  const int32_t* idx;      // N x m
  int m;
  const uint8_t* mask;     // N, may be null: 0 is a row that does not count
  const int32_t* offsets;  // S + 1, may be null: one segment
  int S;
  int64_t rows;            // of a CTA (loss) or of a warp (gradient)
  uint32_t* flags;         // may be null
};

// The segment of row r: the last one that begins at r or before (the first, if none does).  By a
// whole warp; any answer in [0, S) for offsets that do not ascend.
__device__ __forceinline__ int segment_of(const int32_t* offsets, int S, int64_t r) {
  if (!offsets) return 0;
  int lo = 0, n = S;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32, at = min((int)(threadIdx.x & 31) * step, n - 1);
    const uint32_t here = __ballot_sync(0xffffffffu, offsets[lo + at] <= r);
    const int f = here ? 31 - __clz(here) : 0;  // the last probe at r or before
    const int from = min(f * step, n - 1);
    lo += from;
    n = min(step, n - from);
  }
  return lo;
}

// What a piece of a segment (its rows in one CTA) leaves: K sums of p, K counts, the sum of
// lse^2 and the number of rows.
__host__ __device__ __forceinline__ int64_t route_slot(int K) { return 2 * (int64_t)K + 2; }

// How the classes of a row lie in the registers of kLanes lanes, in vectors of 16 bytes of T.
// kMode 1 and 2, rows that start on 16 bytes: as in memory, the row's last vector perhaps a part
// (1) or whole (2: K is a multiple).  kMode 0, rows that start anywhere: entry e of lane l is
// class e kLanes + l, so that the lanes' accesses lie together.
template <typename T, int kLanes, int kMode>
struct RouteMap {
  static constexpr int V = Vec16<T>::n;
  static __device__ __forceinline__ int class_of(int e, int l) {
    return kMode == 0 ? e * kLanes + l : (e / V * kLanes + l) * V + e % V;
  }
  // vector c of lane l, masked classes behind the row's end
  static __device__ __forceinline__ uint4 load(const T* row, int c, int l, int K) {
    const int k0 = (c * kLanes + l) * V;
    if constexpr (kMode == 2) {
      return k0 < K ? load16(row + k0) : Vec16<T>::neg_inf();
    } else if constexpr (kMode == 1) {
      return load_row_vec<T, true>(row, k0, K);
    } else {
      union {
        uint4 r;
        T x[V];
      } u;
      u.r = Vec16<T>::neg_inf();
#pragma unroll
      for (int e = 0; e < V; e++) {
        const int k = class_of(c * V + e, l);
        if (k < K) u.x[e] = row[k];
      }
      return u.r;
    }
  }
  static __device__ __forceinline__ void store(T* row, int c, int l, int K, const float (&x)[V]) {
    const int k0 = (c * kLanes + l) * V;
    if constexpr (kMode == 2) {
      if (k0 < K) *reinterpret_cast<uint4*>(row + k0) = Vec16<T>::pack(x);
    } else if (kMode == 1 && k0 + V <= K) {
      *reinterpret_cast<uint4*>(row + k0) = Vec16<T>::pack(x);
    } else {
#pragma unroll
      for (int e = 0; e < V; e++) {
        const int k = class_of(c * V + e, l);
        if (k < K) from_f32(row + k, x[e]);
      }
    }
  }
};

// The exponentials of a row relative to its largest logit.
template <int kLanes, int kEl, typename T>
struct RouteRow {
  static constexpr int V = Vec16<T>::n;
  static constexpr int kChunks = kEl / V;
  float y[kEl];   // e^{z - largest z}
  float S, xm;
  float ref;
  bool bad, empty;

  __device__ __forceinline__ void make(const uint4 (&r)[kChunks], float scale) {
    xm = max_nan(Vec16<T>::max_of(r), -INFINITY);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) xm = max_nan(xm, __shfl_xor_sync(0xffffffffu, xm, o));
    const float z = xm * scale;
    bad = !(z < INFINITY);
    empty = z == -INFINITY;
    ref = fmaxf(xm, -FLT_MAX);
    const F2 c2 = f2(scale * kLog2e, scale * kLog2e), ref2 = f2(-ref, -ref);
    F2 S2 = f2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < kChunks; v++) {
      float x[V];
      Vec16<T>::unpack(r[v], x);
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        float t0, t1;
        f2_get(f2_mul(f2_add(f2(x[e], x[e + 1]), ref2), c2), t0, t1);
        y[v * V + e] = ex2(t0);
        y[v * V + e + 1] = ex2(t1);
        S2 = f2_add(S2, f2(y[v * V + e], y[v * V + e + 1]));
      }
    }
    float s0, s1;
    f2_get(S2, s0, s1);
    S = s0 + s1;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
    // (a finite logit whose z overflows leaves finite exponentials: what comes of them is NaN too)
    S = fmaf(z, 0.f, S);
  }
  __device__ __forceinline__ float lse(float scale) const { return fmaf(xm, scale, logf(S)); }
};

template <int kLanes>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ------------------------------------------------------------------ load and losses
struct RouteLossOut {
  float *balance, *z, *load;
  int32_t *counts, *rows;
};

// The results of segment s, by one thread each: of an expert (its sum of p and its choices; returns
// its part of balance before scaling), and of the whole segment.
__device__ __forceinline__ double write_expert(const RouteArgs& a, const RouteLossOut& o, int s,
                                               int k, double p, uint32_t c, double L) {
  if (o.load) o.load[(int64_t)s * a.K + k] = (float)(p / L);
  if (o.counts) o.counts[(int64_t)s * a.K + k] = (int32_t)c;
  return (double)c * p;
}
__device__ __forceinline__ void write_segment(const RouteArgs& a, const RouteLossOut& o, int s,
                                              double balance, double z, uint32_t n, bool legal) {
  const float nan = __int_as_float(0x7fffffff);
  const double L = n > 0 ? (double)n : 1.0;
  if (o.balance) o.balance[s] = legal ? (float)(balance * a.K / (a.m * L * L)) : nan;
  if (o.z) o.z[s] = legal ? (float)(z / L) : nan;
  if (o.rows) o.rows[s] = (int32_t)n;
}

// 32 bits of CTA r's shared memory, at the place of `here` in this one's.
__device__ __forceinline__ uint32_t ld_cluster(const void* here, int r) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];"
               : "=r"(v)
               : "r"(sm100::map_to_rank(sm100::smem_u32(here), r))
               : "memory");
  return v;
}

// A CTA takes `rows` rows.  For each segment that they meet, in order, column sums stay in
// registers until the segment or the rows end; the sums of piece (CTA c, segment s) go to slot
// c + s, which no other piece has: from piece to piece c or s grows, or both.
//
// 65,536 rows of 256 fp32, the joining kernel with it: 22 us (10.6 us of bytes), 16.5 of them this
// kernel's, at 3.6 TB/s: few rows per warp, so that the first loads and the joining of the columns
// weigh.  262,144 rows: 54 us (41).  65,536 of 1,024: 71 us (41).
//
// kDirect, for few rows: a cluster of up to 8 CTAs takes a segment, and its first CTA adds up what
// the others left in their shared memory and writes the results, in one launch.  (50 rows in 64
// segments: 3.5 us, 13 with the joining kernel; 512 rows of 64: 4.7 and 7.0.)
template <typename T, int kLanes, int kEl, int kMode, bool kDirect>
__global__ void __launch_bounds__(kRouteThreads, route_ctas(kEl))
    route_load_kernel(RouteArgs a, float* part, RouteLossOut o) {
  constexpr int kRows = 32 / kLanes;
  constexpr int V = Vec16<T>::n;
  constexpr int kChunks = kEl / V;
  constexpr int kPlaces = kLanes * kEl;
  __shared__ float sums[kRouteWarps][kPlaces];
  __shared__ uint32_t hist[kPlaces];
  __shared__ float zsum[kRouteWarps];
  __shared__ uint32_t rsum[kRouteWarps];
  __shared__ double bsum[kRouteWarps];  // with kDirect, and the CTA's z and rows
  __shared__ float z_here;
  __shared__ uint32_t rows_here;
  const int t = threadIdx.x, lane = t & 31, w = t >> 5, l = lane % kLanes;
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t r0 = kDirect ? 0 : blockIdx.x * a.rows;
  const int64_t r1 = kDirect ? a.N : min(r0 + a.rows, a.N);
  const int rank = kDirect ? (int)sm100::cluster_ctarank() : 0;
  const int ctas = kDirect ? (int)sm100::cluster_nctarank() : 1;
  int s = kDirect ? (int)blockIdx.x / ctas : segment_of(a.offsets, a.S, r0);
  const int s_end = kDirect ? s + 1 : a.S;
  for (int i = t; i < a.K; i += kRouteThreads) hist[i] = 0;
  __syncthreads();
  for (; s < s_end; s++) {
    int64_t lo = r0, hi = r1;
    bool legal = true;
    if (a.offsets) {
      const int64_t from = a.offsets[s], to = a.offsets[s + 1];
      legal = from >= 0 && from <= to && to <= a.N;
      lo = max(r0, from);
      hi = min(r1, to);
      if (!kDirect && from >= r1) break;
    }
    if (!kDirect && lo >= hi) continue;  // (the same for all threads)
    if (kDirect && !legal) {
      hi = lo = 0;
      if (t == 0 && a.flags) atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
    }
    if (kDirect) {  // the CTA's share: whole turns of its warps
      constexpr int kTurn = kRouteWarps * kRows;
      const int64_t per = ((hi - lo + ctas - 1) / ctas + kTurn - 1) / kTurn * kTurn;
      lo = min(lo + rank * per, hi);
      hi = min(lo + per, hi);
    }
    float acc[kEl] = {};
    float zs = 0.f;
    uint32_t live_rows = 0;
    uint4 next[kChunks];  // the rows after these are on their way
    int next_k = -1;
    bool next_out = false;
    auto fetch = [&](int64_t n0) {
      const int64_t n = n0 + lane / kLanes;
      const bool in = n < hi;
      const T* row = (const T*)a.Z + (in ? n : n0) * a.ld;
#pragma unroll
      for (int c = 0; c < kChunks; c++)
        next[c] = RouteMap<T, kLanes, kMode>::load(row, c, l, a.K);
      next_k = in && l < a.m ? a.idx[n * a.m + l] : -1;
      next_out = !in || (a.mask && !a.mask[n]);
    };
    if (lo + w * kRows < hi) fetch(lo + w * kRows);
    for (int64_t n0 = lo + w * kRows; n0 < hi; n0 += kRouteWarps * kRows) {
      uint4 r[kChunks];
#pragma unroll
      for (int c = 0; c < kChunks; c++)  // (a row that is out: as if all its classes were masked)
        r[c] = next_out ? Vec16<T>::neg_inf() : next[c];
      const int k = next_k;
      if (n0 + kRouteWarps * kRows < hi) fetch(n0 + kRouteWarps * kRows);
      RouteRow<kLanes, kEl, T> q;
      q.make(r, a.scale);
      const float inv = q.empty ? 0.f : 1.f / q.S;
      const F2 inv2 = f2(inv, inv);
#pragma unroll
      for (int e = 0; e < kEl; e += 2)
        f2_get(f2_fma(f2(q.y[e], q.y[e + 1]), inv2, f2(acc[e], acc[e + 1])), acc[e], acc[e + 1]);
      if (!q.empty) {
        if (l == 0) {
          const float z = q.lse(a.scale);
          zs = fmaf(z, z, zs);
          live_rows++;
          if (q.bad && a.flags) atomicOr(a.flags, GMM_DEVFLAG_NONFINITE_X);
        }
        if ((unsigned)k < (unsigned)a.K) atomicAdd(&hist[k], 1u);
        else if (k != -1 && a.flags) atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
      }
    }
#pragma unroll
    for (int e = 0; e < kEl; e++) {
#pragma unroll
      for (int o = kLanes; o < 32; o <<= 1) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
    }
    zs = warp_sum(zs);
    live_rows = __reduce_add_sync(0xffffffffu, live_rows);
    if (lane < kLanes) {
#pragma unroll
      for (int e = 0; e < kEl; e++)
        sums[w][RouteMap<T, kLanes, kMode>::class_of(e, l)] = acc[e];
    }
    if (lane == 0) zsum[w] = zs, rsum[w] = live_rows;
    __syncthreads();
    float z = 0.f;
    uint32_t rows = 0;
    for (int i = 0; i < kRouteWarps; i++) z += zsum[i], rows += rsum[i];
    float* slot = kDirect ? sums[0] : part + (blockIdx.x + (int64_t)s) * route_slot(a.K);
    for (int k = t; k < a.K; k += kRouteThreads) {
      float p = 0.f;
#pragma unroll
      for (int i = 0; i < kRouteWarps; i++) p += sums[i][k];
      slot[k] = p;
      if constexpr (!kDirect) {
        reinterpret_cast<uint32_t*>(slot)[a.K + k] = hist[k];
        hist[k] = 0;
      }
    }
    if constexpr (kDirect) {
      if (t == 0) z_here = z, rows_here = rows;
      __syncwarp();
      if (ctas > 1) sm100::cluster_sync();
      else __syncthreads();
      if (rank == 0) {
        double z_all = z, balance = 0.0;
        for (int r = 1; r < ctas; r++) {
          z_all += __uint_as_float(ld_cluster(&z_here, r));
          rows += ld_cluster(&rows_here, r);
        }
        const double L = rows > 0 ? (double)rows : 1.0;
        for (int k = t; k < a.K; k += kRouteThreads) {
          double p = sums[0][k];
          uint32_t c = hist[k];
#pragma unroll 7
          for (int r = 1; r < ctas; r++) {
            p += __uint_as_float(ld_cluster(&sums[0][k], r));
            c += ld_cluster(&hist[k], r);
          }
          balance += write_expert(a, o, s, k, p, c, L);
        }
        balance = warp_sum(balance);
        if (lane == 0) bsum[w] = balance;
        __syncthreads();
        if (t == 0) {
          balance = 0.0;
          for (int i = 0; i < kRouteWarps; i++) balance += bsum[i];
          write_segment(a, o, s, balance, z_all, rows, legal);
        }
      }
      __syncwarp();
      if (ctas > 1) sm100::cluster_sync();  // (shared memory is there until it has been read)
    } else {
      if (t == 0) {
        slot[2 * a.K] = z;
        reinterpret_cast<uint32_t*>(slot)[2 * a.K + 1] = rows;
      }
      __syncthreads();
    }
  }
}

// A cluster per segment adds up its slots, in order, in 64 bits; each CTA has a share of the
// experts.  Threads: `cols` columns (a power of two) times groups that take every so many slots.
constexpr int kReduceCtas = 8;  // most
template <int kReduceThreads>
__global__ void __launch_bounds__(kReduceThreads)
    route_reduce_kernel(RouteArgs a, const float* part, RouteLossOut o, int cols) {
  constexpr int kReduceWarps = kReduceThreads / 32;
  __shared__ double sh[kReduceThreads];
  __shared__ uint32_t shc[kReduceThreads];
  __shared__ double zs[kReduceWarps], bs[kReduceWarps];
  __shared__ uint32_t rs[kReduceWarps];
  __shared__ double of_cta[kReduceCtas];  // balance of each CTA's experts, in the first CTA
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const int rank = (int)sm100::cluster_ctarank(), ctas = (int)sm100::cluster_nctarank();
  const int s = blockIdx.x / ctas;
  const int groups = kReduceThreads / cols, g = t / cols, col = t & (cols - 1);
  // (the others of the cluster have started when its first CTA's memory is written below)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t lo = a.offsets ? a.offsets[s] : 0, hi = a.offsets ? a.offsets[s + 1] : a.N;
  const bool legal = lo >= 0 && lo <= hi && hi <= a.N;
  if (!legal && t == 0 && a.flags) atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
  const int64_t size = route_slot(a.K);
  const int64_t first = legal && hi > lo ? lo / a.rows + s : 0;
  const int count = legal && hi > lo ? (int)((hi - 1) / a.rows - lo / a.rows) + 1 : 0;
  part += first * size;
  double z = 0.0;
  uint32_t n = 0;
  for (int q = t; q < count; q += kReduceThreads) {
    z += part[q * size + 2 * a.K];
    n += reinterpret_cast<const uint32_t*>(part)[q * size + 2 * a.K + 1];
  }
  double balance = 0.0, L = 1.0;
  for (int k0 = rank * cols; k0 < a.K || k0 == rank * cols; k0 += ctas * cols) {
    const int k = k0 + col;
    double p = 0.0;
    uint32_t c = 0;
    if (k < a.K) {
#pragma unroll 8
      for (int q = g; q < count; q += groups) {
        p += part[q * size + k];
        c += reinterpret_cast<const uint32_t*>(part)[q * size + a.K + k];
      }
    }
    sh[t] = p;
    shc[t] = c;
    if (k0 == rank * cols) {
      z = warp_sum(z);
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) zs[w] = z, rs[w] = n;
    }
    __syncthreads();
    if (k0 == rank * cols) {
      z = 0.0;
      n = 0;
      for (int i = 0; i < kReduceWarps; i++) z += zs[i], n += rs[i];
      L = n > 0 ? (double)n : 1.0;
    }
    if (g == 0 && k < a.K) {
      for (int i = 1; i < groups; i++) p += sh[i * cols + col], c += shc[i * cols + col];
      balance += write_expert(a, o, s, k, p, c, L);
    }
    __syncthreads();
  }
  balance = warp_sum(balance);
  if (lane == 0) bs[w] = balance;
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (t == 0) {
    balance = 0.0;
    for (int i = 0; i < kReduceWarps; i++) balance += bs[i];
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(
                     sm100::map_to_rank(sm100::smem_u32(of_cta + rank), 0)),
                 "d"(balance)
                 : "memory");
  }
  __syncwarp();
  sm100::cluster_sync();
  if (rank == 0 && t == 0) {
    balance = 0.0;
    for (int r = 0; r < ctas; r++) balance += of_cta[r];
    write_segment(a, o, s, balance, z, n, legal);
  }
}

// ------------------------------------------------------------------ gradient
struct RouteGradArgs {
  RouteArgs r;
  const float* dresp;       // N x m, may be null
  int renorm;
  const int32_t *counts, *live;  // S x K and S; null without dbalance and dz
  const float *dbalance, *dz;    // S each, may be null
  void* dZ;
  int64_t ldd;
  float least;                   // the least x that scale does not take to -inf (a masked class)
};

// A warp takes `rows` consecutive rows, 32 / kLanes at a time; the counts of the segment stay in
// registers while it lasts.  The chosen classes' entries are written once more by the lanes that
// hold the choices: finding them in the registers of the lane that holds the class cost 32
// compares for each (58 us, now 31, for the first of these).
//
// 65,536 rows of 256 fp32 with 8 choices: 31 to 35 us (21 us of bytes).  262,144: 111 us (83), 94
// without the choices' entries.  65,536 of 1,024: 97 us (83).  Of 201 bf16, rows that start
// anywhere: 35 us (9); of 200: 22.
// The fp32 instances from 65 classes on spill 8 to 72 bytes per thread, at 80 registers (up to 128
// classes, three CTAs per SM) or 128 (two).
template <typename T, int kLanes, int kEl, int kMode>
__global__ void __launch_bounds__(kRouteThreads, route_ctas(kEl))
    route_grad_kernel(RouteGradArgs g) {
  constexpr int kRows = 32 / kLanes;
  constexpr int V = Vec16<T>::n;
  constexpr int kChunks = kEl / V;
  const RouteArgs& a = g.r;
  const int lane = threadIdx.x & 31, l = lane % kLanes;
  const int64_t warp = (int64_t)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  const int64_t r0 = warp * a.rows, r1 = min(r0 + a.rows, a.N);
  grid_dependency_wait();
  grid_dependents_launch();
  if (r0 >= r1) return;
  const bool losses = g.dbalance || g.dz;
  int s = losses ? segment_of(a.offsets, a.S, r0) : 0, have = -1;
  float cnt[kEl];
  float coef = 0.f, pull = 0.f;
#pragma unroll
  for (int e = 0; e < kEl; e++) cnt[e] = 0.f;
  uint4 next[kChunks];  // the rows after these are on their way
  int next_k = -1;
  float next_d = 0.f;
  bool next_out = false;
  auto fetch = [&](int64_t n0) {
    const int64_t n = n0 + lane / kLanes;
    const bool in = n < r1;
    const T* row = (const T*)a.Z + (in ? n : n0) * a.ld;
#pragma unroll
    for (int c = 0; c < kChunks; c++)
      next[c] = RouteMap<T, kLanes, kMode>::load(row, c, l, a.K);
    next_k = -1;
    if (g.dresp && in && l < a.m) {
      next_k = a.idx[n * a.m + l];
      next_d = g.dresp[n * a.m + l];
    }
    next_out = a.mask && in && !a.mask[n];
  };
  fetch(r0);
  for (int64_t n0 = r0; n0 < r1; n0 += kRows) {
    const int64_t n = n0 + lane / kLanes;
    const bool in = n < r1;
    const T* row = (const T*)a.Z + (in ? n : n0) * a.ld;
    uint4 r[kChunks];
#pragma unroll
    for (int c = 0; c < kChunks; c++) r[c] = next[c];
    const int k = next_k;
    const float d = next_d;
    bool counts = losses && in && !next_out;
    const bool legal = (unsigned)k < (unsigned)a.K;
    if (!legal && k != -1 && a.flags) atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
    const float xk = legal ? to_f32(row[k]) : -INFINITY;
    if (n0 + kRows < r1) fetch(n0 + kRows);
    if (counts && a.offsets) {
      while (s + 1 < a.S && n >= a.offsets[s + 1]) s++;
      counts = n >= a.offsets[s] && n < a.offsets[s + 1];
    }
    if (counts && s != have) {
      have = s;
      const float L = (float)max(g.live[s], 1);
      coef = g.dbalance ? g.dbalance[s] * (float)a.K / ((float)a.m * L * L) : 0.f;
      pull = g.dz ? 2.f * g.dz[s] / L : 0.f;
      if (g.dbalance) {
        const int32_t* of = g.counts + (int64_t)s * a.K;
#pragma unroll
        for (int e = 0; e < kEl; e++) {
          const int ke = RouteMap<T, kLanes, kMode>::class_of(e, l);
          cnt[e] = ke < a.K ? (float)of[ke] : 0.f;
        }
      }
    }
    RouteRow<kLanes, kEl, T> q;
    q.make(r, a.scale);
    const float c = a.scale * kLog2e, inv = 1.f / q.S;
    // the chosen: their weights and what they pull on
    const float top = a.m > 0 && g.renorm ? fmaxf(group_max<kLanes>(xk), g.least) : q.ref;
    const float ek = legal ? ex2((xk - top) * c) : 0.f;
    const float over = g.renorm ? group_sum<kLanes>(ek) : q.S;
    const float wk = ek > 0.f || !(ek == ek) ? ek / over : 0.f;
    const float wd = legal ? wk * d : 0.f;
    const float R = group_sum<kLanes>(wd);
    const float add = g.renorm ? fmaf(-wk, R, wd) : wd;
    F2 dot2 = f2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < kEl; e += 2)
      dot2 = f2_fma(f2(q.y[e], q.y[e + 1]), f2(cnt[e], cnt[e + 1]), dot2);
    float dot, dot1;
    f2_get(dot2, dot, dot1);
    dot = group_sum<kLanes>(dot + dot1) * inv;
    const float cf = counts ? coef : 0.f;
    const float base = (counts ? pull * q.lse(a.scale) - coef * dot : 0.f) - (g.renorm ? 0.f : R);
    const bool chosen = __ballot_sync(0xffffffffu, legal) >> (lane - l) & group_mask<kLanes>();
    const bool live = !q.empty && (counts || chosen);
    if (q.bad && live && l == 0 && a.flags) atomicOr(a.flags, GMM_DEVFLAG_NONFINITE_X);
    // (a row with a NaN or a z of +inf is NaN throughout: so is S)
    const F2 to2 = f2(inv * a.scale, inv * a.scale), cf2 = f2(cf, cf), base2 = f2(base, base);
#pragma unroll
    for (int e = 0; e < kEl; e += 2)
      f2_get(f2_mul(f2_mul(f2(q.y[e], q.y[e + 1]), to2),
                    f2_fma(cf2, f2(cnt[e], cnt[e + 1]), base2)),
             q.y[e], q.y[e + 1]);
    if (!live) {
#pragma unroll
      for (int e = 0; e < kEl; e++) q.y[e] = 0.f;
    }
    // what a chosen class gets beside that, from every choice that names it
    float more = add;
    const uint32_t same = __match_any_sync(
        0xffffffffu, legal ? (lane - l) << 16 | k : -1 - lane);  // (K is below 2^16)
    if (__any_sync(0xffffffffu, (same & (same - 1u)) != 0u)) {  // a class named twice
      more = 0.f;
      for (int j = 0; j < a.m; j++) {
        const int kj = __shfl_sync(0xffffffffu, k, (lane - l) + j);
        const float aj = __shfl_sync(0xffffffffu, add, (lane - l) + j);
        if (kj == k) more += aj;
      }
    }
    __syncwarp();
    T* out = (T*)g.dZ + (in ? n : n0) * g.ldd;
#pragma unroll
    for (int v = 0; v < kChunks; v++) {
      float x[V];
#pragma unroll
      for (int e = 0; e < V; e++) x[e] = q.y[v * V + e];
      if (in) RouteMap<T, kLanes, kMode>::store(out, v, l, a.K, x);
    }
    __syncwarp();
    // the chosen classes' entries once more, by the lanes that hold the choices
    if (legal && live) {
      const float ck = counts && g.dbalance ? (float)g.counts[(int64_t)s * a.K + k] : 0.f;
      const float pk = ex2((xk - q.ref) * c) * inv;
      from_f32(out + k, fmaf(pk, fmaf(cf, ck, base), more) * a.scale);
    }
  }
}

}  // namespace scem
