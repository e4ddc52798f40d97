// rows.cuh -- log probabilities over rows of logits: kernels of gmm_logprobs,
// gmm_logprobs_backward and gmm_route.
//
// A row holds one logit x_k per class (a mixture component, a vocabulary entry,
// an expert) and z_k = fl32(scale * x_k).  Per row, with M = max_k z_k:
//   S = sum_k e^{z_k - M}      lse = M + log S       log p_k = (z_k - M) - log S
//   U = sum_k e^{z_k - M} (z_k - M)                  H = -sum_k p_k log p_k = log S - U / S
// and the m classes of largest z, equal z in ascending index order.
//
// S and U come from one pass: a thread (or a lane) keeps a reference R, its
// running maximum, and S and U relative to it; when R rises by a, S <- S e^{-a}
// and U <- e^{-a} (U - a S).  Partial results merge by the same rule, in a fixed
// order.  Everything is held in 32 bits.
//
// R starts at the lowest float rather than at -inf, and z - R is clamped from
// below at kFloorD, where e^{z-R} is exactly 0: classes masked by -inf, or by
// the type's lowest value, add 0 to both sums without a 0 * inf.  A row with no
// class left ends with S = 0.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <float.h>

#include "common.cuh"
#include "sm100_prims.cuh"

namespace scem {

constexpr int kMaxAlt = 32;          // most alternatives per row
constexpr float kFloorD = -150.f;    // e^-150 < 2^-149: 0 in float32
constexpr float kLog2e = 1.4426950408889634f;

struct RowArgs {
  const void* Z;
  int64_t N, ld;
  int K;
  float scale;
  const int32_t* ids;   // may be null
  int m;
  float* logp;          // with ids
  float* entropy;       // may be null
  float* lse;           // may be null
  int32_t* top_idx;     // m > 0
  float* top_val;       // log p, or responsibilities (route)
  int route;            // 0: log p; 1: responsibilities over all classes; 2: over the m chosen
  uint32_t* flags;      // may be null
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// 16 bytes of a row as floats.
template <typename T>
struct Vec16;
template <>
struct Vec16<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&x)[4]) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 neg_inf() {
    return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 neg_inf() {
    return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec16<__half> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 neg_inf() {
    return make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const __half2 v = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_f32(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(__half* p, float x) { *p = __float2half_rn(x); }

__device__ __forceinline__ uint4 load16(const void* p) {
  return *reinterpret_cast<const uint4*>(p);
}

// Reference, sum and first moment of a part of a row.
struct Part {
  float R, S, U;
};

__device__ __forceinline__ Part part_empty() { return {-FLT_MAX, 0.f, 0.f}; }

// Move p's reference to R >= p.R.
__device__ __forceinline__ void part_shift(Part& p, float R) {
  const float a = fmaxf(p.R - R, kFloorD);
  const float f = ex2(a * kLog2e);
  p.U = f * fmaf(a, p.S, p.U);
  p.S *= f;
  p.R = R;
}

__device__ __forceinline__ Part part_merge(Part p, Part q) {
  const float R = max_nan(p.R, q.R);
  part_shift(p, R);
  part_shift(q, R);
  return {R, p.S + q.S, p.U + q.U};
}

template <int kLanes>
__device__ __forceinline__ Part part_reduce(Part p) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    Part q;
    q.R = __shfl_xor_sync(0xffffffffu, p.R, o);
    q.S = __shfl_xor_sync(0xffffffffu, p.S, o);
    q.U = __shfl_xor_sync(0xffffffffu, p.U, o);
    p = part_merge(p, q);
  }
  return p;
}

// Key of an entry: larger keys are better, 0 is none.  Larger z first, then the
// lower index; z = -inf (masked) is none.
__device__ __forceinline__ uint64_t entry_key(float z, uint32_t idx) {
  if (z == -INFINITY) return 0;
  const uint32_t b = __float_as_uint(z + 0.f);  // -0 and +0 are equal
  const uint32_t o = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return ((uint64_t)o << 32) | (0xffffffffu - idx);
}
__device__ __forceinline__ uint32_t key_idx(uint64_t k) { return 0xffffffffu - (uint32_t)k; }
__device__ __forceinline__ float key_z(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo =
      __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return ((uint64_t)hi << 32) | lo;
}

// What a row's sums say, written by one thread.  bad: a NaN or +inf in the row.
template <typename T>
__device__ __forceinline__ void write_row(const RowArgs& a, int64_t n, const Part& p, float logS,
                                          bool bad) {
  const float nan = __int_as_float(0x7fffffff);
  const bool empty = p.S == 0.f;
  if (bad && a.flags) atomicOr(a.flags, GMM_DEVFLAG_NONFINITE_X);
  if (a.lse) a.lse[n] = bad ? nan : empty ? -INFINITY : p.R + logS;
  if (a.entropy) a.entropy[n] = bad ? nan : empty ? 0.f : fmaxf(logS - p.U / p.S, 0.f);
  if (a.ids) {
    const int id = a.ids[n];
    float lp;
    if (id == -1) {
      lp = 0.f;  // no label
    } else if (id < 0 || id >= a.K) {
      lp = nan;
      if (a.flags) atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
    } else {
      const float z = to_f32(((const T*)a.Z)[n * a.ld + id]) * a.scale;
      lp = bad ? nan : empty || z == -INFINITY ? -INFINITY : (z - p.R) - logS;
    }
    a.logp[n] = lp;
  }
}

// Alternative j of row n (key 0: none); sel: log-sum of the m chosen relative to p.R.
__device__ __forceinline__ void write_alt(const RowArgs& a, int64_t n, int j, uint64_t key,
                                          const Part& p, float logS, float sel, bool bad) {
  const float nan = __int_as_float(0x7fffffff);
  const bool none = bad || key == 0;
  a.top_idx[n * a.m + j] = none ? -1 : (int32_t)key_idx(key);
  const float d = key_z(key) - p.R;
  float v;
  if (a.route == 0)
    v = bad ? nan : none ? -INFINITY : d - logS;
  else
    v = bad ? nan : none ? 0.f : expf(d - (a.route == 2 ? sel : logS));
  a.top_val[n * a.m + j] = v;
}

// ------------------------------------------------------------------ short rows
// kLanes lanes hold a row of at most kLanes * kEl classes in registers, so a
// warp holds 32 / kLanes rows.  kVec: rows start on 16 bytes.
template <typename T, int kLanes, int kEl, bool kVec>
__global__ void __launch_bounds__(256) row_short_kernel(RowArgs a) {
  constexpr int kRows = 32 / kLanes;
  constexpr int V = kVec ? Vec16<T>::n : 1;
  constexpr int kChunks = kEl / V;
  static_assert(kEl % V == 0, "whole vectors");
  const int lane = threadIdx.x & 31, l = lane % kLanes;
  const int64_t warp = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * 8 * kRows;
  for (int64_t n0 = warp * kRows; n0 < a.N; n0 += step) {
    const int64_t n = n0 + lane / kLanes;
    const bool live = n < a.N;
    const T* row = (const T*)a.Z + (live ? n : n0) * a.ld;
    float z[kEl];
#pragma unroll
    for (int c = 0; c < kChunks; c++) {
      const int k0 = (c * kLanes + l) * V;
      if constexpr (kVec) {
        float x[V];
        if (k0 + V <= a.K) {
          Vec16<T>::unpack(load16(row + k0), x);
        } else {
#pragma unroll
          for (int e = 0; e < V; e++) x[e] = k0 + e < a.K ? to_f32(row[k0 + e]) : -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < V; e++) z[c * V + e] = x[e];
      } else {
        z[c] = k0 < a.K ? to_f32(row[k0]) : -INFINITY;
      }
    }
    Part p = part_empty();
#pragma unroll
    for (int i = 0; i < kEl; i++) {
      z[i] *= a.scale;
      p.R = max_nan(p.R, z[i]);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
      p.R = max_nan(p.R, __shfl_xor_sync(0xffffffffu, p.R, o));
#pragma unroll
    for (int i = 0; i < kEl; i++) {
      const float d = fmaxf(z[i] - p.R, kFloorD);
      const float e = ex2(d * kLog2e);
      p.S += e;
      p.U = fmaf(e, d, p.U);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      p.S += __shfl_xor_sync(0xffffffffu, p.S, o);
      p.U += __shfl_xor_sync(0xffffffffu, p.U, o);
    }
    const bool bad = !(p.R < INFINITY);
    const float logS = logf(p.S);
    if (l == 0 && live) write_row<T>(a, n, p, logS, bad);
    if (a.m > 0) {
      uint64_t mine = 0;  // lane l holds alternatives l, l + kLanes, ... one at a time
      float sel = 0.f;
      // renormalised weights need the chosen sum first: two sweeps over the winners
      // are avoided by keeping the keys (m <= 8 there, see the host's choice)
      uint64_t keep[8];
#pragma unroll
      for (int j = 0; j < 8; j++) keep[j] = 0;
      for (int j = 0; j < a.m; j++) {
        float bv = -INFINITY;
        int bi = -1;
#pragma unroll
        for (int i = 0; i < kEl; i++)
          if (z[i] > bv) {
            bv = z[i];
            bi = i;
          }
        uint64_t key = 0;
        if (bi >= 0) key = entry_key(bv, (uint32_t)((bi / V * kLanes + l) * V + bi % V));
        mine = key;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) {
          const uint64_t other = __shfl_xor_sync(0xffffffffu, key, o);
          key = other > key ? other : key;
        }
        if (mine == key) {
#pragma unroll
          for (int i = 0; i < kEl; i++)
            if (i == bi) z[i] = -INFINITY;
        }
        if (a.route == 2) {
          if (key) sel += expf(key_z(key) - p.R);
#pragma unroll
          for (int t = 0; t < 8; t++)
            if (t == j) keep[t] = key;
        } else if (l == 0 && live) {
          write_alt(a, n, j, key, p, logS, 0.f, bad);
        }
      }
      if (a.route == 2 && l == 0 && live) {
        sel = logf(sel);
#pragma unroll
        for (int j = 0; j < 8; j++)
          if (j < a.m) write_alt(a, n, j, keep[j], p, logS, sel, bad);
      }
    }
  }
}

// ------------------------------------------------------------------ long rows
// One cluster of gridDim-wide C CTAs per row, each CTA a contiguous slice of
// its 16-byte vectors; the row's unaligned ends go to the first and last CTA.
//
// Alternatives without a second pass over the row: let a thread's key be the
// best entry it saw.  An entry among the CTA's m best lies with one of the m
// threads of largest key (otherwise m threads hold a better entry each), so only
// those threads' entries are read again, by a warp each, and only entries not
// below the m-th of those keys are taken from them.  The lists are sorted, and
// merge by m rounds of a warp-wide maximum.
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kRowBatch = 4;  // 16-byte vectors in flight per thread

template <typename T>
struct RowSlice {
  static constexpr int V = Vec16<T>::n;
  const T* row;
  float scale;
  int head, tail0, tailn;  // entries before the first vector; first entry after the last; count
  int v0, v1;              // this CTA's vectors
  bool first, last;

  __device__ __forceinline__ RowSlice(const RowArgs& a, int64_t n, int rank, int C) {
    row = (const T*)a.Z + n * a.ld;
    scale = a.scale;
    const uint32_t off = (uint32_t)((uintptr_t)row & 15u);
    head = min(a.K, (int)(((16u - off) & 15u) / sizeof(T)));
    const int nv = (a.K - head) / V;
    tail0 = head + nv * V;
    tailn = a.K - tail0;
    v0 = (int)((int64_t)nv * rank / C);
    v1 = (int)((int64_t)nv * (rank + 1) / C);
    first = rank == 0;
    last = rank == C - 1;
  }
  __device__ __forceinline__ const T* vec(int v) const { return row + head + (int64_t)v * V; }
  __device__ __forceinline__ float z(int k) const { return to_f32(row[k]) * scale; }
  // best key of vector v below `below`
  __device__ __forceinline__ uint64_t best_of(int v, uint64_t below) const {
    float x[V];
    Vec16<T>::unpack(load16(vec(v)), x);
    uint64_t b = 0;
#pragma unroll
    for (int e = 0; e < V; e++) {
      const uint64_t k = entry_key(x[e] * scale, (uint32_t)(head + v * V + e));
      if (k < below && k > b) b = k;
    }
    return b;
  }
  // best key of thread t's entries below `below`, shared out over the warp's lanes
  __device__ __forceinline__ uint64_t best_of_thread(int t, int lane, uint64_t below) const {
    uint64_t b = 0;
    for (int v = v0 + t + lane * kRowThreads; v < v1; v += 32 * kRowThreads) {
      const uint64_t k = best_of(v, below);
      if (k > b) b = k;
    }
    if (lane == 0 && first && t < head) {
      const uint64_t k = entry_key(z(t), (uint32_t)t);
      if (k < below && k > b) b = k;
    }
    if (lane == 0 && last && t < tailn) {
      const uint64_t k = entry_key(z(tail0 + t), (uint32_t)(tail0 + t));
      if (k < below && k > b) b = k;
    }
    return warp_max_key(b);
  }
  // the thread that owns entry k of this slice
  __device__ __forceinline__ int owner(int k) const {
    if (k < head) return k;
    if (k >= tail0) return k - tail0;
    return ((k - head) / V - v0) % kRowThreads;
  }
};

struct RowShared {
  Part part[kRowWarps];
  Part total;
  uint64_t list[kRowWarps][kMaxAlt];
  uint64_t win[kMaxAlt];
  uint64_t cand[kMaxAlt][kMaxAlt];
  uint64_t out[kMaxAlt];
};

// Merge: lane's list is get(0), get(1), ... (descending, 0 when it ends); the m
// best of all lists, in order, are given to put(j, key) on every lane.
template <typename Get, typename Put>
__device__ __forceinline__ void merge_lists(int m, Get get, Put put) {
  int pos = 0;
  uint64_t head = get(0);
  for (int j = 0; j < m; j++) {
    const uint64_t best = warp_max_key(head);
    put(j, best);
    if (best != 0 && head == best) head = get(++pos);
  }
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) row_long_kernel(RowArgs a, int C) {
  constexpr int V = Vec16<T>::n;
  __shared__ RowShared sh;
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const int rank = C > 1 ? (int)sm100::cluster_ctarank() : 0;
  const int64_t clusters = gridDim.x / C;
  for (int64_t n = blockIdx.x / C; n < a.N; n += clusters) {
    const RowSlice<T> s(a, n, rank, C);
    Part p = part_empty();
    int where = -2;  // batch of the thread's first maximum: -1 head, nb tail
    const int nb = (s.v1 - s.v0 + kRowThreads * kRowBatch - 1) / (kRowThreads * kRowBatch);
    auto single = [&](int k, int b) {
      const float z = s.z(k);
      if (z > p.R || (where == -2 && z == p.R)) where = b;
      part_shift(p, max_nan(p.R, z));
      const float d = fmaxf(z - p.R, kFloorD);
      const float e = ex2(d * kLog2e);
      p.S += e;
      p.U = fmaf(e, d, p.U);
    };
    if (s.first && t < s.head) single(t, -1);
    for (int b = 0; b < nb; b++) {
      uint4 r[kRowBatch];
      const int base = s.v0 + b * kRowThreads * kRowBatch + t;
#pragma unroll
      for (int j = 0; j < kRowBatch; j++) {
        const int v = base + j * kRowThreads;
        r[j] = v < s.v1 ? load16(s.vec(v)) : Vec16<T>::neg_inf();
      }
      float x[kRowBatch][V];
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < kRowBatch; j++) {
        Vec16<T>::unpack(r[j], x[j]);
#pragma unroll
        for (int e = 0; e < V; e++) mx = max_nan(mx, x[j][e]);
      }
      const float zm = mx * s.scale;
      if (zm > p.R || (where == -2 && zm == p.R)) where = b;
      part_shift(p, max_nan(p.R, zm));
#pragma unroll
      for (int j = 0; j < kRowBatch; j++)
#pragma unroll
        for (int e = 0; e < V; e++) {
          const float d = fmaxf(fmaf(x[j][e], s.scale, -p.R), kFloorD);
          const float y = ex2(d * kLog2e);
          p.S += y;
          p.U = fmaf(y, d, p.U);
        }
    }
    if (s.last && t < s.tailn) single(s.tail0 + t, nb);

    const Part wp = part_reduce<32>(p);
    if (lane == 0) sh.part[w] = wp;
    if (a.m > 0) {
      // the thread's key: its first entry equal to its maximum
      uint64_t key = 0;
      if (where == -1) {
        key = entry_key(s.z(t), (uint32_t)t);
      } else if (where == nb) {
        key = entry_key(s.z(s.tail0 + t), (uint32_t)(s.tail0 + t));
      } else if (where >= 0) {
        const int base = s.v0 + where * kRowThreads * kRowBatch + t;
#pragma unroll
        for (int j = 0; j < kRowBatch; j++) {
          const int v = base + j * kRowThreads;
          if (v < s.v1) {
            const uint64_t k = s.best_of(v, ~0ull);
            if (k > key) key = k;
          }
        }
      }
      for (int j = 0; j < a.m; j++) {
        const uint64_t best = warp_max_key(key);
        if (lane == 0) sh.list[w][j] = best;
        if (key == best) key = 0;
      }
    }
    __syncthreads();
    if (w == 0) {
      Part q = lane < kRowWarps ? sh.part[lane] : part_empty();
      q = part_reduce<32>(q);
      if (lane == 0) sh.total = q;
      if (a.m > 0)
        merge_lists(
            a.m,
            [&](int i) { return lane < kRowWarps && i < a.m ? sh.list[lane][i] : 0ull; },
            [&](int j, uint64_t k) {
              if (lane == 0) sh.win[j] = k;
            });
    }
    __syncthreads();
    if (a.m > 0) {
      const uint64_t least = sh.win[a.m - 1];
      for (int j = w; j < a.m; j += kRowWarps) {
        uint64_t k = sh.win[j];
        const int owner = k ? s.owner((int)key_idx(k)) : 0;
        int c = 0;
        for (; c < a.m - j && k != 0 && k >= least; c++) {
          if (lane == 0) sh.cand[j][c] = k;
          k = s.best_of_thread(owner, lane, k);
        }
        if (lane == 0 && c < a.m) sh.cand[j][c] = 0;
      }
      __syncthreads();
      if (w == 0)
        merge_lists(
            a.m, [&](int i) { return lane < a.m && i < a.m - lane ? sh.cand[lane][i] : 0ull; },
            [&](int j, uint64_t k) {
              if (lane == 0) sh.out[j] = k;
            });
    }
    if (w == 0) {
      __syncwarp();
      const Part q = sh.total;
      const bool bad = !(q.R < INFINITY);
      const float logS = logf(q.S);
      if (lane == 0) write_row<T>(a, n, q, logS, bad);
      float sel = 0.f;
      if (a.route == 2) {
        for (int j = 0; j < a.m; j++)
          if (sh.out[j]) sel += expf(key_z(sh.out[j]) - q.R);
        sel = logf(sel);
      }
      if (lane < a.m) write_alt(a, n, lane, sh.out[lane], q, logS, sel, bad);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ gradient
// With a = dlogp at the label, t_j at the alternatives, l = dlse, h = dentropy:
//   dz_k = a [k = id] + sum_j t_j [k = top_j] + p_k (l - a - sum_j t_j - h (log p_k + H))
//   dx_k = scale dz_k
// One read and one write of the row; p from lse, so a row needs no reduction and
// its slices go to any CTA.  kGroup threads share a slice: a warp for short rows.
// Entries that a label or an alternative names are evaluated once more by the
// thread that holds the index, before the row is overwritten (dZ may be Z).
struct RowGradArgs {
  const void* Z;
  void* dZ;
  int64_t N, ld, ldd;
  int K;
  int slices;  // per row
  float scale;
  const int32_t* ids;
  const float *lse, *entropy, *dlogp, *dentropy, *dlse;
  int m;
  const int32_t* top_idx;
  const float* dtop;
  uint32_t* flags;
};

template <int kGroup>
__device__ __forceinline__ void group_sync() {
  if constexpr (kGroup == 32)
    __syncwarp();
  else
    __syncthreads();
}

template <typename T, int kGroup>
__global__ void __launch_bounds__(256) row_grad_kernel(RowGradArgs a) {
  constexpr int V = Vec16<T>::n;
  constexpr int kGroups = 256 / kGroup;
  constexpr int kOwn = (kMaxAlt + 1 + kGroup - 1) / kGroup;
  __shared__ int s_idx[kGroups][kMaxAlt + 1];
  __shared__ float s_coef[kGroups][kMaxAlt + 1];
  const int g = threadIdx.x / kGroup, t = threadIdx.x % kGroup;
  const int64_t items = a.N * a.slices;
  for (int64_t it = (int64_t)blockIdx.x * kGroups + g; it < items;
       it += (int64_t)gridDim.x * kGroups) {
    const int64_t n = it / a.slices;
    const int rank = (int)(it - n * a.slices);
    const T* row = (const T*)a.Z + n * a.ld;
    T* out = (T*)a.dZ + n * a.ldd;
    const uint32_t off = (uint32_t)((uintptr_t)row & 15u);
    const bool together = off == (uint32_t)((uintptr_t)out & 15u);  // else entry by entry
    const int head = together ? min(a.K, (int)(((16u - off) & 15u) / sizeof(T))) : a.K;
    const int nv = (a.K - head) / V;
    const int tail0 = head + nv * V;
    const int h0 = (int)((int64_t)head * rank / a.slices);
    const int h1 = (int)((int64_t)head * (rank + 1) / a.slices);
    const int v0 = (int)((int64_t)nv * rank / a.slices);
    const int v1 = (int)((int64_t)nv * (rank + 1) / a.slices);
    const bool last = rank == a.slices - 1;

    const float lse_in = a.lse[n];
    const bool empty = lse_in == -INFINITY;
    const float lse = empty ? INFINITY : lse_in;
    const int id = a.ids ? a.ids[n] : -1;
    const bool has_id = id >= 0 && id < a.K && !empty;
    const float la = has_id && a.dlogp ? a.dlogp[n] : 0.f;
    // the named entries: alternatives 0..m-1, then the label
    for (int j = t; j <= a.m; j += kGroup) {
      int k = -1;
      float c = 0.f;
      if (j == a.m) {
        if (has_id && a.dlogp) k = id, c = la;
        if (rank == 0 && a.flags && (id < -1 || id >= a.K))
          atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
      } else {
        const int v = a.top_idx[n * a.m + j];
        if (v >= 0 && v < a.K && !empty)
          k = v, c = a.dtop[n * a.m + j];
        else if (rank == 0 && a.flags && (v < -1 || v >= a.K))
          atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
      }
      s_idx[g][j] = k;
      s_coef[g][j] = c;
    }
    group_sync<kGroup>();
    float slope = a.dlse ? a.dlse[n] : 0.f;
    for (int j = 0; j <= a.m; j++) slope -= s_coef[g][j];
    const float h = a.dentropy ? a.dentropy[n] : 0.f;
    const float H = a.dentropy ? a.entropy[n] : 0.f;
    // dx = p (A + B log p) away from the named entries
    const bool bad = !(lse_in < INFINITY);
    const float A = empty ? 0.f
                    : bad ? __int_as_float(0x7fffffff)
                          : a.scale * (slope - h * H);
    const float B = empty || bad ? 0.f : -a.scale * h;
    auto grad = [&](float x) {
      const float lp = fmaxf(fmaf(x, a.scale, -lse), kFloorD);
      return ex2(lp * kLog2e) * fmaf(B, lp, A);
    };
    float named[kOwn];
    bool here[kOwn];  // the named entry lies in this slice
#pragma unroll
    for (int i = 0; i < kOwn; i++) {
      const int j = t + i * kGroup;
      const int k = j <= a.m ? s_idx[g][j] : -1;
      here[i] = k >= 0 && (k < head    ? k >= h0 && k < h1
                           : k < tail0 ? (k - head) / V >= v0 && (k - head) / V < v1
                                       : last);
      if (here[i]) {
        float c = 0.f;  // an entry may be named more than once
        for (int q = 0; q <= a.m; q++) c += s_idx[g][q] == k ? s_coef[g][q] : 0.f;
        named[i] = fmaf(a.scale, c, grad(to_f32(row[k])));
      }
    }
    group_sync<kGroup>();
    for (int k = h0 + t; k < h1; k += kGroup) from_f32(out + k, grad(to_f32(row[k])));
    const T* vin = row + head;
    T* vout = out + head;
    constexpr int kBatch = 4;
    for (int v = v0 + t; v < v1; v += kBatch * kGroup) {
      uint4 r[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; j++)
        if (v + j * kGroup < v1) r[j] = load16(vin + (int64_t)(v + j * kGroup) * V);
#pragma unroll
      for (int j = 0; j < kBatch; j++)
        if (v + j * kGroup < v1) {
          float x[V];
          Vec16<T>::unpack(r[j], x);
#pragma unroll
          for (int e = 0; e < V; e++) x[e] = grad(x[e]);
          *reinterpret_cast<uint4*>(vout + (int64_t)(v + j * kGroup) * V) = Vec16<T>::pack(x);
        }
    }
    if (last)
      for (int k = tail0 + t; k < a.K; k += kGroup) from_f32(out + k, grad(to_f32(row[k])));
    group_sync<kGroup>();
#pragma unroll
    for (int i = 0; i < kOwn; i++) {
      const int j = t + i * kGroup;
      if (here[i]) from_f32(out + s_idx[g][j], named[i]);
    }
    group_sync<kGroup>();
  }
}

}  // namespace scem
