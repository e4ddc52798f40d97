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

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float y;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Two floats in a register pair: one instruction for both.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_get(F2 p, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p.v));
}
__device__ __forceinline__ F2 f2_add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 f2_fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
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
  // the largest of kN vectors' entries, a NaN if there is one
  template <int kN>
  static __device__ __forceinline__ float max_of(const uint4 (&r)[kN]) {
    float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < kN; j++) {
      m[0] = max3_nan(m[0], __uint_as_float(r[j].x), __uint_as_float(r[j].y));
      m[1] = max3_nan(m[1], __uint_as_float(r[j].z), __uint_as_float(r[j].w));
    }
    return max_nan(m[0], m[1]);
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
  template <int kN>
  static __device__ __forceinline__ float max_of(const uint4 (&r)[kN]) {
    uint32_t m = 0xff80ff80u;
#pragma unroll
    for (int j = 0; j < kN; j++) {
      const uint32_t w[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
      for (int i = 0; i < 4; i++)
        asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
    }
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
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
  template <int kN>
  static __device__ __forceinline__ float max_of(const uint4 (&r)[kN]) {
    uint32_t m = 0xfc00fc00u;
#pragma unroll
    for (int j = 0; j < kN; j++) {
      const uint32_t w[4] = {r[j].x, r[j].y, r[j].z, r[j].w};
#pragma unroll
      for (int i = 0; i < 4; i++)
        asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
    }
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
    return max_nan(f.x, f.y);
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
// warp holds 32 / kLanes rows; lane l takes vectors l, l + kLanes, ... of 16
// bytes.  kVec: rows start on 16 bytes (else the same entries one by one).
//
// Alternatives in m rounds.  Only each vector's largest entry stays in registers;
// a round finds the lowest vector that holds the row's largest, reads it again
// (it is in L1) and leaves it with its largest entry behind the one just taken.
template <typename T, bool kVec>
__device__ __forceinline__ uint4 load_row_vec(const T* row, int k0, int K) {
  constexpr int V = Vec16<T>::n;
  if (kVec && k0 + V <= K) return load16(row + k0);
  union {
    uint4 r;
    T x[V];
  } u;
  u.r = Vec16<T>::neg_inf();
#pragma unroll
  for (int e = 0; e < V; e++)
    if (k0 + e < K) u.x[e] = row[k0 + e];
  return u.r;
}

template <typename T, int kLanes, int kEl, bool kVec>
__global__ void __launch_bounds__(256, kEl <= 16 ? 6 : 4) row_short_kernel(RowArgs a) {
  constexpr int kRows = 32 / kLanes;
  constexpr int V = Vec16<T>::n;
  constexpr int kChunks = kEl / V;
  static_assert(kEl % V == 0 && kLanes >= 8, "whole vectors; a lane for each chosen expert");
  const int lane = threadIdx.x & 31, l = lane % kLanes;
  const int64_t warp = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t step = (int64_t)gridDim.x * 8 * kRows;
  for (int64_t n0 = warp * kRows; n0 < a.N; n0 += step) {
    const int64_t n = n0 + lane / kLanes;
    const bool live = n < a.N;
    const T* row = (const T*)a.Z + (live ? n : n0) * a.ld;
    uint4 r[kChunks];
    float top[kChunks];  // the largest z of each vector
#pragma unroll
    for (int c = 0; c < kChunks; c++)
      r[c] = load_row_vec<T, kVec>(row, (c * kLanes + l) * V, a.K);
    float R = -FLT_MAX;
#pragma unroll
    for (int c = 0; c < kChunks; c++) {
      const uint4 one[1] = {r[c]};
      top[c] = Vec16<T>::max_of(one) * a.scale;
      R = max_nan(R, top[c]);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) R = max_nan(R, __shfl_xor_sync(0xffffffffu, R, o));
    F2 S2 = f2(0.f, 0.f), U2 = S2;
    const F2 scale2 = f2(a.scale, a.scale), ref2 = f2(-R, -R), log2 = f2(kLog2e, kLog2e);
#pragma unroll
    for (int c = 0; c < kChunks; c++) {
      float x[V];
      Vec16<T>::unpack(r[c], x);
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        float d0, d1, t0, t1;
        f2_get(f2_fma(f2(x[e], x[e + 1]), scale2, ref2), d0, d1);
        const F2 d = f2(fmaxf(d0, kFloorD), fmaxf(d1, kFloorD));
        f2_get(f2_mul(d, log2), t0, t1);
        const F2 y = f2(ex2(t0), ex2(t1));
        S2 = f2_add(S2, y);
        U2 = f2_fma(y, d, U2);
      }
    }
    Part p;
    float s0, s1;
    p.R = R;
    f2_get(S2, s0, s1);
    p.S = s0 + s1;
    f2_get(U2, s0, s1);
    p.U = s0 + s1;
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      p.S += __shfl_xor_sync(0xffffffffu, p.S, o);
      p.U += __shfl_xor_sync(0xffffffffu, p.U, o);
    }
    const bool bad = !(p.R < INFINITY);
    const float logS = logf(p.S);
    if (l == 0 && live) write_row<T>(a, n, p, logS, bad);
    float sel = 0.f;
    float last_z = INFINITY;  // the entry taken last: what follows it in the order is left
    int last_k = -1;
    for (int j0 = 0; j0 < a.m; j0 += kLanes) {
      const int cnt = min(kLanes, a.m - j0);
      uint64_t mine = 0;  // lane l keeps alternative j0 + l
      for (int j = 0; j < cnt; j++) {
        float best = top[0];
#pragma unroll
        for (int c = 1; c < kChunks; c++) best = fmaxf(best, top[c]);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
          best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
        int at = 1 << 30;  // the lowest vector that holds it
#pragma unroll
        for (int c = kChunks - 1; c >= 0; c--)
          if (top[c] == best) at = c * kLanes + l;
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1)
          at = min(at, __shfl_xor_sync(0xffffffffu, at, o));
        const bool none = best == -INFINITY || at == 1 << 30;
        const int k0 = none ? 0 : at * V;
        float x[V];
        Vec16<T>::unpack(load_row_vec<T, kVec>(row, k0, a.K), x);
        int e0 = 0;
#pragma unroll
        for (int e = V - 1; e >= 0; e--) {
          x[e] *= a.scale;
          if (x[e] == best && (best < last_z || k0 + e > last_k)) e0 = e;
        }
        float next = -INFINITY;
#pragma unroll
        for (int e = 0; e < V; e++)
          if (x[e] < best || (x[e] == best && e > e0)) next = fmaxf(next, x[e]);
#pragma unroll
        for (int c = 0; c < kChunks; c++)
          if (at == c * kLanes + l) top[c] = next;
        last_z = best;
        last_k = k0 + e0;
        if (!none) {
          sel += ex2((best - p.R) * kLog2e);
          if (l == j) mine = entry_key(best, (uint32_t)last_k);
        }
      }
      if (l < cnt && live) write_alt(a, n, j0 + l, mine, p, logS, a.route == 2 ? logf(sel) : 0.f, bad);
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
      const float zm = Vec16<T>::max_of(r) * s.scale;
      if (zm > p.R || (where == -2 && zm == p.R)) where = b;
      part_shift(p, max_nan(p.R, zm));
      const F2 scale2 = f2(s.scale, s.scale), ref2 = f2(-p.R, -p.R), log2 = f2(kLog2e, kLog2e);
      F2 S2 = f2(p.S, 0.f), U2 = f2(p.U, 0.f);
#pragma unroll
      for (int j = 0; j < kRowBatch; j++) {
        float x[V];
        Vec16<T>::unpack(r[j], x);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          float d0, d1, t0, t1;
          f2_get(f2_fma(f2(x[e], x[e + 1]), scale2, ref2), d0, d1);
          const F2 d = f2(fmaxf(d0, kFloorD), fmaxf(d1, kFloorD));
          f2_get(f2_mul(d, log2), t0, t1);
          const F2 y = f2(ex2(t0), ex2(t1));
          S2 = f2_add(S2, y);
          U2 = f2_fma(y, d, U2);
        }
      }
      float s0, s1;
      f2_get(S2, s0, s1);
      p.S = s0 + s1;
      f2_get(U2, s0, s1);
      p.U = s0 + s1;
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
