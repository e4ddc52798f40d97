// rows.cuh -- log probabilities over rows of logits: kernels of gmm_logprobs,
// gmm_logprobs_backward and gmm_route.
//
// A row holds one logit x_k per class (a mixture component, a vocabulary entry,
// an expert) and z_k = fl32(scale * x_k).  With c = scale * log2 e, a reference B
// near the largest c x_k, and t_k = c x_k - B:
//   S = sum_k 2^{t_k}            lse = log 2 (B + log2 S)
//   U = sum_k 2^{t_k} t_k        log p_k = log 2 (t_k - log2 S)
//                                H = -sum_k p_k log p_k = log 2 (log2 S - U / S)
// and the m classes of largest z, equal z in ascending index order.
//
// S and U come from one pass.  Any B does as long as no 2^t overflows; partial
// results with other references merge by S <- S 2^a, U <- 2^a (U + a S) for a
// difference a of theirs, in a fixed order.  t is one fused multiply-add, so a
// rounded B takes nothing from log p and H.  Everything is held in 32 bits.
#pragma once
#include <float.h>

#include "common.cuh"
#include "sm100_prims.cuh"
#include "vec16.cuh"

namespace scem {

constexpr int kMaxAlt = 32;          // most alternatives per row
constexpr float kFloorT = -200.f;    // 2^-200 is 0 in float32
constexpr float kFloorD = -150.f;    // and so is e^-150
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

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

// Reference, S and U of a part of a row.
struct Part {
  float B, S, U;
};

constexpr float kFar = 1e30f;  // rows with a |c x| beyond kNear take a path of their own
constexpr float kNear = 1e29f;

__device__ __forceinline__ Part part_empty() { return {-kFar, 0.f, 0.f}; }

// S and U to a reference a powers of two lower (a <= 0: higher).
__device__ __forceinline__ void sums_shift(float& S, float& U, float a) {
  a = fmaxf(a, kFloorT);
  const float f = ex2(a);
  U = f * fmaf(a, S, U);
  S *= f;
}

// Over groups of kLanes lanes, in a fixed order.
template <int kLanes>
__device__ __forceinline__ Part part_reduce(Part p) {
  float B = p.B;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) B = max_nan(B, __shfl_xor_sync(0xffffffffu, B, o));
  sums_shift(p.S, p.U, p.B - B);
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) {
    p.S += __shfl_xor_sync(0xffffffffu, p.S, o);
    p.U += __shfl_xor_sync(0xffffffffu, p.U, o);
  }
  return {B, p.S, p.U};
}

// Floats as unsigned integers of the same order; 0 for -inf (masked).
__device__ __forceinline__ uint32_t float_order(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);  // -0 and +0 are equal
  return z == -INFINITY ? 0u : b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_float(uint32_t o) {
  return o == 0u ? -INFINITY : __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

// Key of an entry: larger keys are better, 0 is none.  Larger z first, then the
// lower index; z = -inf (masked) is none.
__device__ __forceinline__ uint64_t entry_key(float z, uint32_t idx) {
  const uint32_t o = float_order(z);
  return o == 0u ? 0ull : ((uint64_t)o << 32) | (0xffffffffu - idx);
}
__device__ __forceinline__ uint32_t key_idx(uint64_t k) { return 0xffffffffu - (uint32_t)k; }
__device__ __forceinline__ float key_z(uint64_t k) { return order_float((uint32_t)(k >> 32)); }

__device__ __forceinline__ uint64_t warp_max_key(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo =
      __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return ((uint64_t)hi << 32) | lo;
}

// What a row's sums say.
struct RowSums {
  float B, L, H;     // lse = log 2 (B + L), or scale B + L where B is an x
  float scale;
  bool bad, empty;   // a NaN or +inf in the row; nothing but masked classes
  bool logit;
  // relative to B = about the largest c x
  static __device__ __forceinline__ RowSums near(const Part& p, float scale) {
    const float l = log2f(p.S);
    return {p.B, l, fmaxf(kLn2 * (l - p.U / p.S), 0.f), scale, false, false, false};
  }
  // relative to the largest x, t = c (x_k - x)
  static __device__ __forceinline__ RowSums at(float x, float scale, float S, float U) {
    const float Z = x * scale, l = logf(S);
    return {x, l, fmaxf(fmaf(-kLn2, U / S, l), 0.f), scale, !(Z < INFINITY), Z == -INFINITY, true};
  }
  __device__ __forceinline__ float lse() const {
    return logit ? fmaf(B, scale, L) : kLn2 * (B + L);
  }
  // Of a class at x: from the exponent that the sums had for it.  (From z, a product rounded
  // otherwise, log p is off by up to |z| 2^-23, and above 0 for a class that has the row to
  // itself: 3e-4 at a scale of 100 and an x of 60.)
  __device__ __forceinline__ float log_p(float x) const {
    const float z = x * scale;
    const float d = logit             ? fmaf(x - B, scale, -L)
                    : fabsf(z) < kNear ? kLn2 * (fmaf(x, scale * kLog2e, -B) - L)
                                       : z - lse();
    return fminf(d, 0.f);
  }
};

// By one thread: lse, entropy and the log p of row n's label id, which stands at x.
__device__ __forceinline__ void write_row(const RowArgs& a, int64_t n, const RowSums& s, int id,
                                          float x) {
  const float nan = __int_as_float(0x7fffffff);
  if (s.bad && a.flags) atomicOr(a.flags, GMM_DEVFLAG_NONFINITE_X);
  if (a.lse) a.lse[n] = s.bad ? nan : s.empty ? -INFINITY : s.lse();
  if (a.entropy) a.entropy[n] = s.bad ? nan : s.empty ? 0.f : s.H;
  if (a.ids) {
    const bool legal = id >= 0 && id < a.K;
    if (id != -1 && !legal && a.flags) atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
    a.logp[n] = id == -1                   ? 0.f  // no label
                : s.bad || !legal          ? nan
                : x * a.scale == -INFINITY ? -INFINITY
                                           : s.log_p(x);
  }
}

// Alternative j of row n: class k (-1: none) of this log p; sel: log of the m chosen classes'
// probability.
__device__ __forceinline__ void write_alt(const RowArgs& a, int64_t n, int j, int k, float lp,
                                          const RowSums& s, float sel) {
  const float nan = __int_as_float(0x7fffffff);
  const bool none = s.bad || k < 0;
  a.top_idx[n * a.m + j] = none ? -1 : k;
  float v;
  if (a.route == 0)
    v = s.bad ? nan : none ? -INFINITY : lp;
  else
    v = s.bad ? nan : none ? 0.f : expf(a.route == 2 ? lp - sel : lp);
  a.top_val[n * a.m + j] = v;
}

// ------------------------------------------------------------------ short rows
// kLanes lanes hold a row of at most kLanes * kEl classes in registers, so a
// warp holds 32 / kLanes rows; lane l takes vectors l, l + kLanes, ... of 16
// bytes.  kVec: rows start on 16 bytes (else the same entries one by one).
//
// Alternatives in m rounds.  Only each vector's largest entry stays in registers;
// a round finds the lowest vector that holds the row's largest, reads it again
// (it is in L1), an entry per lane, and leaves it with its largest entry behind the
// one just taken.
//
// Few lanes with many entries each: 1e6 rows of 256 fp32 with two alternatives take 221 us
// with 8 lanes of 32, 297 with 16 of 16 and 464 with 32 of 8 (shuffles and the rounds'
// fixed part are shared by 32 / kLanes rows).  A few hundred rows take 32 lanes of 8
// (2.2 against 2.4 us).  Without alternatives the rows above take 165 us (6.2 TB/s); each
// alternative adds about 30 us, and issue slots bound it (73 % busy).  Those are short runs; back
// to back the GPU is at its power limit and clocks down to 1.67 GHz: 246 to 252 us.
// The fp32 instances with 32 entries per lane spill 48 to 180 bytes per thread at the 48 registers
// that 5 CTAs per SM leave.  A row narrower than its places pays for all of them, and has its
// exponents clamped: 2e8 fp32 logits in rows of 300 (512 places) take 202 us where rows of 512
// take 150, in rows of 600 (1,024) 187; in rows of 1,024, 179.
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

// Over groups of kLanes lanes.
template <int kLanes>
__device__ __forceinline__ float group_max(float v) {
  if constexpr (kLanes == 32) {
    return order_float(__reduce_max_sync(0xffffffffu, float_order(v)));
  } else {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int kLanes>
__device__ __forceinline__ int group_min(int v) {
  if constexpr (kLanes == 32) {
    return __reduce_min_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
  }
}
template <int kLanes>
__device__ __forceinline__ uint32_t group_mask() {
  return kLanes == 32 ? 0xffffffffu : (1u << (kLanes & 31)) - 1u;
}

template <typename T, int kLanes, int kEl, bool kVec>
__global__ void __launch_bounds__(256, kEl <= 16 ? 6 : 5) row_short_kernel(RowArgs a) {
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
    float xm = -INFINITY, S, U;
#pragma unroll
    for (int c = 0; c < kChunks; c++) {
      const uint4 one[1] = {r[c]};
      const float x = Vec16<T>::max_of(one);
      top[c] = x * a.scale;
      xm = max_nan(xm, x);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
      xm = max_nan(xm, __shfl_xor_sync(0xffffffffu, xm, o));
    const float ref = fmaxf(xm, -FLT_MAX);
    const F2 c2 = f2(a.scale * kLog2e, a.scale * kLog2e), ref2 = f2(-ref, -ref);
    auto sums = [&](bool clamp) {
      F2 S2 = f2(0.f, 0.f), U2 = S2;
#pragma unroll
      for (int c = 0; c < kChunks; c++) {
        float x[V];
        Vec16<T>::unpack(r[c], x);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          float t0, t1;
          f2_get(f2_mul(f2_add(f2(x[e], x[e + 1]), ref2), c2), t0, t1);
          if (clamp) t0 = fmaxf(t0, kFloorT), t1 = fmaxf(t1, kFloorT);
          const F2 y = f2(ex2(t0), ex2(t1));
          S2 = f2_add(S2, y);
          U2 = f2_fma(y, f2(t0, t1), U2);
        }
      }
      float s0, s1;
      f2_get(S2, s0, s1);
      S = s0 + s1;
      f2_get(U2, s0, s1);
      U = s0 + s1;
    };
    // a masked class gives 0 * -inf: only then the exponents are clamped
    if (a.K < kLanes * kEl) {
      sums(true);
    } else {
      sums(false);
      if (__any_sync(0xffffffffu, !(U == U))) sums(true);
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      S += __shfl_xor_sync(0xffffffffu, S, o);
      U += __shfl_xor_sync(0xffffffffu, U, o);
    }
    const RowSums row_sums = RowSums::at(xm, a.scale, S, U);
    if (l == 0 && live) {
      const int id = a.ids ? a.ids[n] : -1;
      const bool legal = id >= 0 && id < a.K;
      write_row(a, n, row_sums, id, legal ? to_f32(row[id]) : 0.f);
    }
    float last_z = INFINITY;  // the entry taken last: what follows it in the order is left
    int last_k = -1;
    for (int j0 = 0; j0 < a.m; j0 += kLanes) {
      const int cnt = min(kLanes, a.m - j0);
      float mine_z = -INFINITY;  // lane l keeps alternative j0 + l
      int mine_k = -1;
#pragma unroll 1
      for (int j = 0; j < cnt; j++) {
        float best = top[0];
#pragma unroll
        for (int c = 1; c < kChunks; c++) best = fmaxf(best, top[c]);
        best = group_max<kLanes>(best);
        int at = 1 << 30;  // the lowest vector that holds it
#pragma unroll
        for (int c = kChunks - 1; c >= 0; c--)
          if (top[c] == best) at = c * kLanes + l;
        at = group_min<kLanes>(at);
        const bool none = best == -INFINITY || at == 1 << 30;
        // lane e looks at entry e of it
        const int k = none ? 0 : at * V + l;
        const float z = l < V && !none && k < a.K ? to_f32(row[k]) * a.scale : -INFINITY;
        const uint32_t equal = __ballot_sync(
            0xffffffffu, z == best && (best < last_z || k > last_k) && !none);
        const int first = __ffs((equal >> (lane - l)) & group_mask<kLanes>()) - 1;
        if (j0 + j + 1 < a.m) {
          // what follows in that vector is left (lanes V and up reduce among themselves: the
          // vector's owner asks lane 0 of the group)
          const float next =
              group_max<(V < kLanes ? V : kLanes)>(z < best || (z == best && l > first)
                                                       ? z
                                                       : -INFINITY);
          const float left = __shfl_sync(0xffffffffu, next, lane - l);
#pragma unroll
          for (int c = 0; c < kChunks; c++)
            if (at == c * kLanes + l) top[c] = left;
        }
        last_z = best;
        last_k = none ? last_k : at * V + first;
        if (l == j && !none) {
          mine_z = best;
          mine_k = last_k;
        }
      }
      // (at a scale of 1 z is x, else x is still in L1)
      const float lp = row_sums.log_p(a.scale == 1.f || mine_k < 0 ? mine_z : to_f32(row[mine_k]));
      float sel = 0.f;
      if (a.route == 2) {  // (m is at most 8: all of them in this one round)
        sel = mine_k < 0 ? 0.f : expf(lp);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sel += __shfl_xor_sync(0xffffffffu, sel, o);
        sel = logf(sel);
      }
      if (l < cnt && live) write_alt(a, n, j0 + l, mine_k, lp, row_sums, sel);
    }
  }
}

// ------------------------------------------------------------------ long rows
// One cluster of C CTAs per row, each CTA a contiguous slice of its 16-byte
// vectors, each warp a contiguous slice of that; the row's unaligned ends go to
// the first and the last warp.  A warp walks its slice in batches of kRowBatch
// vectors per lane.  Each lane copies its own vectors into its own places of a ring
// in shared memory, kRowStages batches ahead, and reads them back itself: the loads
// in flight cost no registers and nobody waits for anybody.
//
// Alternatives without a second pass over the row.  Each warp finds the Q largest of its
// lanes' maxima (Q a little over m / 8); the m-th largest of the 8 Q is a lower bound of the
// CTA's m-th largest entry.  Each warp also keeps the largest entry of each of its units (up to
// kRowUnits runs of consecutive batches).  Only units that reach the bound are read again,
// and only entries that reach it are candidates: about m of them, put in order by counting,
// for each, how many are better.  Where ties or masks leave more candidates than the buffer
// holds, the m units of largest entry (which hold the m best, or m units would hold a better
// one each) give a sorted list of their best each, and those merge.
//
// Measured: 4096 rows of 131,072 bf16 without alternatives 203 to 214 us back to back (5.0 to
// 5.3 TB/s; 164 us at the copy rate), at the 1000 W limit, which holds the clock at 1.54 GHz; 175 to
// 190 us in short runs.  The exponentials bind (the pipe that makes them is 70 % busy, 16 per
// clock and SM) with the issue slots (55 %).  Exponentials by polynomial on the
// multiply-add pipe (1 or 2 in 16), batches of 8 vectors, and 3 to 8 CTAs per SM of other
// sizes gave nothing or lost.  1023 rows of 100,003 fp32, partly masked, with five
// alternatives: 82 to 86 us (4.8 to 5.0 TB/s).  One row: 4.9 us, 10.5 with eight alternatives.
// Many rows of little more than 1,024 classes are far from the copy rate: a CTA's fixed part for
// a row, 3 us and twice that with alternatives, is then most of its time.  2e8 bf16 logits (61 us
// at the copy rate) in rows of 1,100 take 1,243 us, of 2,048 635, of 5,000 265, of 8,192 169; with
// eight alternatives twice as much.
constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kRowBatch = 4;
constexpr int kRowCtas = 4;  // resident per SM
constexpr int kRowStages = 3;
constexpr int kRowStep = 32 * kRowBatch;  // vectors of a warp's batch
constexpr int kRowUnits = 32;  // per warp, at most (a lane each)
constexpr int kRowCand = 512;
constexpr int kRowLists = kMaxAlt / kRowWarps + 3;  // most lane maxima kept per warp
constexpr float kLargeSum = 1048576.f;  // of a lane: its reference is raised beyond
__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sm100::smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

template <typename T>
struct RowSlice {
  static constexpr int V = Vec16<T>::n;
  const T* row;
  float scale;
  int head, tail0, tailn;  // entries before the first vector; first entry after the last; count
  int v0, v1;              // this CTA's vectors
  int per_unit;            // batches per unit
  bool first, last;

  __device__ __forceinline__ RowSlice(const RowArgs& a, int64_t n, int rank, int C) {
    row = (const T*)a.Z + n * a.ld;
    scale = a.scale;
    const uint32_t off = (uint32_t)((uintptr_t)row & 15u);
    head = min(a.K, (int)(((16u - off) & 15u) / sizeof(T)));
    const int nv = (a.K - head) / V;
    tail0 = head + nv * V;
    tailn = a.K - tail0;
    v0 = nv * rank / C;  // (K is at most 2^24 and C at most 8)
    v1 = nv * (rank + 1) / C;
    const int most = (v1 - v0 + kRowWarps - 1) / kRowWarps;  // vectors of a warp
    per_unit = max(1, (most + kRowUnits * kRowStep - 1) / (kRowUnits * kRowStep));
    first = rank == 0;
    last = rank == C - 1;
  }
  // first vector of warp w's slice
  __device__ __forceinline__ int begin(int w) const {
    return v0 + (v1 - v0) * w / kRowWarps;
  }
  __device__ __forceinline__ int batches(int w) const {
    return (begin(w + 1) - begin(w) + kRowStep - 1) / kRowStep;
  }
  // the last unit of the last warp, which has the row's tail
  __device__ __forceinline__ int tail_unit() const {
    return max(0, batches(kRowWarps - 1) - 1) / per_unit;
  }
  __device__ __forceinline__ const T* vec(int v) const { return row + head + (int64_t)v * V; }
  __device__ __forceinline__ float x(int k) const { return to_f32(row[k]); }

  // f(z, k) for the entries with z >= least of unit u of warp w, shared out over the lanes
  // (most vectors have none)
  template <typename Fn>
  __device__ __forceinline__ void each(int w, int u, int lane, float least, Fn f) const {
    const int end = min(begin(w) + (u + 1) * per_unit * kRowStep, begin(w + 1));
#pragma unroll 1
    for (int v = begin(w) + u * per_unit * kRowStep + lane; v < end; v += kRowStep) {
      uint4 r[kRowBatch];  // all on their way before the first is looked at
#pragma unroll
      for (int j = 0; j < kRowBatch; j++)
        r[j] = v + 32 * j < end ? load16(vec(v + 32 * j)) : Vec16<T>::neg_inf();
      uint32_t hit = 0;
#pragma unroll
      for (int j = 0; j < kRowBatch; j++) {
        const uint4 one[1] = {r[j]};
        if (Vec16<T>::max_of(one) * scale >= least) hit |= 1u << j;
      }
#pragma unroll 1
      for (; hit; hit &= hit - 1) {
        const int j = __ffs(hit) - 1;
        uint4 q = r[0];
#pragma unroll
        for (int i = 1; i < kRowBatch; i++)
          if (j == i) q = r[i];
        float e[V];
        Vec16<T>::unpack(q, e);
#pragma unroll
        for (int i = 0; i < V; i++)
          if (e[i] * scale >= least) f(e[i] * scale, head + (v + 32 * j) * V + i);
      }
    }
    auto single = [&](int k) {
      const float z = x(k) * scale;
      if (z >= least) f(z, k);
    };
    if (first && w == 0 && u == 0 && lane < head) single(lane);
    if (last && w == kRowWarps - 1 && u == tail_unit() && lane < tailn) single(tail0 + lane);
  }
};

// S and U with the largest logit X as the reference: t = c (x - X).
struct FarSums {
  float X, S, U;
};

struct RowShared {
  Part part[kRowWarps];
  Part total;
  FarSums far;  // with near == 0
  int near;     // total is good
  int id;       // the row's label and its x
  float id_x;
  int count;
  float least;  // lower bound of the m-th largest z
  uint32_t lane_top[kRowWarps * kRowLists];
  uint64_t list[kRowWarps][kMaxAlt];
  uint64_t win[kMaxAlt];
  uint64_t out[kMaxAlt];
  // the candidates, or a list of them per winning unit (list j from j * (2 m - j + 1) / 2:
  // unit j, j better units before it, gives at most m - j)
  uint64_t cand[kMaxAlt * (kMaxAlt + 1) / 2];
};
static_assert(kRowCand <= kMaxAlt * (kMaxAlt + 1) / 2, "candidate buffer");

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

// Sum over the CTA, and largest value of it, in every thread.
__device__ __forceinline__ float cta_sum(RowShared& sh, float v) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.part[threadIdx.x >> 5].S = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < kRowWarps; i++) v += sh.part[i].S;
  return v;
}
__device__ __forceinline__ float cta_max(RowShared& sh, float v) {
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.part[threadIdx.x >> 5].S = v;
  __syncthreads();
  v = -INFINITY;
  for (int i = 0; i < kRowWarps; i++) v = max_nan(v, sh.part[i].S);
  return v;
}

// The slice once more, from memory, with its largest logit X as the reference and
// t = c (x - X): for what the pass above does not cover, a NaN or an infinity, or logits so
// far from 0 that c x overflows (all at the type's lowest value, say).
template <typename T>
__device__ __noinline__ FarSums far_sums(RowArgs a, int64_t n, int rank, int C, RowShared& sh) {
  const RowSlice<T> s(a, n, rank, C);
  const int t = threadIdx.x;
  const float c = a.scale * kLog2e;
  float X = -INFINITY, S = 0.f, U = 0.f;
  auto each = [&](auto f) {
    if (s.first && t < s.head) f(s.x(t));
    for (int v = s.v0 + t; v < s.v1; v += kRowBatch * kRowThreads) {
      uint4 r[kRowBatch];
#pragma unroll
      for (int j = 0; j < kRowBatch; j++)
        r[j] = v + j * kRowThreads < s.v1 ? load16(s.vec(v + j * kRowThreads))
                                          : Vec16<T>::neg_inf();
#pragma unroll
      for (int j = 0; j < kRowBatch; j++) {
        float x[Vec16<T>::n];
        Vec16<T>::unpack(r[j], x);
#pragma unroll
        for (int e = 0; e < Vec16<T>::n; e++) f(x[e]);
      }
    }
    if (s.last && t < s.tailn) f(s.x(s.tail0 + t));
  };
  each([&](float x) { X = max_nan(X, x); });
  X = cta_max(sh, X);
  const float ref = fmaxf(X, -FLT_MAX);
  each([&](float x) {
    const float e = fmaxf((x - ref) * c, kFloorT), y = ex2(e);
    S += y;
    U = fmaf(y, e, U);
  });
  return {X, cta_sum(sh, S), cta_sum(sh, U)};
}

// The q largest of the warp's lane keys, in order, into the warp's list.
__device__ __forceinline__ void warp_top(RowShared& sh, int q, uint64_t key) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll 1
  for (int j = 0; j < q; j++) {
    const uint64_t best = warp_max_key(key);
    if (lane == 0) sh.list[w][j] = best;
    if (key == best) key = 0;
  }
}

// The m best of keys[0 .. n), different where not 0, in order into out (0 where they run out),
// by the whole CTA: a key's place is the number of better ones.
__device__ __forceinline__ void cta_rank(const uint64_t* keys, int n, int m, uint64_t* out) {
  if (threadIdx.x < m) out[threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kRowThreads) {
    const uint64_t k = keys[i];
    if (k == 0) continue;
    int place = 0;
#pragma unroll 2
    for (int q = 0; q < n; q++) place += keys[q] > k;
    if (place < m) out[place] = k;
  }
}

// Lane maxima that a warp keeps.
__device__ __forceinline__ int row_lists(int m) {
  return min(m, (m + kRowWarps - 1) / kRowWarps + 3);
}

// The warp's largest lane maxima (z), any order among equal ones.
__device__ __forceinline__ void lane_tops(RowShared& sh, int q, float z) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t o = float_order(z);
#pragma unroll 1
  for (int j = 0; j < q; j++) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, o);
    if (lane == 0) sh.lane_top[w * q + j] = best;
    if (lane == __ffs(__ballot_sync(0xffffffffu, o == best)) - 1) o = 0;
  }
}

// By one warp: the m-th largest of the warps' lane maxima into sh.least.
__device__ __forceinline__ void lane_bound(RowShared& sh, int m) {
  const int lane = threadIdx.x & 31, n = kRowWarps * row_lists(m);
  static_assert(kRowWarps * kRowLists <= 64, "two per lane");
  uint32_t mine[2];
  int above[2] = {0, 0}, equal[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 2; h++) mine[h] = lane + 32 * h < n ? sh.lane_top[lane + 32 * h] : 0;
#pragma unroll 2
  for (int i = 0; i < n; i++) {
    const uint32_t o = sh.lane_top[i];
#pragma unroll
    for (int h = 0; h < 2; h++) {
      above[h] += o > mine[h];
      equal[h] += o == mine[h];
    }
  }
  uint32_t found = 0;
#pragma unroll
  for (int h = 0; h < 2; h++)
    if (mine[h] != 0 && above[h] < m && m <= above[h] + equal[h]) found = mine[h];
  found = __reduce_max_sync(0xffffffffu, found);
  if (lane == 0) sh.least = found ? order_float(found) : -FLT_MAX;
}

// The m best of the slice into sh.out, given the bound sh.least and each lane's unit_z, the
// largest z of the warp's unit `lane`.  Ends with a barrier.
template <typename T>
__device__ __forceinline__ void row_alternatives(const RowSlice<T>& s, RowShared& sh, int m,
                                                 float unit_z) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const float least = sh.least;
  for (uint32_t units = __ballot_sync(0xffffffffu, unit_z >= least); units; units &= units - 1)
    s.each(w, __ffs(units) - 1, lane, least, [&](float z, int k) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < kRowCand) sh.cand[at] = entry_key(z, (uint32_t)k);
    });
  __syncthreads();
  const int count = sh.count;
  if (count <= kRowCand) {
    cta_rank(sh.cand, count, m, sh.out);
    __syncthreads();
    return;
  }
  __syncthreads();  // everyone has read the lists and the count; the buffer is free
  warp_top(sh, m, entry_key(unit_z, (uint32_t)threadIdx.x));
  __syncthreads();
  if (w == 0)
    merge_lists(
        m, [&](int i) { return lane < kRowWarps && i < m ? sh.list[lane][i] : 0ull; },
        [&](int j, uint64_t k) {
          if (lane == 0) sh.win[j] = k;
        });
  __syncthreads();
  for (int j = w; j < m; j += kRowWarps) {
    const int unit = (int)key_idx(sh.win[j]);
    uint64_t* list = sh.cand + j * (2 * m - j + 1) / 2;
    uint64_t last = ~0ull;
    for (int i = 0; i < m - j; i++) {
      uint64_t best = 0;
      if (last != 0 && sh.win[j] != 0)
        s.each(unit >> 5, unit & 31, lane, -FLT_MAX, [&](float z, int k) {
          const uint64_t key = entry_key(z, (uint32_t)k);
          if (key < last && key > best) best = key;
        });
      last = warp_max_key(best);
      if (lane == 0) list[i] = last;
    }
  }
  __syncthreads();
  if (w == 0)
    merge_lists(
        m,
        [&](int i) {
          return lane < m && i < m - lane ? sh.cand[lane * (2 * m - lane + 1) / 2 + i] : 0ull;
        },
        [&](int j, uint64_t k) {
          if (lane == 0) sh.out[j] = k;
        });
  __syncthreads();
}

// What the C CTAs of a row found, joined by one warp of the first: lane r reads CTA r's
// sums.  Parts of the same kind merge; a NaN or infinity decides the row, then logits far
// above 0, ordinary ones, logits far below, and nothing.
__device__ __forceinline__ uint32_t ld_cta(const void* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];"
               : "=r"(v)
               : "r"(sm100::map_to_rank(sm100::smem_u32(p), rank))
               : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_cta64(const uint64_t* p, int rank) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];"
               : "=l"(v)
               : "r"(sm100::map_to_rank(sm100::smem_u32(p), rank))
               : "memory");
  return v;
}
__device__ __forceinline__ RowSums join_sums(const RowShared& sh, int C, float scale) {
  const int lane = threadIdx.x & 31;
  const float c = scale * kLog2e;
  Part p = part_empty();
  FarSums f = {-INFINITY, 0.f, 0.f};
  int kind = -1;
  if (lane < C) {
    if (ld_cta(&sh.near, lane)) {
      kind = 1;
      p = {__uint_as_float(ld_cta(&sh.total.B, lane)), __uint_as_float(ld_cta(&sh.total.S, lane)),
           __uint_as_float(ld_cta(&sh.total.U, lane))};
    } else {
      f = {__uint_as_float(ld_cta(&sh.far.X, lane)), __uint_as_float(ld_cta(&sh.far.S, lane)),
           __uint_as_float(ld_cta(&sh.far.U, lane))};
      const float Z = f.X * scale;
      kind = !(Z < INFINITY) ? 3 : Z == -INFINITY ? -1 : f.X > 0.f ? 2 : 0;
    }
  }
  const int best = __reduce_max_sync(0xffffffffu, kind);
  if (best == 1) return RowSums::near(part_reduce<32>(kind == 1 ? p : part_empty()), scale);
  if (kind != best) f = {-INFINITY, 0.f, 0.f};
  float X = f.X;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) X = max_nan(X, __shfl_xor_sync(0xffffffffu, X, o));
  sums_shift(f.S, f.U, (f.X - X) * c);
  return RowSums::at(X, scale, warp_sum(f.S), warp_sum(f.U));
}

// kAlt: with alternatives.
template <typename T, bool kAlt>
__global__ void __launch_bounds__(kRowThreads, kRowCtas) row_long_kernel(RowArgs a, int C) {
  constexpr int V = Vec16<T>::n;
  extern __shared__ uint4 ring[];  // [warp][stage][batch vector][lane]
  __shared__ RowShared sh;
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const int rank = C > 1 ? (int)sm100::cluster_ctarank() : 0;
  const int64_t clusters = gridDim.x / C;
  const float c = a.scale * kLog2e;
  uint4* own = ring + w * kRowStages * kRowStep + lane;
  const T* from;  // the lane's first vector of the batch to copy next
  int left;       // vectors of the warp's slice from there on
  auto fetch_from = [&](const RowSlice<T>& s) {
    from = s.vec(s.begin(w) + lane);
    left = s.begin(w + 1) - s.begin(w) - lane;
  };
  auto fetch = [&](uint4* dst) {
    if (left >= kRowStep) {
#pragma unroll
      for (int j = 0; j < kRowBatch; j++) copy_async16(dst + 32 * j, from + j * 32 * V);
    } else {
#pragma unroll
      for (int j = 0; j < kRowBatch; j++)
        if (left > 32 * j) copy_async16(dst + 32 * j, from + j * 32 * V);
    }
    copy_async_commit();
    from += kRowStep * V;
    left -= kRowStep;
  };
  fetch_from(RowSlice<T>(a, blockIdx.x / C, rank, C));
#pragma unroll
  for (int b = 0; b < kRowStages; b++) fetch(own + b * kRowStep);
  for (int64_t n = blockIdx.x / C; n < a.N; n += clusters) {
    const RowSlice<T> s(a, n, rank, C);
    float B = -kFar, S = 0.f, U = 0.f;
    float xm = -INFINITY;      // the lane's largest x: with kAlt, or while S is 0
    float unit_z = -INFINITY;  // kAlt: the largest z of the warp's unit `lane`
    bool masked = false;
    if (rank == 0 && t == kRowThreads - 1 && a.ids) {  // read while the row streams
      const int id = a.ids[n];
      sh.id = id;
      sh.id_x = id >= 0 && id < a.K ? s.x(id) : 0.f;
    }
    if (kAlt && t == 0) sh.count = 0;
    auto raise = [&](float x) {
      const float to = fmaxf(x * c, B);
      sums_shift(S, U, B - to);
      B = to;
    };
    // um: the lane's largest x in the warp's unit u, which ends here
    auto unit_end = [&](float um, int u) {
      const float z = order_float(__reduce_max_sync(0xffffffffu, float_order(um))) * a.scale;
      xm = fmaxf(xm, um);
      if (lane == u) unit_z = fmaxf(unit_z, z);
    };
    auto single = [&](bool mine, int k, int u) {
      const float x = mine ? s.x(k) : -INFINITY;
      if (mine) {
        raise(x);
        xm = fmaxf(xm, x);
        const float e = max_nan(fmaf(x, c, -B), kFloorT);
        const float y = ex2(e);
        S += y;
        U = fmaf(y, e, U);
      }
      if (kAlt) unit_end(x, u);
    };
    if (s.first && w == 0 && s.head > 0) single(lane < s.head, lane, 0);

    const int nb = s.batches(w);
    int here = s.begin(w + 1) - s.begin(w) - lane;  // vectors from this lane's first on
    // Adds a batch, `left` vectors of it from this lane on.  Returns its largest x.
    auto add = [&](const uint4* batch, bool clamp, int left) {
      const F2 c2 = f2(c, c), B2 = f2(-B, -B);
      F2 S2 = f2(S, 0.f), U2 = f2(U, 0.f);
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < kRowBatch; j++) {
        uint4 r[1] = {batch[32 * j]};
        if (clamp && left <= 32 * j) r[0] = Vec16<T>::neg_inf();
        if (kAlt) top = max_nan(top, Vec16<T>::max_of(r));
        float x[V];
        Vec16<T>::unpack(r[0], x);
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          F2 tt = f2_fma(f2(x[e], x[e + 1]), c2, B2);
          float t0, t1;
          f2_get(tt, t0, t1);
          if (clamp) {
            t0 = max_nan(t0, kFloorT), t1 = max_nan(t1, kFloorT);
            tt = f2(t0, t1);
          }
          const F2 y = f2(ex2(t0), ex2(t1));
          S2 = f2_add(S2, y);
          U2 = f2_fma(y, tt, U2);
        }
      }
      float s0, s1;
      f2_get(S2, s0, s1);
      S = s0 + s1;
      f2_get(U2, s0, s1);
      U = s0 + s1;
      return top;
    };
    int unit = 0, in_unit = s.per_unit;
    float um = -INFINITY;
    uint4* batch = own;
    for (int b = 0; b < nb; b++) {
      copy_async_wait<kRowStages - 1>();
      const bool whole = here + lane >= kRowStep;
      const float S0 = S, U0 = U;
      float top = -INFINITY;
      bool done = false;
      if (b > 0) {
        // The reference stays while the sums stay small: no maximum is needed.  A masked
        // class gives 0 * -inf (then the exponents are clamped from there on), a logit far
        // above the others a large or infinite sum.
        top = masked || !whole ? add(batch, true, here) : add(batch, false, here);
        done = !__any_sync(0xffffffffu, !(U == U) || !(S < kLargeSum));
        if (!done) {
          masked |= __any_sync(0xffffffffu, !(U == U) && S < kLargeSum);
          S = S0;
          U = U0;
        }
      }
      if (!done || (!kAlt && S == 0.f)) {
        float x = -INFINITY;
#pragma unroll
        for (int j = 0; j < kRowBatch; j++) {
          const uint4 r[1] = {batch[32 * j]};
          if (here > 32 * j) x = max_nan(x, Vec16<T>::max_of(r));
        }
        xm = fmaxf(xm, x);
        if (!done) {
          raise(x);
          top = add(batch, true, here);
        }
      }
      if (kAlt) {
        um = fmaxf(um, top);
        if (--in_unit == 0 || b == nb - 1) {
          unit_end(um, unit++);
          in_unit = s.per_unit;
          um = -INFINITY;
        }
      }
      fetch(batch);
      here -= kRowStep;
      batch = batch == own + (kRowStages - 1) * kRowStep ? own : batch + kRowStep;
    }
    copy_async_wait<0>();
    if (n + clusters < a.N) {  // the next row is on its way while this one is finished
      fetch_from(RowSlice<T>(a, n + clusters, rank, C));
#pragma unroll
      for (int b = 0; b < kRowStages; b++) fetch(own + b * kRowStep);
    }
    if (s.last && w == kRowWarps - 1 && s.tailn > 0)
      single(lane < s.tailn, s.tail0 + lane, s.tail_unit());

    const Part p = part_reduce<32>({B, S, U});
    if (lane == 0) sh.part[w] = p;
    if (kAlt) lane_tops(sh, row_lists(a.m), xm * a.scale);
    const bool some = __syncthreads_or(xm > -INFINITY || !(S == 0.f));
    if (w == 0) {
      const Part q = part_reduce<8>(sh.part[lane % 8]);
      if (lane == 0) {
        sh.total = q;
        sh.near = q.S > 0.f && q.S < INFINITY && fabsf(q.B) < kNear;
        sh.far = {-INFINITY, 0.f, 0.f};  // every class masked
      }
    } else if (kAlt && w == 1) {
      lane_bound(sh, a.m);
    }
    __syncthreads();
    if (kAlt) row_alternatives(s, sh, a.m, unit_z);
    if (!sh.near && some) {
      const FarSums far = far_sums<T>(a, n, rank, C, sh);
      if (t == 0) sh.far = far;
    }
    const uint64_t* alt = sh.out;
    RowSums sums;
    if (C == 1) {
      // (thread 0 wrote these; only its warp uses them)
      if (w == 0) {
        __syncwarp();
        sums = sh.near ? RowSums::near(sh.total, a.scale)
                       : RowSums::at(sh.far.X, a.scale, sh.far.S, sh.far.U);
      }
    } else {
      sm100::cluster_sync();
      if (rank == 0) {
        if (w == 0) sums = join_sums(sh, C, a.scale);
        if (kAlt) {
          for (int i = t; i < C * a.m; i += kRowThreads)
            sh.cand[i] = ld_cta64(&sh.out[i % a.m], i / a.m);
          __syncthreads();
          cta_rank(sh.cand, C * a.m, a.m, sh.win);
          __syncthreads();
          alt = sh.win;
        }
      }
    }
    if (rank == 0 && w == 0) {
      if (lane == 0) write_row(a, n, sums, a.ids ? sh.id : -1, sh.id_x);
      if (kAlt) {
        // (at a scale of 1 z is x, else x is read once more)
        const uint64_t key = lane < a.m ? alt[lane] : 0;
        const int k = key ? (int)key_idx(key) : -1;
        const float lp = sums.log_p(a.scale == 1.f || k < 0 ? key_z(key) : s.x(k));
        const float sel = a.route == 2 ? logf(warp_sum(k < 0 ? 0.f : expf(lp))) : 0.f;
        if (lane < a.m) write_alt(a, n, lane, k, lp, sums, sel);
      }
    }
    if (C > 1)
      sm100::cluster_sync();  // the others' shared memory has been read
    else
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
//
// What lse's rounding costs p is 3 |lse| 2^-24 in relation.  Rows with an |lse| from kFarLse on
// (2^-12) are therefore summed once more, by one group for the whole row: at the type's lowest value,
// say, lse has no digit of log K left.
//
// HBM bounds it: 4096 rows of 131,072 bf16 take 326 us (6.6 TB/s read and written).  Short
// rows wait for their scalars first, so those and the first vectors are loaded together:
// 60,001 rows of 1,024 fp32 with four alternatives 95 us (5.2 TB/s; 112 one after another, before
// rows far from 0 had blocks of their own).  Rows of 256 fp32 leave half a warp's vectors
// empty: 1e6 of them take 781 us where the copy rate would take 317.
// Where a row of Z and its row of dZ start in different places of 16 bytes, it is read and written
// entry by entry: 2,000 rows of 50,000 bf16 take 279 us from a pitch of 50,003, and 71 from 50,000.
struct RowGradArgs {
  const void* Z;
  void* dZ;
  int64_t N, ld, ldd;
  int K;
  int slices;  // per row
  unsigned blocks;  // of the grid, for the slices
  float scale;
  const int32_t* ids;
  const float *lse, *entropy, *dlogp, *dentropy, *dlse;
  int m;
  const int32_t* top_idx;
  const float* dtop;
  uint32_t* flags;
};

constexpr float kFarLse = 1024.f;

template <int kGroup>
__device__ __forceinline__ void group_sync() {
  if constexpr (kGroup == 32)
    __syncwarp();
  else
    __syncthreads();
}

// The row's largest x and log sum_k e^{scale (x_k - x)}, by a group; part: a float per warp.
template <typename T, int kGroup>
__device__ __noinline__ float2 grad_row_sums(const T* row, int K, float scale, float* part) {
  const int t = threadIdx.x % kGroup, w = t >> 5;
  constexpr int kAhead = 8;
  auto each = [&](auto f) {
    for (int k = t; k < K; k += kAhead * kGroup) {
      float x[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; j++)
        x[j] = k + j * kGroup < K ? to_f32(row[k + j * kGroup]) : -INFINITY;
#pragma unroll
      for (int j = 0; j < kAhead; j++) f(x[j]);
    }
  };
  auto join = [&](float v, auto f) {  // in a fixed order
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(0xffffffffu, v, o));
    if constexpr (kGroup > 32) {
      __syncthreads();
      if ((t & 31) == 0) part[w] = v;
      __syncthreads();
      v = part[0];
      for (int i = 1; i < kGroup / 32; i++) v = f(v, part[i]);
    }
    return v;
  };
  float X = -FLT_MAX, S = 0.f;
  each([&](float x) { X = fmaxf(X, x); });
  X = join(X, [](float a, float b) { return fmaxf(a, b); });
  const float c = scale * kLog2e;
  each([&](float x) { S += ex2(fmaxf((x - X) * c, kFloorT)); });
  return make_float2(X, logf(join(S, [](float a, float b) { return a + b; })));
}

struct GradShared {  // of a group
  int idx[kMaxAlt + 1];
  float coef[kMaxAlt + 1];
  float part[8];  // a float per warp
};

__device__ __forceinline__ bool grad_is_far(float lse) {
  return fabsf(lse) >= kFarLse && fabsf(lse) < INFINITY;
}

// Slice `rank` of `slices` of row n; of a row far from 0 the first slice is all of it (without kFar
// it is left as it is).
template <typename T, int kGroup, bool kFar>
__device__ __forceinline__ void grad_row(const RowGradArgs& a, int64_t n, int rank, int slices,
                                         GradShared& sh) {
  constexpr int V = Vec16<T>::n;
  constexpr int kBatch = 4;  // 16-byte vectors in flight per thread
  constexpr int kOwn = (kMaxAlt + 1 + kGroup - 1) / kGroup;
  const int t = threadIdx.x % kGroup;
  const T* row = (const T*)a.Z + n * a.ld;
  T* out = (T*)a.dZ + n * a.ldd;
  const uint32_t off = (uint32_t)((uintptr_t)row & 15u);
  const bool together = off == (uint32_t)((uintptr_t)out & 15u);  // else entry by entry
  const int head = together ? min(a.K, (int)(((16u - off) & 15u) / sizeof(T))) : a.K;
  const int nv = (a.K - head) / V;
  const int tail0 = head + nv * V;
  int h0 = (int)((int64_t)head * rank / slices);
  int h1 = (int)((int64_t)head * (rank + 1) / slices);
  int v0 = (int)((int64_t)nv * rank / slices);
  int v1 = (int)((int64_t)nv * (rank + 1) / slices);
  bool last = rank == slices - 1;

  // The first vectors are on their way while the row's scalars are read.  (Nobody else
  // writes this slice, so what is loaded early is what stands there.)
  const T* vin = row + head;
  T* vout = out + head;
  uint4 r[kBatch];
  auto load = [&](int v) {
#pragma unroll
    for (int j = 0; j < kBatch; j++)
      if (v + j * kGroup < v1) r[j] = load16(vin + (int64_t)(v + j * kGroup) * V);
  };
  load(v0 + t);

  // So are the scalars, all at once, and then the named entries: alternatives 0..m-1, the label.
  const float lse_in = a.lse[n];
  const int id = a.ids ? a.ids[n] : -1;
  float slope = a.dlse ? a.dlse[n] : 0.f;
  const float h = a.dentropy ? a.dentropy[n] : 0.f;
  const float H = a.dentropy ? a.entropy[n] : 0.f;
  int named_k[kOwn];
  float named_c[kOwn], named_x[kOwn];
  bool here[kOwn];  // the entry exists and lies in this slice
#pragma unroll
  for (int i = 0; i < kOwn; i++) {
    const int j = t + i * kGroup;
    named_k[i] = j < a.m ? a.top_idx[n * a.m + j] : j == a.m ? id : -1;
    named_c[i] = j < a.m ? a.dtop[n * a.m + j] : j == a.m && a.dlogp ? a.dlogp[n] : 0.f;
  }
  const bool empty = lse_in == -INFINITY;
  float X = 0.f, lse = empty ? INFINITY : lse_in;  // log p = scale (x - X) - lse
  if (grad_is_far(lse_in)) {
    if (!kFar || rank > 0) return;
    const float2 sums = grad_row_sums<T, kGroup>(row, a.K, a.scale, sh.part);
    X = sums.x;
    lse = sums.y;
    h0 = v0 = 0;
    h1 = head;
    v1 = nv;
    last = true;
    load(t);
  }
#pragma unroll
  for (int i = 0; i < kOwn; i++) {
    const int j = t + i * kGroup, k = named_k[i];
    const bool legal = k >= 0 && k < a.K;
    if (!legal && k != -1 && rank == 0 && a.flags) atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
    const bool used = legal && !empty && (j < a.m || a.dlogp);
    here[i] = used && (k < head    ? k >= h0 && k < h1
                       : k < tail0 ? (k - head) / V >= v0 && (k - head) / V < v1
                                   : last);
    named_x[i] = here[i] ? to_f32(row[k]) : 0.f;
    if (j <= a.m) {
      sh.idx[j] = used ? k : -1;
      sh.coef[j] = used ? named_c[i] : 0.f;
    }
  }
  group_sync<kGroup>();
  for (int j = 0; j <= a.m; j++) slope -= sh.coef[j];
  // dx = p (A + B log p) away from the named entries
  const bool bad = !(lse_in < INFINITY);
  const float A = empty ? 0.f
                  : bad ? __int_as_float(0x7fffffff)
                        : a.scale * (slope - h * H);
  const float B = empty || bad ? 0.f : -a.scale * h;
  auto grad = [&](float x) {
    const float lp = fmaxf(fmaf(kFar ? x - X : x, a.scale, -lse), kFloorD);
    return ex2(lp * kLog2e) * fmaf(B, lp, A);
  };
  float named[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; i++) {
    named[i] = 0.f;
    if (here[i]) {
      float c = 0.f;  // an entry may be named more than once
      for (int q = 0; q <= a.m; q++) c += sh.idx[q] == named_k[i] ? sh.coef[q] : 0.f;
      named[i] = fmaf(a.scale, c, grad(named_x[i]));
    }
  }
  group_sync<kGroup>();
  for (int k = h0 + t; k < h1; k += kGroup) from_f32(out + k, grad(to_f32(row[k])));
  for (int v = v0 + t; v < v1;) {
#pragma unroll
    for (int j = 0; j < kBatch; j++)
      if (v + j * kGroup < v1) {
        float x[V];
        Vec16<T>::unpack(r[j], x);
#pragma unroll
        for (int e = 0; e < V; e++) x[e] = grad(x[e]);
        *reinterpret_cast<uint4*>(vout + (int64_t)(v + j * kGroup) * V) = Vec16<T>::pack(x);
      }
    v += kBatch * kGroup;
    load(v);
  }
  if (last)
    for (int k = tail0 + t; k < a.K; k += kGroup) from_f32(out + k, grad(to_f32(row[k])));
  group_sync<kGroup>();
#pragma unroll
  for (int i = 0; i < kOwn; i++)
    if (here[i]) from_f32(out + named_k[i], named[i]);
  group_sync<kGroup>();
}

// Rows of a warp each: those far from 0 go to blocks of their own behind the others (in the others'
// loop they cost every row: 60,001 x 1,024 fp32 took 103 us, so it takes 95, without them 91).
template <typename T>
__device__ __forceinline__ void grad_far_rows(const RowGradArgs& a, GradShared& sh) {
  const int lane = threadIdx.x & 31;
  const int64_t step = (int64_t)(gridDim.x - a.blocks) * 8;
  for (int64_t n0 = (int64_t)(blockIdx.x - a.blocks) * 8 + (threadIdx.x >> 5); n0 < a.N;
       n0 += 32 * step) {
    const int64_t n = n0 + lane * step;
    for (uint32_t todo = __ballot_sync(0xffffffffu, n < a.N && grad_is_far(a.lse[n])); todo;
         todo &= todo - 1)
      grad_row<T, 32, true>(a, n0 + (__ffs(todo) - 1) * step, 0, 1, sh);
  }
}

template <typename T, int kGroup>
__global__ void __launch_bounds__(256, kGroup == 32 ? 4 : 5) row_grad_kernel(RowGradArgs a) {
  constexpr int kGroups = 256 / kGroup;
  __shared__ GradShared sh[kGroups];
  const int g = threadIdx.x / kGroup;
  if constexpr (kGroup == 32)
    if (blockIdx.x >= a.blocks) return grad_far_rows<T>(a, sh[g]);
  const int64_t items = a.N * a.slices;
  for (int64_t it = (int64_t)blockIdx.x * kGroups + g; it < items; it += (int64_t)a.blocks * kGroups) {
    const int64_t n = it / a.slices;
    grad_row<T, kGroup, kGroup != 32>(a, n, (int)(it - n * a.slices), a.slices, sh[g]);
  }
}

}  // namespace scem
