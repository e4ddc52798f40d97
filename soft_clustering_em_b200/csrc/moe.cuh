// moe.cuh -- a mixture-of-experts layer for a few tokens: kernels of gmm_moe.
//
// Token t goes to the experts idx[t][j] with weights resp[t][j] (as gmm_route or
// gmm_assign_topm return them):
//   y_t = sum_j resp_tj W_down[e] h,   h = act(W_gate[e] x_t) * (W_lin[e] x_t),  e = idx_tj
// where W_up[e] (2F x D) stacks W_gate over W_lin and W_down[e] is D x F.
//
// With few tokens the layer is bound by reading the chosen experts' weights
// (3 D F elements each) once.  Experts with more tokens than a job has columns (16, or 32 and in
// the up kernel 64 where that costs no stage) have them streamed again for each further group,
// mostly from L2.  Both kernels are a stream of jobs on one CTA per SM: 128
// weight rows of one expert against up to kN of its tokens, on the tensor cores.  The
// weights are the M operand (rows of the tile), the tokens the N operand, accumulators
// in tensor memory, two of them in turn.  The warps have a part each:
//   - four copy weight tiles and, four rows at a time (gather4), the tokens' elements by TMA
//     into a ring of stages of 64 along K (mostly 8 to 16, some 130 KB of weights per SM on
//     their way at any time, on across the jobs);
//   - four issue the products, each into an accumulator of its own;
//   - four take finished accumulators out of tensor memory and add them up.
// One thread alone takes about 600 cycles to issue a stage's copies and as many for its
// products, twice what the memory needs to deliver it, so warps take the stages in turn (two
// instead of four of each: 280 us instead of 222 for 32 tokens of 128 experts).
// (Gathering the tokens with loads instead costs a proxy fence per stage, which waits for
// every copy of the thread: a microsecond.)
// A 128-row tile may be partly filled, and columns may be empty: what stands there from
// before only reaches results that nobody takes.
//
// Kernel 1 (up) holds 64 rows of W_gate over the same 64 rows of W_lin in a tile and
// writes h for every (token, choice) into the workspace; kernel 2 (down) forms y, summing
// a token's experts in shared memory, in ascending order.  h is kept as two halves of
// the weights' type, hi + lo: columns of their own of the same product, added when they leave
// tensor memory.  bf16 has float32's range, and the pair 2^-17 of h at worst (2.5e-6 on average,
// which turns about 0.3 % of y's own roundings; a third half would take as many columns again).
// fp16 would lose lo below its smallest number, so lo is kept 2^11 times as large, never above hi:
// the pair then has 2^-22 of h, or 2^-36 where hi itself is below 2^-14.
//
// Measured: 32 tokens with 8 of 128 experts, 2048 x 768 bf16 (about 1.05 GB of weights):
// 179 to 189 us, 5.6 to 5.9 TB/s; kernel 1 alone reads 6.0 TB/s, kernel 2 5.2.  100 tokens, 4 of 32
// experts, 4096 x 1432 fp16: 224 to 229 us, 4.9 TB/s (kernel 2 on 128 SMs, 4.3).  One token, 8 of 64
// experts, 2048 x 1024: 27 us for 100 MB, of which 15 are the reading and 6 the two kernels'
// starts.  The tensor pipe is 5 to 13 % busy.  Many tokens per expert, with the routing: 64 tokens,
// 2 of 8 experts of 4096 x 1024, 71 us (31 at the copy rate); 256 tokens, 4 of 16 of 2048 x 704, 134
// (21); 256 tokens, 8 of 128 of 2048 x 768, 276 (185).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "sm100_prims.cuh"
#include "vec16.cuh"

namespace scem {

constexpr int kMoeMaxT = 256;
constexpr int kMoeMaxE = 1024;
constexpr int kMoeMaxSlots = kMoeMaxT * kMaxTopM;
constexpr int kMoeCopyWarps = 4, kMoeMmaWarps = 4;
constexpr int kMoeThreads = (4 + kMoeCopyWarps + kMoeMmaWarps) * 32;
constexpr int kMoeTile = 128;     // weight rows of a job
constexpr int kMoeK = 64;         // elements along K of a stage
constexpr int kMoeAccCols = 64;   // of an accumulator, at most
constexpr int kMoeTmemCols = 2 * kMoeMmaWarps * kMoeAccCols;
constexpr uint64_t kMoeDrainNs = 1000000000ull;

// What lo is kept multiplied by.
template <typename T>
constexpr float kMoeLo = 1.f;
template <>
constexpr float kMoeLo<__half> = 2048.f;

struct MoeArgs {
  void* Y;
  const int32_t* idx;
  const float* resp;
  void *h_hi, *h_lo;  // T * m x F each, lo directly behind hi
  int T, m, E, D, F;
  int64_t ldy;
  int act;
  int block_rows;  // down: rows of y per cluster
  int ring_bytes;  // shared memory of the stages
  uint64_t wait_ns;
  unsigned int* status;
};

// The T * m choices sorted by expert: active experts a = 0..n-1 in ascending
// order, act[a] the expert, its choices slot[off[a] .. off[a+1]) with their weights.  A
// choice that repeats an expert within its token is left out; its weight counts with the
// first one.  The order inside an expert is free: it only decides the column of a product.
struct MoeLists {
  uint16_t *act, *off, *slot;
  float* gate;
  int warp_n[8], warp_a[8], warp_most[8];
  int n;     // active experts
  int most;  // choices of the busiest
  uint32_t inv_m;
  // slot / m: exact for slots below 2^11 and m up to 8 with inv_m = ceil(2^16 / m)
  __device__ __forceinline__ int token(int slot) const { return (int)(slot * inv_m >> 16); }
};

// Bytes of the lists behind the struct, and their places.
__host__ __device__ constexpr int moe_list_bytes(int E, int slots) {
  return (E * 2 + (E + 2) * 2 + slots * 2 + slots * 4 + 3 * 16 + 255) / 256 * 256;
}
__device__ __forceinline__ void moe_place_lists(MoeLists& L, char* at, int E, int slots) {
  L.gate = (float*)at;
  at += (slots * 4 + 15) / 16 * 16;
  L.act = (uint16_t*)at;
  at += (E * 2 + 15) / 16 * 16;
  L.off = (uint16_t*)at;
  L.slot = L.off + E + 2;
}

// Up to 32 choices: by one warp, a choice per lane (a microsecond less than the general way, at
// the start of both kernels).
__device__ __forceinline__ void moe_sort_few(const MoeArgs& a, MoeLists& L) {
  const int lane = threadIdx.x, n = a.T * a.m, t0 = lane - lane % a.m;
  const uint32_t below = (1u << lane) - 1u;
  int e = lane < n ? __ldcg(a.idx + lane) : -1;
  const float weight = lane < n ? __ldcg(a.resp + lane) : 0.f;
  if (e < 0 || e >= a.E) e = -1;
  const uint32_t same = __match_any_sync(0xffffffffu, e);  // the lanes of its expert
  bool first = e >= 0;                                     // of its token's with this expert
  float gate = 0.f;
  for (int q = 0; q < a.m; q++) {
    const int j = (t0 + q) & 31;
    const float v = __shfl_sync(0xffffffffu, weight, j);
    if (same >> j & 1u) {
      gate += v;
      first = first && j >= lane;
    }
  }
  const uint32_t firsts = __ballot_sync(0xffffffffu, first), mine = same & firsts;
  const int count = __popc(mine);
  const bool leads = first && (mine & below) == 0;
  const uint32_t leaders = __ballot_sync(0xffffffffu, leads);
  int rank = 0, start = 0;  // active experts before this one, and their choices
  for (uint32_t m = leaders; m; m &= m - 1) {
    const int j = __ffs(m) - 1;
    const int other = __shfl_sync(0xffffffffu, e, j), c = __shfl_sync(0xffffffffu, count, j);
    if (other < e) rank++, start += c;
  }
  if (leads) {
    L.act[rank] = (uint16_t)e;
    L.off[rank] = (uint16_t)start;
  }
  if (first) {
    const int at = start + __popc(mine & below);
    L.slot[at] = (uint16_t)lane;
    L.gate[at] = gate;
  }
  const int most = __reduce_max_sync(0xffffffffu, leads ? count : 0);
  if (lane == 0) {
    L.n = __popc(leaders);
    L.inv_m = (65536u + a.m - 1) / a.m;
    L.off[L.n] = (uint16_t)__popc(firsts);
    L.most = most;
  }
}

// By the first 256 threads, a token each; the whole CTA calls it.  cnt: kMoeMaxE ints of shared
// memory.
__device__ __forceinline__ void moe_sort(const MoeArgs& a, MoeLists& L, int* cnt) {
  if (a.T * a.m <= 32) {
    if (threadIdx.x < 32) moe_sort_few(a, L);
    __syncthreads();
    return;
  }
  constexpr int kThreads = 256, kPer = kMoeMaxE / kThreads;
  static_assert(kMoeMaxT <= kThreads, "a token per thread");
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  int e[kMaxTopM];
  float gate[kMaxTopM];
#pragma unroll
  for (int q = 0; q < kMaxTopM; q++) {  // all on their way at once
    const bool mine = tid < a.T && q < a.m;
    e[q] = mine ? __ldcg(a.idx + tid * a.m + q) : -1;
    gate[q] = mine ? __ldcg(a.resp + tid * a.m + q) : 0.f;
  }
  for (int i = tid; i < kMoeMaxE; i += kMoeThreads) cnt[i] = 0;
#pragma unroll
  for (int q = 0; q < kMaxTopM; q++) {
    if (e[q] >= a.E) e[q] = -1;
#pragma unroll
    for (int r = 0; r < q; r++)
      if (e[q] >= 0 && e[r] == e[q]) {
        gate[r] += gate[q];
        e[q] = -1;
      }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kMaxTopM; q++)
    if (e[q] >= 0) atomicAdd(&cnt[e[q]], 1);
  __syncthreads();
  int c[kPer], sum = 0, act = 0, most = 0, xs = 0, xa = 0;
  if (tid < kThreads) {
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      c[i] = cnt[tid * kPer + i];
      sum += c[i];
      act += c[i] > 0;
      most = max(most, c[i]);
    }
    xs = sum;
    xa = act;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ys = __shfl_up_sync(0xffffffffu, xs, o), ya = __shfl_up_sync(0xffffffffu, xa, o);
      if (lane >= o) xs += ys, xa += ya;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 31) L.warp_n[w] = xs, L.warp_a[w] = xa, L.warp_most[w] = most;
  }
  __syncthreads();
  if (tid < kThreads) {
    xs -= sum;
    xa -= act;
#pragma unroll
    for (int q = 0; q < kThreads / 32; q++)
      if (q < w) xs += L.warp_n[q], xa += L.warp_a[q];
#pragma unroll
    for (int i = 0; i < kPer; i++) {
      cnt[tid * kPer + i] = xs;
      if (c[i]) {
        L.act[xa] = (uint16_t)(tid * kPer + i);
        L.off[xa++] = (uint16_t)xs;
      }
      xs += c[i];
    }
    if (tid == kThreads - 1) {
      L.n = xa;
      L.inv_m = (65536u + a.m - 1) / a.m;
      L.off[xa] = (uint16_t)xs;
      for (int q = 0; q < kThreads / 32; q++) most = max(most, L.warp_most[q]);
      L.most = most;
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kMaxTopM; q++)
    if (e[q] >= 0) {
      const int at = atomicAdd(&cnt[e[q]], 1);
      L.slot[at] = (uint16_t)(tid * a.m + q);
      L.gate[at] = gate[q];
    }
  __syncthreads();
}

// Instruction descriptor of a 128 x n product, both operands K-major.
__device__ __forceinline__ uint32_t moe_idesc(__nv_bfloat16, int n) {
  return sm100::idesc_bf16_f32(128, n, false, false);
}
__device__ __forceinline__ uint32_t moe_idesc(__half, int n) {
  return sm100::idesc_f16_f32(128, n, false, false);
}

__device__ __forceinline__ float moe_act(float x, int act) {
  if (act == GMM_ACT_GELU) {
    // x Phi(x) with the tanh form of Phi: (1 + tanh u) / 2 = 1 / (1 + e^-2u), which keeps its
    // digits where tanh u is near -1
    const float u = 0.7978845608028654f * fmaf(0.044715f * x * x, x, x);
    return x / (1.f + expf(-2.f * u));
  }
  return x / (1.f + expf(-x));
}

// One job.  Up: rows f0 .. f0 + rows of the expert's F, of which every active expert has `per`
// units of `size` rows; the units are shared out evenly, and up to 64 rows of consecutive ones
// make a job.  Down: the CTA's block of rows of y, one active expert after the other (every
// stride-th).
template <bool kDown, int kN>
struct MoeJob {
  int act, f0, rows, s0, ntok;
  int unit, end, per, size;  // up
  int stride;                // down: CTAs of the cluster

  __device__ __forceinline__ bool more(const MoeLists& L) const {
    if constexpr (kDown) return act < L.n;
    return unit < end;
  }
  __device__ __forceinline__ void tokens(const MoeLists& L) {
    ntok = min(kN, L.off[act + 1] - s0);
  }
  __device__ __forceinline__ void fit(const MoeArgs& a, const MoeLists& L) {
    if constexpr (!kDown) {
      act = unit / per;
      f0 = (unit - act * per) * size;
      rows = min(min(64, a.F - f0), (end - unit) * size);
    }
    s0 = L.off[act];
    tokens(L);
  }
  __device__ __forceinline__ void next(const MoeArgs& a, const MoeLists& L) {
    s0 += kN;
    if (s0 < L.off[act + 1]) return tokens(L);
    if constexpr (kDown)
      act += stride;
    else
      unit += (rows + size - 1) / size;
    if (more(L)) fit(a, L);
  }
};

struct MoeBarriers {
  uint64_t full[16], empty[16];  // per stage
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drained;
  unsigned int abort;  // a wait of this CTA gave up
  uint32_t tmem;
};

// Shared memory: the two structs, the lists; up: 2 x 128 x 33 floats, down: T x block_rows floats;
// the stages on a 1024-byte boundary.
constexpr int kMoeStructs =
    (int)((sizeof(MoeLists) + 255) / 256 * 256 + (sizeof(MoeBarriers) + 255) / 256 * 256);
__host__ __device__ constexpr int moe_fixed(int E, int slots) {
  return kMoeStructs + moe_list_bytes(E, slots);
}
constexpr int kMoeSwap = 2 * kMoeTile * 33 * 4;
// Of a stage: `rows` weight rows and the tokens.
__host__ __device__ constexpr int moe_stage_bytes(bool down, int kN, int rows) {
  return rows * 128 + (down ? 2 : 1) * kN * 128;
}

// Bounded wait on a phase, as mbar_wait_bounded, for waits on the path of every stage: the
// clock is read only after some tries (reading it takes longer than most waits).  kSleep:
// nanoseconds between tries, for waits whose polling would slow down the others'.
template <int kSleep = 0>
__device__ __forceinline__ bool moe_wait(uint64_t* bar, uint32_t parity,
                                         volatile unsigned int* abort, uint64_t budget_ns) {
  uint64_t t0 = 0;
  const uint32_t tries = budget_ns < 100000 ? 0 : 31;  // between looks at the clock
  for (uint32_t i = 0;; i++) {
    if (sm100::mbar_try_wait(bar, parity)) return true;
    if ((i & tries) == tries) {
      if (*abort & GMM_DEVFLAG_WAIT_TIMEOUT) return false;
      const uint64_t now = sm100::globaltimer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > budget_ns) {
        atomicOr(const_cast<unsigned int*>(abort), GMM_DEVFLAG_WAIT_TIMEOUT);
        return false;
      }
    }
    if (kSleep) __nanosleep(kSleep);
  }
}
// The same by a warp's first lane for the warp.
template <int kSleep = 0>
__device__ __forceinline__ bool moe_warp_wait(uint64_t* bar, uint32_t parity,
                                              volatile unsigned int* abort, uint64_t budget_ns) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = moe_wait<kSleep>(bar, parity, abort, budget_ns);
  ok = __shfl_sync(0xffffffffu, ok, 0);
  // every lane sees the phase itself, for the order of what it reads next
  return ok && (sm100::mbar_try_wait(bar, parity) || moe_wait(bar, parity, abort, budget_ns));
}

// (A product reads a whole tile from a stage's start on, of a small last stage past its end.)
__host__ __device__ constexpr int moe_stages(int ring_bytes, bool down, int kN, int rows) {
  const int bytes = moe_stage_bytes(down, kN, rows), past = kMoeTile * 128 - bytes;
  const int s = (ring_bytes - (past > 0 ? past : 0)) / bytes / kMoeCopyWarps * kMoeCopyWarps;
  return s < 16 ? s : 16;
}
static_assert(kMoeCopyWarps % kMoeMmaWarps == 0, "a stage has one warp of each kind");
// Columns of a job's product: more where an expert has more tokens, unless that costs stages.
__device__ __forceinline__ int moe_columns(int ring_bytes, bool down, int rows, int most) {
  int n = 16;
  for (int wide = 32; wide <= (down ? 32 : 64); wide *= 2)
    if (most > wide / 2 &&
        moe_stages(ring_bytes, down, wide, rows) >= moe_stages(ring_bytes, down, n, rows))
      n = wide;
  return n;
}

// Four rows of a matrix (a tensor map with a box of one row) at column k, one below the other.
__device__ __forceinline__ void tma_gather4(void* dst, const CUtensorMap* map, int k, int4 rows,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(sm100::smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(k), "r"(rows.x), "r"(rows.y), "r"(rows.z),
      "r"(rows.w), "r"(sm100::smem_u32(bar))
      : "memory");
}

// Rows [row, row + rows) of a weight matrix at column k: boxes of 64 and of 16 rows.
__device__ __forceinline__ void moe_load_rows(char* dst, const CUtensorMap* tm64,
                                              const CUtensorMap* tm16, int k, int row, int rows,
                                              uint64_t* bar) {
  int r = 0;
  for (; r + 64 <= rows; r += 64) sm100::tma_load_2d(dst + r * 128, tm64, k, row + r, bar);
  for (; r < rows; r += 16) sm100::tma_load_2d(dst + r * 128, tm16, k, row + r, bar);
}
__device__ __forceinline__ int moe_box_rows(int rows) { return (rows + 15) / 16 * 16; }

template <typename T, bool kDown, int kN>
__device__ __forceinline__ void moe_stream(const MoeArgs& a, const MoeLists& L, MoeBarriers& bar,
                                           MoeJob<kDown, kN> job, char* ring, float* side,
                                           const CUtensorMap* tm64, const CUtensorMap* tm16,
                                           const CUtensorMap* tok) {
  using namespace sm100;
  constexpr int kH = kDown ? 2 : 1;  // halves of a token: x, or h hi and lo
  const int tile = kDown ? a.block_rows : kMoeTile;  // weight rows that a stage has room for
  const int stage_bytes = moe_stage_bytes(kDown, kN, tile);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int K = kDown ? a.F : a.D, steps = (K + kMoeK - 1) / kMoeK;
  // Stages: a multiple of the warps that take them in turn, so that a stage always belongs to
  // the same copying and the same multiplying warp.  (A wait on a phase by its parity means that
  // phase only while the phase before is known to be over.)
  const int S = moe_stages(a.ring_bytes, kDown, kN, tile);
  volatile unsigned int* abort = &bar.abort;
  auto wait = [&](uint64_t* b, uint32_t parity) {
    return moe_wait(b, parity, abort, a.wait_ns);
  };
  // Step s of the stream uses stage s % S for the (s / S)-th time.  A warp takes every kTurns-th
  // step; `at` is its next one.
  int at = 0, stage = 0;
  uint32_t parity = 0;
  auto advance = [&](int turns) {
    at += turns;
    for (stage += turns; stage >= S; stage -= S) parity ^= 1u;
  };

  if (w >= 4 && w < 4 + kMoeCopyWarps) {
    // ---- copies: lane 0 the weights, lane l token rows 4 l .. (down: the hi, then the lo rows)
    static_assert(kH * kN / 4 <= 32, "a lane for four token rows");
    bool ok = true;
    int4 from;  // lane l's rows 4 l .. of the stage, of them kN / 4 lanes for each half
    bool mine4 = false;
    auto aim = [&](const MoeJob<kDown, kN>& j) {
      const int col = lane * 4 % kN;
      mine4 = lane * 4 < kH * kN && col < j.ntok;
      int r[4];
#pragma unroll
      for (int i = 0; i < 4; i++) {  // (past the last token: the last again)
        const int slot = L.slot[j.s0 + min(col + i, j.ntok - 1)];
        r[i] = kDown ? slot + (lane * 4 < kN ? 0 : a.T * a.m) : L.token(slot);  // lo behind hi
      }
      from = make_int4(r[0], r[1], r[2], r[3]);
    };
    auto weights = [&](const MoeJob<kDown, kN>& j, int c) {  // by lane 0
      const uint32_t bytes = (uint32_t)((kDown ? tile : 2 * moe_box_rows(j.rows)) +
                                        (j.ntok + 3) / 4 * 4 * kH) * 128u;
      const int e = L.act[j.act];
      const int row = kDown ? e * a.D + j.f0 : e * 2 * a.F + j.f0;
      char* dst = ring + stage * stage_bytes;
      mbar_arrive_expect_tx(&bar.full[stage], bytes);
      if (kDown) {  // (the box is the block; of the last one it may reach past the expert)
        tma_load_2d(dst, tm64, c * kMoeK, row, &bar.full[stage]);
      } else {
        moe_load_rows(dst, tm64, tm16, c * kMoeK, row, j.rows, &bar.full[stage]);
        moe_load_rows(dst + 64 * 128, tm64, tm16, c * kMoeK, row + a.F, j.rows, &bar.full[stage]);
      }
    };
    auto tokens = [&](int c) {
      if (mine4)
        tma_gather4(ring + stage * stage_bytes + tile * 128 + lane * 512, tok, c * kMoeK, from,
                    &bar.full[stage]);
    };
    // Down: the weights of the first steps do not depend on the kernel before, h does.
    int early = 0;
    if (kDown) {
      MoeJob<kDown, kN> j = job;
      int base = 0;
      advance(w - 4);
      for (; at < S && j.more(L); j.next(a, L), base += steps)
        for (; at < S && at < base + steps; advance(kMoeCopyWarps))
          if (lane == 0) weights(j, at - base);
      early = at;
      at = stage = 0;
      parity = 0;
      asm volatile("griddepcontrol.wait;" ::: "memory");
    }
    int base = 0, mine = 0;  // first step of the job; steps of this warp so far
    advance(w - 4);
    for (; ok && job.more(L); job.next(a, L), base += steps) {
      aim(job);
      for (; at < base + steps; advance(kMoeCopyWarps)) {
        ok = __all_sync(0xffffffffu,
                        moe_warp_wait(&bar.empty[stage], parity ^ 1u, abort, a.wait_ns));
        if (!ok) break;
        if (lane == 0 && at >= early) weights(job, at - base);
        __syncwarp();
        tokens(at - base);
        mine++;
      }
    }
    // What is on its way has to land before the CTA ends, also when it was another warp whose wait
    // gave up: the last step of each of this warp's stages.  (A wait of its own that gave up is
    // for a step beyond the first S, and so beyond the early ones.)
    if (lane == 0)
      for (int left = min(mine, S / kMoeCopyWarps); left > 0; left--) {
        at -= kMoeCopyWarps;
        mbar_wait_bounded(&bar.full[at % S], (uint32_t)(at / S) & 1u, abort, 0u, kMoeDrainNs);
      }
  } else if (w >= 4 + kMoeCopyWarps) {
    // ---- products
    if (lane == 0) {
      const int turn = w - 4 - kMoeCopyWarps;
      bool ok = true;
      uint32_t n = 0;  // jobs so far
      int base = 0;
      const uint32_t idesc = moe_idesc(T(), kH * kN);
      static_assert(kH * kN <= kMoeAccCols, "accumulator columns");
      const uint64_t a0 = sw128_desc(smem_u32(ring), 16, 1024);
      const uint64_t b0 = sw128_desc(smem_u32(ring) + tile * 128, 16, 1024);
      advance(turn);
      for (; ok && job.more(L); job.next(a, L), base += steps, n++) {
        // the accumulator goes by the step within the job, so that a sum's parts do not depend
        // on the jobs before
        const uint32_t buf = n & 1u, part = (uint32_t)(turn - base) % kMoeMmaWarps;
        const uint32_t acc = bar.tmem + (buf * kMoeMmaWarps + part) * kMoeAccCols;
        if (!(ok = wait(&bar.acc_empty[buf], ((n >> 1) & 1u) ^ 1u))) break;
        tc_fence_after_sync();
        bool more = false;  // the accumulator holds something
        for (; at < base + steps; advance(kMoeMmaWarps)) {
          if (!(ok = wait(&bar.full[stage], parity))) break;
          tc_fence_after_sync();
          const uint64_t off = (uint64_t)((uint32_t)(stage * stage_bytes) >> 4);
#pragma unroll
          for (int ks = 0; ks < kMoeK / 16; ks++)
            mma_bf16(acc, a0 + off + 2 * ks, b0 + off + 2 * ks, idesc, more || ks > 0);
          more = true;
          mma_commit(&bar.empty[stage]);
        }
        if (ok) mma_commit(&bar.acc_full[buf]);
      }
      // tensor memory is given back when every product is done
      mma_commit(&bar.drained);
      mbar_wait_bounded(&bar.drained, 0, abort, 0u, kMoeDrainNs);
    }
  } else if (w < 4) {
    // ---- out of tensor memory: thread t has weight row t of the tile
    uint32_t n = 0;
    int swap = 0;
    bool ok = true;
    const uint32_t lanes = (uint32_t)(w * 32) << 16;
    for (; job.more(L); job.next(a, L), n++) {  // to the end even when a wait gave up (what it
      const uint32_t buf = n & 1u;              // was for is NaN then): the warps meet at barriers
      ok = ok && moe_warp_wait<100>(&bar.acc_full[buf], (n >> 1) & 1u, abort, a.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after_sync();
      for (int j0 = 0; j0 < job.ntok; j0 += 32) {
        const int cnt = min(32, job.ntok - j0);
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; j++) v[j] = ok ? 0.f : __int_as_float(0x7fffffff);
        if (ok) {
          // the warps' shares of K (a job of few steps has not all of them), in order
#pragma unroll 1
          for (int i = 0; i < min(steps, kMoeMmaWarps); i++) {
            const uint32_t at = bar.tmem + lanes + (buf * kMoeMmaWarps + i) * kMoeAccCols;
            float u[32];
            tmem_ld32(at + (uint32_t)j0, u);
#pragma unroll
            for (int j = 0; j < 32; j++) v[j] += u[j];
            if constexpr (kDown && kN == 16) {  // lo beside hi
#pragma unroll
              for (int j = 0; j < 16; j++) v[j] = fmaf(u[j + 16], 1.f / kMoeLo<T>, v[j]);
            } else if constexpr (kDown) {
              tmem_ld32(at + (uint32_t)kN, u);
#pragma unroll
              for (int j = 0; j < 32; j++) v[j] = fmaf(u[j], 1.f / kMoeLo<T>, v[j]);
            }
          }
        }
        if constexpr (kDown) {
          if (tid < job.rows) {
#pragma unroll
            for (int j = 0; j < (kN < 32 ? kN : 32); j++)
              if (j < cnt) {
                const int s = job.s0 + j0 + j;
                float* at = side + L.token(L.slot[s]) * tile + tid;
                *at = fmaf(L.gate[s], v[j], *at);
              }
          }
        } else {
          // Rows 64.. are the linear half of rows 0..  Two threads share a row's columns, in a
          // loop (unrolled over the columns the code is so long that fetching it costs 8 us).
          float* x = side + swap * kMoeTile * 33 + tid * 33;
#pragma unroll
          for (int j = 0; j < 32; j++) x[j] = v[j];
          asm volatile("bar.sync 1, 128;" ::: "memory");
          const int row = tid & 63;
          const float* gate = side + swap * kMoeTile * 33 + row * 33;
          swap ^= 1;
          if (row < job.rows) {
#pragma unroll 1
            for (int j = tid >> 6; j < cnt; j += 2) {
              const float h = moe_act(gate[j], a.act) * gate[64 * 33 + j];
              const int64_t at = (int64_t)L.slot[job.s0 + j0 + j] * a.F + job.f0 + row;
              T hi, lo;
              from_f32(&hi, h);
              const float left = (h - to_f32(hi)) * kMoeLo<T>;
              from_f32(&lo, isfinite(left) ? left : 0.f);  // h beyond the type's range stays so
              ((T*)a.h_hi)[at] = hi;
              ((T*)a.h_lo)[at] = lo;
            }
          }
        }
      }
      tc_fence_before_sync();
      mbar_arrive(&bar.acc_empty[buf]);
    }
  }
  __syncwarp();
}

// Start of both kernels: barriers, tensor memory.
__device__ __forceinline__ void moe_begin(MoeBarriers& bar) {
  using namespace sm100;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 16; i++) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; i++) {
      mbar_init(&bar.acc_full[i], kMoeMmaWarps);
      mbar_init(&bar.acc_empty[i], 128);
    }
    mbar_init(&bar.drained, kMoeMmaWarps);
    bar.abort = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < 32) {
    tmem_alloc(&bar.tmem, kMoeTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
}
// And their end.
__device__ __forceinline__ void moe_end(const MoeArgs& a, MoeBarriers& bar) {
  sm100::tc_fence_before_sync();
  __syncthreads();
  sm100::tc_fence_after_sync();
  if (threadIdx.x < 32) sm100::tmem_dealloc(bar.tmem, kMoeTmemCols);
  if (threadIdx.x == 0 && bar.abort) atomicOr(a.status, GMM_DEVFLAG_WAIT_TIMEOUT);
}

__device__ __forceinline__ char* align1024(char* p) {
  return (char*)(((uintptr_t)p + 1023) & ~(uintptr_t)1023);
}

template <typename T, int kN>
__device__ __forceinline__ void moe_up_run(const MoeArgs& a, MoeLists& L, MoeBarriers& bar,
                                           char* ring, float* side, const CUtensorMap* tm64,
                                           const CUtensorMap* tm16, const CUtensorMap* tok) {
  MoeJob<false, kN> job;
  // Units of 64 rows, or of 32 or 16 where they share out so much better that it makes up for
  // their steps, which take 0.6 and 0.45 of a full one's time.
  int64_t all = 0;
  float best = 0.f;
  for (int size = 64; size >= 16; size /= 2) {
    const int per = (a.F + size - 1) / size;
    const int64_t units = (int64_t)L.n * per;
    const float cost = (float)((units + gridDim.x - 1) / gridDim.x) *
                       (size == 64 ? 1.f : size == 32 ? 0.6f : 0.45f);
    if (size == 64 || cost < best) {
      best = cost;
      all = units;
      job.size = size;
      job.per = per;
    }
  }
  job.unit = (int)(all * blockIdx.x / gridDim.x);
  job.end = (int)(all * (blockIdx.x + 1) / gridDim.x);
  if (job.more(L)) job.fit(a, L);
  moe_stream<T, false, kN>(a, L, bar, job, ring, side, tm64, tm16, tok);
}

template <typename T>
__global__ void __launch_bounds__(kMoeThreads, 1)
    moe_up_kernel(MoeArgs a, const __grid_constant__ CUtensorMap tm64,
                  const __grid_constant__ CUtensorMap tm16,
                  const __grid_constant__ CUtensorMap tok) {
  extern __shared__ __align__(256) char smem[];
  MoeLists& L = *(MoeLists*)smem;
  MoeBarriers& bar = *(MoeBarriers*)(smem + (sizeof(MoeLists) + 255) / 256 * 256);
  const int fixed = moe_fixed(a.E, a.T * a.m);
  float* side = (float*)(smem + fixed);
  char* ring = align1024(smem + fixed + kMoeSwap);
  if (threadIdx.x == 0) moe_place_lists(L, smem + kMoeStructs, a.E, a.T * a.m);
  moe_begin(bar);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.T * a.m; i += kMoeThreads) {
      const int e = __ldcg(a.idx + i);
      if (e < -1 || e >= a.E) atomicOr(a.status, GMM_DEVFLAG_BAD_INDEX);
    }
  moe_sort(a, L, (int*)side);
  const int columns = moe_columns(a.ring_bytes, false, kMoeTile, L.most);
  if (columns == 16)
    moe_up_run<T, 16>(a, L, bar, ring, side, &tm64, &tm16, &tok);
  else if (columns == 32)
    moe_up_run<T, 32>(a, L, bar, ring, side, &tm64, &tm16, &tok);
  else
    moe_up_run<T, 64>(a, L, bar, ring, side, &tm64, &tm16, &tok);
  moe_end(a, bar);
}

template <typename T, int kN>
__device__ __forceinline__ void moe_down_run(const MoeArgs& a, MoeLists& L, MoeBarriers& bar,
                                             char* ring, float* y, int d0, int rows, int rank,
                                             int C, const CUtensorMap* weights,
                                             const CUtensorMap* h) {
  MoeJob<true, kN> job;
  job.f0 = d0;
  job.rows = rows;
  job.act = rank;
  job.stride = C;
  if (job.more(L)) job.fit(a, L);
  moe_stream<T, true, kN>(a, L, bar, job, ring, y, weights, weights, h);
}

template <typename T>
__global__ void __launch_bounds__(kMoeThreads, 1)
    moe_down_kernel(MoeArgs a, int C, const __grid_constant__ CUtensorMap weights,
                    const __grid_constant__ CUtensorMap h) {
  extern __shared__ __align__(256) char smem[];
  MoeLists& L = *(MoeLists*)smem;
  MoeBarriers& bar = *(MoeBarriers*)(smem + (sizeof(MoeLists) + 255) / 256 * 256);
  const int tid = threadIdx.x, per = a.T * a.block_rows;
  const int fixed = moe_fixed(a.E, a.T * a.m);
  float* y = (float*)(smem + fixed);  // [token][row of the block]
  char* ring = align1024(smem + fixed + per * 4);
  const int rank = C > 1 ? (int)sm100::cluster_ctarank() : 0;
  const int d0 = (int)(blockIdx.x / C) * a.block_rows, rows = min(a.block_rows, a.D - d0);
  if (tid == 0) moe_place_lists(L, smem + kMoeStructs, a.E, a.T * a.m);
  moe_begin(bar);
  // (idx and resp were complete before the up kernel let this one start)
  moe_sort(a, L, (int*)ring);
  for (int i = tid; i < per; i += kMoeThreads) y[i] = 0.f;
  sm100::fence_proxy_async_smem();  // the sort's counters lay where TMA writes
  __syncthreads();
  if (moe_columns(a.ring_bytes, true, a.block_rows, L.most) == 16)
    moe_down_run<T, 16>(a, L, bar, ring, y, d0, rows, rank, C, &weights, &h);
  else
    moe_down_run<T, 32>(a, L, bar, ring, y, d0, rows, rank, C, &weights, &h);
  asm volatile("griddepcontrol.wait;" ::: "memory");  // before Y is written
  moe_end(a, bar);
  if (C > 1) sm100::cluster_sync();
  T* Y = (T*)a.Y;
  for (int i = tid; i < per; i += kMoeThreads) {
    const int tok = i / a.block_rows, row = i - tok * a.block_rows;
    if (tok % C != rank || row >= rows) continue;
    float v = y[i];
    if (C > 1) {  // the cluster's copies, in CTA order
      v = 0.f;
      const uint32_t at = sm100::smem_u32(y + i);
      for (int q = 0; q < C; q++) {
        float x;
        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                     : "=f"(x)
                     : "r"(sm100::map_to_rank(at, q))
                     : "memory");
        v += x;
      }
    }
    from_f32(Y + (int64_t)tok * a.ldy + d0 + row, v);
  }
  if (C > 1) sm100::cluster_sync();  // the others' shared memory has been read
}

}  // namespace scem
