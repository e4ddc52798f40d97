// beam.cuh -- kernels of gmm_beam_select and gmm_beam_reorder.
//
// A group of w beams, rows b w .. b w + w - 1 of the logits, has the candidates (i, k) of score
//   scores_i + log p_i(k),
// and its m best are among the m best classes of each row, which row_short_kernel or
// row_long_kernel finds while the logits go through once.  What is left is a merge of w sorted
// lists.  64 groups of 8 beams over 100,003 fp32, partly masked, m = 16: 58 us (31 us of bytes at
// the rate of a large copy), 52 of them the rows' and 6 the merge's; over 131,072 bf16 47 us
// (20).  One group of 4 beams over those: 14 us, both kernels' latency.
#pragma once

#include "rows.cuh"

namespace scem {

constexpr int kMostBeams = 32;  // a lane for each

struct BeamArgs {
  const void* Z;
  int64_t ld;
  float scale;
  int64_t B;
  int w, m;
  const float* scores;     // B x w
  const uint8_t* ended;    // B x w, may be null
  int end_id;
  const int32_t* top_idx;  // B w x m: each row's best classes, and their log p
  const float* top_logp;
  float* out;              // B x m
  int32_t *parent, *token;
  uint32_t* flags;
};

// Doubles as unsigned integers of the same order; 0 for -inf.
__device__ __forceinline__ uint64_t double_order(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
  return v == -INFINITY ? 0ull
                        : b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double order_double(uint64_t o) {
  return o == 0 ? -INFINITY
                : __longlong_as_double((long long)(o >> 63 ? o ^ 0x8000000000000000ull : ~o));
}

// A CTA per group: its threads form the candidates' scores, a warp with a lane per beam merges
// them. Scores are 64 bits wide: those of different rows lie close together, and in 32 bits a log
// p of -15 is rounded by 5e-7.  A row's first log p is the smallest in size and so the most exact
// one (1.6e-6 off at most in 256 rows of 262,144 each, of several widths; 2e-7 in rows of 50); the
// others stand as far behind it as their logits.  Equal scores go to the lower beam,
// then in the order of the row: of z = fl32(scale x), then of the class.  That is the order of the
// scores too, but for logits that the scale rounds to one z.
constexpr int kMergeThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(BeamArgs a) {
  __shared__ uint64_t cand[2 * kMostBeams * kMaxAlt];  // [beam][m], then the same by score
  __shared__ uint8_t place[kMostBeams * kMaxAlt];      // where those stood
  const int t = threadIdx.x, lane = t & 31;
  const int64_t b = blockIdx.x;
  grid_dependency_wait();
  grid_dependents_launch();
  float score = -INFINITY;
  bool ended = false;
  if (lane < a.w) {
    score = a.scores[b * a.w + lane];
    ended = a.ended && a.ended[b * a.w + lane];
  }
  const float first = lane < a.w ? a.top_logp[(b * a.w + lane) * a.m] : 0.f;
  bool climbs = false;  // a candidate scores more than the one before it in its row's order
  for (int c0 = 0; c0 < a.w * a.m; c0 += kMergeThreads) {
    const int c = c0 + t, i = min(c / a.m, a.w - 1), j = c % a.m;
    const float s = __shfl_sync(0xffffffffu, score, i);
    const float lp = __shfl_sync(0xffffffffu, first, i);
    const bool e = __shfl_sync(0xffffffffu, (int)ended, i);
    if (c >= a.w * a.m) continue;
    uint64_t key = 0;
    if (e) {
      if (j == 0) key = double_order((double)s);
    } else if (s != -INFINITY) {
      const int64_t row = b * a.w + i;
      const int k0 = a.top_idx[row * a.m], k = a.top_idx[row * a.m + j];
      const int before = a.scale != 1.f ? a.top_idx[row * a.m + max(j - 1, 0)] : k0;
      if (k >= 0) {
        const T* z = (const T*)a.Z + row * a.ld;
        const float x = to_f32(z[k]);
        climbs |= x > to_f32(z[before]) && a.scale != 1.f;
        const double d = (double)x - (double)to_f32(z[k0]);
        key = double_order((double)s + ((double)lp + d * (double)a.scale));
      }
    }
    cand[c] = key;
  }
  // Logits that the scale rounds to one z: then each beam's candidates are ranked by score first.
  const bool ranked = __syncthreads_or(climbs);
  const int list = ranked ? kMostBeams * kMaxAlt : 0;
  if (ranked) {
    for (int c = t; c < a.w * a.m; c += kMergeThreads) {
      const int from = c - c % a.m;
      const uint64_t key = cand[c];
      int rank = 0;
      for (int q = from; q < from + a.m; q++) rank += cand[q] > key || (cand[q] == key && q < c);
      cand[list + from + rank] = key;
      place[from + rank] = (uint8_t)(c - from);
    }
    __syncthreads();
  }
  if (t >= 32) return;
  const bool dead = score == -INFINITY;
  const bool bad = !(score < INFINITY) || (!dead && !ended && !(first == first));
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0 && a.flags) atomicOr(a.flags, GMM_DEVFLAG_NONFINITE_X);
    if (lane < a.m) {
      a.out[b * a.m + lane] = __int_as_float(0x7fffffff);
      a.parent[b * a.m + lane] = -1;
      a.token[b * a.m + lane] = -1;
    }
    return;
  }
  int pos = 0, my_parent = -1, my_rank = 0;
  double my_score = -INFINITY;
  uint64_t head = lane < a.w ? cand[list + lane * a.m] : 0;
  for (int j = 0; j < a.m; j++) {
    const uint64_t best = warp_max_key(head);
    if (best == 0) break;
    const int from = __ffs(__ballot_sync(0xffffffffu, head == best)) - 1;
    const int rank = __shfl_sync(0xffffffffu, pos, from);
    if (lane == j) {
      my_score = order_double(best);
      my_parent = from;
      my_rank = rank;
    }
    if (lane == from) head = ++pos < a.m ? cand[list + lane * a.m + pos] : 0;
  }
  if (ranked && my_parent >= 0) my_rank = place[my_parent * a.m + my_rank];
  const bool end = __shfl_sync(0xffffffffu, (int)ended, max(my_parent, 0));
  if (lane < a.m) {
    a.out[b * a.m + lane] = (float)my_score;
    a.parent[b * a.m + lane] = my_parent;
    a.token[b * a.m + lane] = my_parent < 0 ? -1
                              : end         ? a.end_id
                                            : a.top_idx[(b * a.w + my_parent) * a.m + my_rank];
  }
}

// ------------------------------------------------------------------ states after their parents
// In place: a thread owns a column of a group, the same few bytes of all its beams, and has read
// every beam's source before it writes any.  Beams that stay where they are are neither read
// (unless another wants them) nor written.
//
// Bound by memory.  16 groups of 8 beams, four caches of 8 x 1,024 x 128 bf16, 300 to 1,024
// positions used: 191 to 209 us, 5.2 TB/s (157 us at the rate of a large copy; reads and writes
// take turns on 16 streams per block).  2 groups of 32: 324 us (258).  16 of 4: 151 (125).
struct BeamState {
  char* base;
  int64_t row_stride, outer_stride;  // bytes
};

constexpr int kStates = 64;  // of one launch
constexpr int kReorderThreads = 256;
constexpr int kReorderGroups = 1024;  // looked at in one go

// States of one shape.
struct ReorderArgs {
  BeamState state[kStates];
  const int32_t* parent;  // B x w
  const int32_t* lens;    // B, or null: all positions are used
  int64_t B;
  int n, w;
  uint32_t outer, inner, per_pos;  // pieces of a row; columns of a piece and of a position
  uint32_t* flags;
};

// Columns of a thread in a tile, and CTAs per SM: all of a launch are resident at once.  (16 groups
// of 4 beams take 149 us with four columns and two CTAs, 175 with two and three; groups of 8 193 us
// with one column and three CTAs, 200 with two and two.)
constexpr int reorder_cols(int w) { return w <= 4 ? 4 : 1; }
constexpr int reorder_ctas(int w) { return w <= 2 ? 3 : w <= 4 ? 2 : w <= 8 ? 3 : w <= 16 ? 2 : 1; }

// kW: at least w.  The blocks share out tiles of columns: of the groups in which a beam moves, up
// to their lengths, for every state.
template <typename Vec, int kW>
__global__ void __launch_bounds__(kReorderThreads, reorder_ctas(kW))
    beam_reorder_kernel(ReorderArgs a) {
  __shared__ uint32_t upto[kReorderGroups];  // tiles of the groups up to and with this one
  __shared__ uint32_t warp_total[kReorderThreads / 32];
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  grid_dependency_wait();
  grid_dependents_launch();
  constexpr int kEach = kReorderGroups / kReorderThreads, kCols = reorder_cols(kW);
  constexpr int kTile = kCols * kReorderThreads;
  const int positions = (int)(a.inner / a.per_pos);
  auto length = [&](int64_t b) {  // columns of a piece that are used
    return a.lens ? (uint32_t)max(0, min(a.lens[b], positions)) * a.per_pos : a.inner;
  };
  for (int64_t b0 = 0; b0 < a.B; b0 += kReorderGroups) {
    uint32_t tiles_to[kEach], total = 0;
#pragma unroll
    for (int q = 0; q < kEach; q++) {
      const int64_t b = b0 + t * kEach + q;
      uint32_t tiles = 0;
      if (b < a.B) {
        bool moves = false;
        for (int i = 0; i < a.w; i++) {
          const int p = a.parent[b * a.w + i];
          if ((unsigned)p < (unsigned)a.w) moves |= p != i;
          else if (p != -1 && a.flags) atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
        }
        if (a.lens && a.flags && (unsigned)a.lens[b] > (unsigned)positions)
          atomicOr(a.flags, GMM_DEVFLAG_BAD_INDEX);
        if (moves)
          tiles = (uint32_t)(((uint64_t)a.outer * length(b) + kTile - 1) / kTile);
      }
      total += tiles;
      tiles_to[q] = total;
    }
    uint32_t scan = total;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) warp_total[w] = scan;
    __syncthreads();
    uint32_t before = scan - total;
    for (int q = 0; q < w; q++) before += warp_total[q];
#pragma unroll
    for (int q = 0; q < kEach; q++) upto[t * kEach + q] = before + tiles_to[q];
    __syncthreads();
    // this block's share: consecutive tiles, so that it seldom comes to another group
    const uint64_t all = upto[kReorderGroups - 1], every = all * a.n;
    uint64_t tile = every * blockIdx.x / gridDim.x;
    const uint64_t stop = every * (blockIdx.x + 1) / gridDim.x;
    int state = -1, group = 0;
    uint32_t here = 0, first = 0, upper = 0;  // the tile in its state; those of its group
    uint32_t len = 0, moved = 0;
    int mine = 0;
    int64_t b = 0;
    for (; tile < stop; tile++, here++) {
      if (state < 0 || here >= upper) {  // (the same for all threads)
        if (state < 0 || here >= all) {
          state = (int)(tile / all);
          here = (uint32_t)(tile - state * all);
          group = 0;
          int hi = kReorderGroups - 1;  // the first group with upto > here
          while (group < hi) {
            const int mid = (group + hi) / 2;
            if (upto[mid] > here) hi = mid;
            else group = mid + 1;
          }
        } else {
          do group++;
          while (upto[group] <= here);
        }
        first = group ? upto[group - 1] : 0;
        upper = upto[group];
        b = b0 + group;
        len = length(b);
        mine = lane < a.w ? a.parent[b * a.w + lane] : -1;  // a parent per lane
        moved = __ballot_sync(0xffffffffu, (unsigned)mine < (unsigned)a.w && mine != lane);
      }
      const int64_t stride = a.state[state].row_stride;
      char* p[kCols];
      bool in[kCols];
      Vec v[kCols][kW];
#pragma unroll
      for (int q = 0; q < kCols; q++) {
        const uint64_t c = (uint64_t)(here - first) * kTile + q * kReorderThreads + t;
        in[q] = c < (uint64_t)a.outer * len;
        const uint32_t o = in[q] ? (uint32_t)c / len : 0;  // (below 2^32: checked on the host)
        p[q] = a.state[state].base + b * a.w * stride + o * a.state[state].outer_stride +
               ((uint64_t)c - (uint64_t)o * len) * sizeof(Vec);
      }
#pragma unroll
      for (int i = 0; i < kW; i++) {
        const int from = __shfl_sync(0xffffffffu, mine, i);
#pragma unroll
        for (int q = 0; q < kCols; q++)
          if (in[q] && (moved >> i & 1))
            v[q][i] = *reinterpret_cast<const Vec*>(p[q] + from * stride);
      }
#pragma unroll
      for (int i = 0; i < kW; i++) {
#pragma unroll
        for (int q = 0; q < kCols; q++)
          if (in[q] && (moved >> i & 1)) *reinterpret_cast<Vec*>(p[q] + i * stride) = v[q][i];
      }
    }
    __syncthreads();
  }
}

}  // namespace scem
