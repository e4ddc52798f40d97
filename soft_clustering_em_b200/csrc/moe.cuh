// moe.cuh -- a mixture-of-experts layer for a few tokens: kernels of gmm_moe.
//
// Token t goes to the experts idx[t][j] with weights resp[t][j] (as gmm_route or
// gmm_assign_topm return them):
//   y_t = sum_j resp_tj W_down[e] h,   h = act(W_gate[e] x_t) * (W_lin[e] x_t),  e = idx_tj
// where W_up[e] (2F x D) stacks W_gate over W_lin and W_down[e] is D x F.
//
// With few tokens the layer is bound by reading the chosen experts' weights
// (3 D F elements each) once: an expert's tokens, 8 at a time, are the columns of
// one warp-level matrix product, so every weight read is used for all of them.
// The weights go straight from global memory to the fragments of the
// m16n8k16 product: a contraction may run over its index in any order, so a
// thread takes 8 consecutive elements of a row (16 bytes) as its share of two
// k-steps, and the same 8 of its token.  There is nothing for shared memory to
// rearrange, and tensor memory with its 128-row tiles would only add latency to
// a kernel whose products take a few percent of its time.
//
// Kernel 1 (up) writes h for every (token, choice) into the workspace; kernel 2
// (down) forms y.  Both sort the T * m choices by expert in shared memory first.
// h is kept as two halves of the weights' type, hi + lo, so that rounding it
// adds nothing visible to y.
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
constexpr int kMoeThreads = 256;
constexpr int kMoeWarps = kMoeThreads / 32;
constexpr int kMoeRows = 16;  // weight rows per tile

struct MoeArgs {
  const void *X, *W_up, *W_down;
  void* Y;
  const int32_t* idx;
  const float* resp;
  void *h_hi, *h_lo;  // T * m x F
  int T, m, E, D, F;
  int64_t ldx, ldy;
  int act;
  int row_blocks;  // down: blocks of rows of y
  unsigned int* status;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1, __nv_bfloat16) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1, __half) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Both k-steps of 8 elements per thread: rows g (lo) and g + 8 (hi) of the
// weights against column g of the tokens.
template <typename T>
__device__ __forceinline__ void mma_k32(float (&c)[4], const uint4& lo, const uint4& hi,
                                        const uint4& b) {
  mma_16816(c, lo.x, hi.x, lo.y, hi.y, b.x, b.y, T());
  mma_16816(c, lo.z, hi.z, lo.w, hi.w, b.z, b.w, T());
}

__device__ __forceinline__ uint4 zero16() { return make_uint4(0, 0, 0, 0); }

// The T * m choices sorted by expert: active experts a = 0..n-1 in ascending
// order, act[a] the expert, its choices slot[off[a] .. off[a+1]).  A choice that
// repeats an expert within its token is left out; its weight counts with the
// first one.  The order inside an expert is free: it only decides the column of
// a product.
struct MoeLists {
  int cnt[kMoeMaxE];
  uint16_t act[kMoeMaxE];
  uint16_t off[kMoeMaxE + 1];
  uint16_t slot[kMoeMaxSlots];
  int warp_n[kMoeWarps], warp_a[kMoeWarps];
  int n;
};

// The expert of choice i, or -1: unused, out of range, or repeated.
__device__ __forceinline__ int moe_expert(const MoeArgs& a, int i) {
  const int e = a.idx[i];
  if (e < 0 || e >= a.E) return -1;
  for (int q = i - i % a.m; q < i; q++)
    if (a.idx[q] == e) return -1;
  return e;
}

__device__ __forceinline__ void moe_sort(const MoeArgs& a, MoeLists& L) {
  constexpr int kPer = kMoeMaxE / kMoeThreads;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, n = a.T * a.m;
  for (int e = tid; e < kMoeMaxE; e += kMoeThreads) L.cnt[e] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += kMoeThreads) {
    const int e = moe_expert(a, i);
    if (e >= 0) atomicAdd(&L.cnt[e], 1);
  }
  __syncthreads();
  int c[kPer], sum = 0, act = 0;
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    c[i] = L.cnt[tid * kPer + i];
    sum += c[i];
    act += c[i] > 0;
  }
  int xs = sum, xa = act;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ys = __shfl_up_sync(0xffffffffu, xs, o), ya = __shfl_up_sync(0xffffffffu, xa, o);
    if (lane >= o) xs += ys, xa += ya;
  }
  if (lane == 31) L.warp_n[w] = xs, L.warp_a[w] = xa;
  __syncthreads();
  xs -= sum;
  xa -= act;
  for (int q = 0; q < w; q++) xs += L.warp_n[q], xa += L.warp_a[q];
#pragma unroll
  for (int i = 0; i < kPer; i++) {
    L.cnt[tid * kPer + i] = xs;
    if (c[i]) {
      L.act[xa] = (uint16_t)(tid * kPer + i);
      L.off[xa++] = (uint16_t)xs;
    }
    xs += c[i];
  }
  if (tid == kMoeThreads - 1) {
    L.n = xa;
    L.off[xa] = (uint16_t)xs;
  }
  __syncthreads();
  for (int i = tid; i < n; i += kMoeThreads) {
    const int e = moe_expert(a, i);
    if (e >= 0) L.slot[atomicAdd(&L.cnt[e], 1)] = (uint16_t)i;
  }
  __syncthreads();
}

__device__ __forceinline__ float moe_act(float x, int act) {
  if (act == GMM_ACT_GELU) {
    // x Phi(x) with the tanh form of Phi
    const float u = 0.7978845608028654f * fmaf(0.044715f * x * x, x, x);
    return 0.5f * x * (1.f + tanhf(u));
  }
  return x / (1.f + expf(-x));
}

// ------------------------------------------------------------------ up
// The active experts' F rows are laid end to end and cut evenly over the CTAs,
// to the row; a CTA takes its range in tiles of up to 16 rows of one expert.  The
// warps split D, so a CTA reads 512 bytes in a row of each weight row at a time.
template <typename T, int kNT, int kU>
__device__ __forceinline__ void up_product(const MoeArgs& a, const T* gate, const T* lin, int rows,
                                           const int64_t (&xoff)[kNT], float (&acc)[2][kNT][4]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const T* X = (const T*)a.X;
  const int64_t r0 = (int64_t)g * a.D, r1 = (int64_t)(g + 8) * a.D;
  const bool ok0 = g < rows, ok1 = g + 8 < rows;
  for (int k0 = w * 32 + t * 8; k0 < a.D + t * 8; k0 += kMoeWarps * 32 * kU) {
    uint4 A[kU][4], B[kU][kNT];
#pragma unroll
    for (int u = 0; u < kU; u++) {
      const int k = k0 + u * kMoeWarps * 32;
      const bool in = k < a.D;
      A[u][0] = in && ok0 ? __ldg((const uint4*)(gate + r0 + k)) : zero16();
      A[u][1] = in && ok1 ? __ldg((const uint4*)(gate + r1 + k)) : zero16();
      A[u][2] = in && ok0 ? __ldg((const uint4*)(lin + r0 + k)) : zero16();
      A[u][3] = in && ok1 ? __ldg((const uint4*)(lin + r1 + k)) : zero16();
#pragma unroll
      for (int q = 0; q < kNT; q++)
        B[u][q] = in && xoff[q] >= 0 ? load16(X + xoff[q] + k) : zero16();
    }
#pragma unroll
    for (int u = 0; u < kU; u++)
#pragma unroll
      for (int q = 0; q < kNT; q++) {
        mma_k32<T>(acc[0][q], A[u][0], A[u][1], B[u][q]);
        mma_k32<T>(acc[1][q], A[u][2], A[u][3], B[u][q]);
      }
  }
}

template <typename T, int kNT, int kU>
__device__ __forceinline__ void up_tile(const MoeArgs& a, int e, int f0, int rows,
                                        const uint16_t* slot, int ntok, float* red) {
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, g = lane >> 2;
  const T* gate = (const T*)a.W_up + ((int64_t)e * 2 * a.F + f0) * a.D;
  const T* lin = gate + (int64_t)a.F * a.D;
  int64_t xoff[kNT];
#pragma unroll
  for (int q = 0; q < kNT; q++) {
    const int col = q * 8 + g;
    xoff[q] = col < ntok ? (int64_t)(slot[col] / a.m) * a.ldx : -1;
  }
  float acc[2][kNT][4];
#pragma unroll
  for (int q = 0; q < kNT; q++)
#pragma unroll
    for (int i = 0; i < 4; i++) acc[0][q][i] = acc[1][q][i] = 0.f;
  up_product<T, kNT, kU>(a, gate, lin, rows, xoff, acc);
  // sum over the warps' shares of D, in warp order
  constexpr int kHalf = kNT * 128;
#pragma unroll
  for (int s = 0; s < 2; s++)
#pragma unroll
    for (int q = 0; q < kNT; q++)
#pragma unroll
      for (int i = 0; i < 4; i++)
        red[(w * 2 + s) * kHalf + (q * 4 + i) * 32 + lane] = acc[s][q][i];
  __syncthreads();
  for (int o = tid; o < kHalf; o += kMoeThreads) {
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int v = 0; v < kMoeWarps; v++) {
      x += red[(v * 2) * kHalf + o];
      y += red[(v * 2 + 1) * kHalf + o];
    }
    const int ol = o & 31, i = (o >> 5) & 3, q = o >> 7;
    const int row = (ol >> 2) + (i >> 1) * 8, col = q * 8 + (ol & 3) * 2 + (i & 1);
    if (row < rows && col < ntok) {
      const float h = moe_act(x, a.act) * y;
      const int64_t at = (int64_t)slot[col] * a.F + f0 + row;
      T hi, lo;
      from_f32(&hi, h);
      const float left = h - to_f32(hi);
      from_f32(&lo, isfinite(left) ? left : 0.f);  // h beyond the type's range stays infinite
      ((T*)a.h_hi)[at] = hi;
      ((T*)a.h_lo)[at] = lo;
    }
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kMoeThreads, 2) moe_up_kernel(MoeArgs a) {
  __shared__ MoeLists L;
  __shared__ float red[kMoeWarps * 2 * 4 * 128];
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.T * a.m; i += kMoeThreads)
      if (a.idx[i] < -1 || a.idx[i] >= a.E) atomicOr(a.status, GMM_DEVFLAG_BAD_INDEX);
  moe_sort(a, L);
  const int64_t all = (int64_t)L.n * a.F;
  const int64_t end = all * (blockIdx.x + 1) / gridDim.x;
  int64_t r = all * blockIdx.x / gridDim.x;
  while (r < end) {
    const int act = (int)(r / a.F), f0 = (int)(r - (int64_t)act * a.F);
    const int rows = (int)min((int64_t)min(kMoeRows, a.F - f0), end - r);
    const int e = L.act[act];
    for (int s0 = L.off[act]; s0 < L.off[act + 1];) {
      const int left = L.off[act + 1] - s0;
      const uint16_t* slot = L.slot + s0;
      if (left <= 8)
        up_tile<T, 1, 4>(a, e, f0, rows, slot, left, red);
      else if (left <= 16)
        up_tile<T, 2, 2>(a, e, f0, rows, slot, left, red);
      else
        up_tile<T, 4, 2>(a, e, f0, rows, slot, min(left, 32), red);
      s0 += left <= 8 ? 8 : left <= 16 ? 16 : 32;
    }
    r += rows;
  }
}

// ------------------------------------------------------------------ down
// A cluster owns a block of up to 16 rows of y for every token.  Its warps share
// out (expert, slice of F) units; a warp adds each unit's weighted product to
// its own copy of the block, and the copies are summed in warp and CTA order, so
// no addition depends on timing.
template <typename T, int kNT, int kU>
__device__ __forceinline__ void down_unit(const MoeArgs& a, int e, int d0, int rows, int c0, int c1,
                                          const uint16_t* slot, int ntok, float* y) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const T* W = (const T*)a.W_down + ((int64_t)e * a.D + d0) * a.F;
  const int64_t r0 = (int64_t)g * a.F, r1 = (int64_t)(g + 8) * a.F;
  const bool ok0 = g < rows, ok1 = g + 8 < rows;
  int64_t hoff[kNT];
#pragma unroll
  for (int q = 0; q < kNT; q++) hoff[q] = q * 8 + g < ntok ? (int64_t)slot[q * 8 + g] * a.F : -1;
  float acc[kNT][4];
#pragma unroll
  for (int q = 0; q < kNT; q++)
#pragma unroll
    for (int i = 0; i < 4; i++) acc[q][i] = 0.f;
  for (int c = c0; c < c1; c += kU) {
    uint4 A[kU][2], B[kU][kNT][2];
#pragma unroll
    for (int u = 0; u < kU; u++) {
      const int k = (c + u) * 32 + t * 8;
      const bool in = c + u < c1 && k < a.F;
      A[u][0] = in && ok0 ? __ldg((const uint4*)(W + r0 + k)) : zero16();
      A[u][1] = in && ok1 ? __ldg((const uint4*)(W + r1 + k)) : zero16();
#pragma unroll
      for (int q = 0; q < kNT; q++) {
        B[u][q][0] = in && hoff[q] >= 0 ? load16((const T*)a.h_hi + hoff[q] + k) : zero16();
        B[u][q][1] = in && hoff[q] >= 0 ? load16((const T*)a.h_lo + hoff[q] + k) : zero16();
      }
    }
#pragma unroll
    for (int u = 0; u < kU; u++)
#pragma unroll
      for (int q = 0; q < kNT; q++) {
        mma_k32<T>(acc[q], A[u][0], A[u][1], B[u][q][0]);
        mma_k32<T>(acc[q], A[u][0], A[u][1], B[u][q][1]);
      }
  }
#pragma unroll
  for (int q = 0; q < kNT; q++)
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int col = q * 8 + t * 2 + i;
      if (col < ntok) {
        const int s = slot[col], tok = s / a.m;
        float gate = 0.f;
        for (int j = s; j < (tok + 1) * a.m; j++) gate += a.idx[j] == e ? a.resp[j] : 0.f;
        y[tok * kMoeRows + g] = fmaf(gate, acc[q][i], y[tok * kMoeRows + g]);
        y[tok * kMoeRows + g + 8] = fmaf(gate, acc[q][i + 2], y[tok * kMoeRows + g + 8]);
      }
    }
  __syncwarp();
}

template <typename T>
__global__ void __launch_bounds__(kMoeThreads, 2) moe_down_kernel(MoeArgs a, int C) {
  __shared__ MoeLists L;
  extern __shared__ float yw[];  // [warp][token][kMoeRows]
  const int tid = threadIdx.x, w = tid >> 5;
  const int rank = C > 1 ? (int)sm100::cluster_ctarank() : 0;
  const int blk = blockIdx.x / C;
  const int d0 = (int)((int64_t)a.D * blk / a.row_blocks);
  const int rows = (int)((int64_t)a.D * (blk + 1) / a.row_blocks) - d0;
  const int per = a.T * kMoeRows;
  for (int i = tid; i < per * kMoeWarps; i += kMoeThreads) yw[i] = 0.f;
  moe_sort(a, L);
  const int chunks = (a.F + 31) / 32, W = kMoeWarps * C;
  const int S = max(1, min((4 * W + L.n - 1) / max(L.n, 1), chunks / 4));
  float* y = yw + w * per;
  for (int u = rank * kMoeWarps + w; u < L.n * S; u += W) {
    const int act = u / S, s = u - act * S, e = L.act[act];
    const int c0 = chunks * s / S, c1 = chunks * (s + 1) / S;
    for (int s0 = L.off[act]; s0 < L.off[act + 1];) {
      const int left = L.off[act + 1] - s0;
      const uint16_t* slot = L.slot + s0;
      if (left <= 8)
        down_unit<T, 1, 4>(a, e, d0, rows, c0, c1, slot, left, y);
      else if (left <= 16)
        down_unit<T, 2, 2>(a, e, d0, rows, c0, c1, slot, left, y);
      else
        down_unit<T, 4, 2>(a, e, d0, rows, c0, c1, slot, min(left, 32), y);
      s0 += left <= 8 ? 8 : left <= 16 ? 16 : 32;
    }
  }
  __syncthreads();
  for (int i = tid; i < per; i += kMoeThreads) {
    float v = yw[i];
#pragma unroll
    for (int q = 1; q < kMoeWarps; q++) v += yw[q * per + i];
    yw[i] = v;
  }
  if (C > 1)
    sm100::cluster_sync();
  else
    __syncthreads();
  T* Y = (T*)a.Y;
  for (int i = tid; i < per; i += kMoeThreads) {
    const int tok = i / kMoeRows, row = i % kMoeRows;
    if (tok % C != rank || row >= rows) continue;
    float v = yw[i];
    if (C > 1) {
      v = 0.f;
      const uint32_t at = sm100::smem_u32(yw + i);
      for (int q = 0; q < C; q++) {
        float x;
        asm volatile("ld.shared::cluster.f32 %0, [%1];"
                     : "=f"(x)
                     : "r"(sm100::map_to_rank(at, q)));
        v += x;
      }
    }
    from_f32(Y + (int64_t)tok * a.ldy + d0 + row, v);
  }
  if (C > 1) sm100::cluster_sync();
}

}  // namespace scem
