// beam_api.cu -- host side of gmm_beam_select and gmm_beam_reorder: argument checks and launches.
#include <algorithm>

#include "api_common.h"
#include "beam.cuh"

using namespace scem;

namespace {

// Workspace of a selection: each row's best classes and their log p.
size_t select_bytes(int64_t N, int32_t m) { return 2 * align_up((size_t)N * m * 4, 256); }

gmm_status check_select(const gmm_rows* r, int32_t w, int32_t m) {
  if (!r || r->N < 0 || w < 1 || w > kMostBeams || m < 1 || m > kMaxAlt || r->N % w != 0)
    return GMM_ERR_INVALID_ARG;
  if (r->N >= (int64_t)1 << 31) return GMM_ERR_UNSUPPORTED;
  return GMM_OK;
}

template <typename T>
gmm_status merge_launch(const BeamArgs& a, cudaStream_t st) {
  return api_launch_next(beam_merge_kernel<T>, dim3((unsigned)a.B), kMergeThreads, 0, st, a);
}

// As many CTAs as are resident at once: each finds its tiles once.
template <typename Vec, int kW>
gmm_status reorder_launch(const ReorderArgs& a, cudaStream_t st) {
  int sms = 0;
  gmm_status s = api_device_sms(&sms);
  if (s != GMM_OK) return s;
  constexpr int kTile = kReorderThreads * reorder_cols(kW);
  const double tiles = (double)a.n * a.B * (((double)a.outer * a.inner + kTile - 1) / kTile);
  const unsigned grid =
      (unsigned)std::max(1.0, std::min(tiles, (double)sms * reorder_ctas(kW)));
  return api_launch_next(beam_reorder_kernel<Vec, kW>, dim3(grid), kReorderThreads, 0, st, a);
}

template <typename Vec>
gmm_status reorder_width(const ReorderArgs& a, cudaStream_t st) {
  return a.w <= 2    ? reorder_launch<Vec, 2>(a, st)
         : a.w <= 4  ? reorder_launch<Vec, 4>(a, st)
         : a.w <= 8  ? reorder_launch<Vec, 8>(a, st)
         : a.w <= 16 ? reorder_launch<Vec, 16>(a, st)
                     : reorder_launch<Vec, 32>(a, st);
}

// Bytes of a column: 16, 4 or 1, the most that every address of the state is a multiple of.
int column_bytes(const gmm_beam_state& s) {
  const uint64_t all = (uint64_t)(uintptr_t)s.base | (uint64_t)s.row_stride |
                       (uint64_t)s.outer_stride | (uint64_t)s.pos_bytes;
  return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 1;
}

}  // namespace

extern "C" {

gmm_status gmm_beam_workspace_size(const gmm_rows* r, int32_t w, int32_t m, size_t* bytes) {
  gmm_status s = check_select(r, w, m);
  if (s != GMM_OK) return s;
  if (!bytes) return GMM_ERR_INVALID_ARG;
  *bytes = select_bytes(r->N, m);
  return GMM_OK;
}

gmm_status gmm_beam_select(const gmm_rows* r, const void* Z, int32_t w, const float* scores,
                           const uint8_t* ended, int32_t end_id, int32_t m, float* out_scores,
                           int32_t* parent, int32_t* token, uint32_t* dev_flags, void* ws,
                           size_t ws_bytes, void* stream) {
  gmm_status s = check_select(r, w, m);
  if (s != GMM_OK) return s;
  if (ended && (end_id < 0 || end_id >= r->K)) return GMM_ERR_INVALID_ARG;
  if (r->N > 0) {
    if (!scores || !out_scores || !parent || !token) return GMM_ERR_INVALID_ARG;
    if (!ws || (uintptr_t)ws % 256 != 0 || ws_bytes < select_bytes(r->N, m))
      return GMM_ERR_WORKSPACE;
  }
  int32_t* top_idx = (int32_t*)ws;
  float* top_logp = (float*)((char*)ws + align_up((size_t)r->N * m * 4, 256));
  // (checks what is left of r and Z; flags are raised by the merge, for beams that are alive)
  s = gmm_logprobs(r, Z, nullptr, m, nullptr, nullptr, nullptr, top_idx, top_logp, nullptr,
                   stream);
  if (s != GMM_OK || r->N == 0) return s;
  const BeamArgs a = {Z,     r->ld,  r->scale, r->N / w, w,          m,      scores,
                      ended, end_id, top_idx,  top_logp, out_scores, parent, token,
                      dev_flags};
  cudaStream_t st = (cudaStream_t)stream;
  if (r->dtype == GMM_F32) return merge_launch<float>(a, st);
  if (r->dtype == GMM_BF16) return merge_launch<__nv_bfloat16>(a, st);
  return merge_launch<__half>(a, st);
}

gmm_status gmm_beam_reorder(int64_t B, int32_t w, const int32_t* parent, const int32_t* lens,
                            int32_t n, const gmm_beam_state* states, uint32_t* dev_flags,
                            void* stream) {
  if (B < 0 || w < 1 || w > kMostBeams || n < 0 || (n > 0 && !states)) return GMM_ERR_INVALID_ARG;
  if (B > ((int64_t)1 << 31) / w) return GMM_ERR_UNSUPPORTED;
  for (int i = 0; i < n; i++) {
    const gmm_beam_state& s = states[i];
    if (s.outer < 0 || s.count < 0 || s.pos_bytes < 0 || s.row_stride < 0 || s.outer_stride < 0)
      return GMM_ERR_INVALID_ARG;
    const double row = (double)s.outer * (double)s.count * (double)s.pos_bytes;
    if (row == 0 || B == 0) continue;
    if (row > 1e18) return GMM_ERR_UNSUPPORTED;
    for (int j = 0; j < i; j++)  // (one state named twice would be reordered twice at once)
      if (states[j].base == s.base && states[j].outer && states[j].count && states[j].pos_bytes)
        return GMM_ERR_INVALID_ARG;
    const int64_t piece = s.count * s.pos_bytes;  // (rows and pieces lie apart)
    if (!s.base || (B * w > 1 && s.row_stride < piece) || (s.outer > 1 && s.outer_stride < piece))
      return GMM_ERR_INVALID_ARG;
    if (row / column_bytes(s) >= 4294967296.0 - 256 || s.count > 0x7fffffff ||
        (double)B * w * (double)s.row_stride > 1e18 ||
        (double)s.outer * (double)s.outer_stride > 1e18)
      return GMM_ERR_UNSUPPORTED;
    // tiles are counted in 32 bits, 1,024 groups at a time
    if (std::min<double>(B, kReorderGroups) * (row / column_bytes(s) / kReorderThreads + 1) >=
        2147483648.0)
      return GMM_ERR_UNSUPPORTED;
  }
  if (B == 0 || n == 0) return GMM_OK;
  if (!parent) return GMM_ERR_INVALID_ARG;
  // One launch for the states of a shape, up to kStates of them.  (A state that has been taken is
  // one with an earlier state of its shape: no memory is needed to tell.)
  auto empty = [&](const gmm_beam_state& s) {
    return s.outer == 0 || s.count == 0 || s.pos_bytes == 0;
  };
  auto alike = [&](const gmm_beam_state& s, const gmm_beam_state& q) {
    return s.outer == q.outer && s.count == q.count && s.pos_bytes == q.pos_bytes &&
           (lens == nullptr || (s.by_len != 0) == (q.by_len != 0)) &&
           column_bytes(s) == column_bytes(q);
  };
  for (int i = 0; i < n; i++) {
    bool taken = empty(states[i]);
    for (int j = 0; j < i && !taken; j++) taken = !empty(states[j]) && alike(states[i], states[j]);
    if (taken) continue;
    const int bytes = column_bytes(states[i]);
    ReorderArgs a = {};
    a.parent = parent;
    a.lens = states[i].by_len ? lens : nullptr;
    a.B = B;
    a.w = w;
    a.outer = (uint32_t)states[i].outer;
    a.per_pos = (uint32_t)(states[i].pos_bytes / bytes);
    a.inner = (uint32_t)states[i].count * a.per_pos;
    a.flags = dev_flags;
    for (int j = i; j <= n; j++) {
      if (a.n == kStates || (j == n && a.n > 0)) {
        cudaStream_t st = (cudaStream_t)stream;
        const gmm_status s = bytes == 16  ? reorder_width<uint4>(a, st)
                             : bytes == 4 ? reorder_width<uint32_t>(a, st)
                                          : reorder_width<uint8_t>(a, st);
        if (s != GMM_OK) return s;
        a.n = 0;
      }
      if (j < n && alike(states[j], states[i]))
        a.state[a.n++] = {(char*)states[j].base, states[j].row_stride, states[j].outer_stride};
    }
  }
  return GMM_OK;
}

}  // extern "C"
