// chunk_capi.cu -- the extern "C" boundary of the operators that serve chunks
// of new tokens: argument validation, workspace sizing and launches.  As in
// msa_capi.cu, nothing is allocated here.
#include "capi_common.h"
#include "chunk_launch.h"

namespace {

constexpr int64_t kInt31 = int64_t(1) << 31;

// Sizes of a chunk call; need_*: which of them the call uses.
msa_status check_chunk(const msa_chunk_dims* d, bool need_dh, bool need_didx, bool need_q) {
  if (d == nullptr || d->S < 1 || d->T < 0 || d->max_pages < 1 || d->n_pages < 1 || d->H_kv < 1)
    return MSA_ERR_INVALID_ARG;
  if (!(d->attn_scale >= 0.0f) || !(d->idx_scale >= 0.0f) || isinf(d->attn_scale) ||
      isinf(d->idx_scale))
    return MSA_ERR_INVALID_ARG;
  if (need_q && (d->H_q < 1 || d->H_q % d->H_kv != 0 || d->k < 1)) return MSA_ERR_INVALID_ARG;
  if (d->B_k != 64 && d->B_k != 128) return MSA_ERR_UNSUPPORTED;
  if (d->H_kv > 8) return MSA_ERR_UNSUPPORTED;
  if (need_dh && d->d_h != 64 && d->d_h != 128) return MSA_ERR_UNSUPPORTED;
  if (need_didx && d->d_idx != 64 && d->d_idx != 128) return MSA_ERR_UNSUPPORTED;
  if (need_q && (d->H_q / d->H_kv > 16 || d->k > 32)) return MSA_ERR_UNSUPPORTED;
  // positions, page numbers, row numbers and grids stay in 31 bits
  if (int64_t(d->max_pages) * d->B_k >= kInt31 || d->n_pages >= kInt31)
    return MSA_ERR_UNSUPPORTED;
  if (int64_t(d->T) * d->H_kv * 16 >= kInt31) return MSA_ERR_UNSUPPORTED;
  if (need_q && int64_t(d->T) * d->H_q >= kInt31) return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

msa::ChunkSeqs chunk_seqs(const msa_chunk_dims* d, const int32_t* cu, const int32_t* seq_len,
                          const int32_t* table) {
  msa::ChunkSeqs c{};
  c.cu = cu;
  c.seq_len = seq_len;
  c.table = table;
  c.S = d->S;
  c.T = d->T;
  c.max_pages = d->max_pages;
  c.n_pages = d->n_pages;
  c.B_k = d->B_k;
  return c;
}

// A workspace that holds the status word only: absent, or cleared.
msa_status clear_status(void* ws, size_t ws_bytes, cudaStream_t s) {
  if (ws == nullptr) return MSA_OK;
  if (!aligned16(ws)) return MSA_ERR_INVALID_ARG;
  if (ws_bytes < kStatusBytes) return MSA_ERR_WORKSPACE_TOO_SMALL;
  return msa_from_cuda(cudaMemsetAsync(ws, 0, sizeof(msa::DevStatus), s));
}

template <size_t N>
bool all_aligned(const void* const (&ptrs)[N]) {
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return false;
  return true;
}

msa_status check_norm_rope(const msa_norm_rope_dims* d, const double* inv_freq, bool need_freq) {
  if (d == nullptr || d->T < 0 || d->H_q < 1 || d->H_k < 1 || d->d < 1 || d->rot < 0 ||
      d->rot > d->d || (d->interleaved != 0 && d->interleaved != 1) || !(d->eps >= 0.0f) ||
      isinf(d->eps))
    return MSA_ERR_INVALID_ARG;
  if (d->d != 32 && d->d != 64 && d->d != 128) return MSA_ERR_UNSUPPORTED;
  if (d->rot % 16 != 0) return MSA_ERR_UNSUPPORTED;
  if (need_freq && d->rot > 0) {
    if (inv_freq == nullptr) return MSA_ERR_INVALID_ARG;
    for (int j = 0; j < d->rot / 2; ++j)
      if (!(fabs(inv_freq[j]) < 1e9)) return MSA_ERR_INVALID_ARG;
  }
  return MSA_OK;
}

msa::NormRopeLaunch norm_rope_launch(const msa_norm_rope_dims* d, const double* inv_freq) {
  msa::NormRopeLaunch a{};
  a.inv_freq = inv_freq;
  a.T = d->T;
  a.H_q = d->H_q;
  a.H_k = d->H_k;
  a.d = d->d;
  a.rot = d->rot;
  a.interleaved = d->interleaved != 0;
  a.eps = d->eps;
  return a;
}

size_t scores_bytes(const msa_chunk_dims* d) {
  return msa::align256(sizeof(float) * static_cast<size_t>(d->T) * d->H_kv * d->max_pages);
}
size_t pos_bytes(const msa_chunk_dims* d) { return msa::align256(sizeof(int32_t) * d->T); }

}  // namespace

extern "C" {

// ------------------------------------------------- per-head norm + rotation --
msa_status msa_qk_norm_rope(const msa_norm_rope_dims* d, const double* inv_freq, const void* q,
                            const void* k, const void* w_q, const void* w_k, const int32_t* pos,
                            void* q_out, void* k_out, void* stream) {
  msa::NvtxRange nvtx_range("msa_qk_norm_rope");
  msa_status st = check_norm_rope(d, inv_freq, true);
  if (st != MSA_OK) return st;
  if (d->T == 0) return MSA_OK;
  const void* ptrs[] = {q, k, pos, q_out, k_out};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return MSA_ERR_INVALID_ARG;
  if (!aligned16(w_q) || !aligned16(w_k)) return MSA_ERR_INVALID_ARG;
  msa::NormRopeLaunch a = norm_rope_launch(d, inv_freq);
  a.q = q;
  a.k = k;
  a.w_q = w_q;
  a.w_k = w_k;
  a.pos = pos;
  a.q_out = q_out;
  a.k_out = k_out;
  return msa_from_cuda(msa::launch_norm_rope(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t msa_qk_norm_rope_bwd_workspace(const msa_norm_rope_dims* d) {
  if (check_norm_rope(d, nullptr, false) != MSA_OK) return 0;
  return kStatusBytes + msa::norm_rope_bwd_workspace_bytes(d->T, d->d);
}

msa_status msa_qk_norm_rope_bwd(const msa_norm_rope_dims* d, const double* inv_freq, const void* q,
                                const void* k, const void* w_q, const void* w_k,
                                const int32_t* pos, const void* dq_out, const void* dk_out,
                                void* dq, void* dk, float* dw_q, float* dw_k, void* ws,
                                size_t ws_bytes, void* stream) {
  msa::NvtxRange nvtx_range("msa_qk_norm_rope_bwd");
  msa_status st = check_norm_rope(d, inv_freq, true);
  if (st != MSA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d->T == 0) {  // no rows: the weights' gradients are zero
    for (float* w : {dw_q, dw_k})
      if (w != nullptr &&
          msa_from_cuda(cudaMemsetAsync(w, 0, sizeof(float) * d->d, s)) != MSA_OK)
        return MSA_ERR_CUDA;
    return MSA_OK;
  }
  const void* ptrs[] = {q, k, pos, dq_out, dk_out, dq, dk, ws};
  for (const void* p : ptrs)
    if (p == nullptr || !aligned16(p)) return MSA_ERR_INVALID_ARG;
  const void* opt[] = {w_q, w_k, dw_q, dw_k};
  for (const void* p : opt)
    if (!aligned16(p)) return MSA_ERR_INVALID_ARG;
  if (ws_bytes < msa_qk_norm_rope_bwd_workspace(d)) return MSA_ERR_WORKSPACE_TOO_SMALL;
  if (msa_from_cuda(cudaMemsetAsync(ws, 0, sizeof(msa::DevStatus), s)) != MSA_OK)
    return MSA_ERR_CUDA;
  msa::NormRopeLaunch a = norm_rope_launch(d, inv_freq);
  a.q = q;
  a.k = k;
  a.w_q = w_q;
  a.w_k = w_k;
  a.pos = pos;
  a.dq_out = dq_out;
  a.dk_out = dk_out;
  a.q_out = dq;
  a.k_out = dk;
  a.dw_q = dw_q;
  a.dw_k = dw_k;
  a.ws = static_cast<uint8_t*>(ws) + kStatusBytes;
  return msa_from_cuda(msa::launch_norm_rope(a, s));
}

// ---------------------------------------------------------- paged FP8 cache --
msa_status msa_chunk_positions(const msa_chunk_dims* d, const int32_t* cu_new,
                               const int32_t* seq_len, int32_t* pos, void* stream) {
  msa::NvtxRange nvtx_range("msa_chunk_positions");
  msa_status st = check_chunk(d, false, false, false);
  if (st != MSA_OK) return st;
  if (d->T == 0) return MSA_OK;
  if (!all_aligned({cu_new, seq_len, pos})) return MSA_ERR_INVALID_ARG;
  return msa_from_cuda(msa::launch_chunk_positions(chunk_seqs(d, cu_new, seq_len, nullptr), pos,
                                                   reinterpret_cast<cudaStream_t>(stream)));
}

msa_status msa_paged_append_fp8(const msa_chunk_dims* d, const void* k_new, const void* v_new,
                                const void* k_idx_new, void* k_pages, float* k_scale,
                                void* v_pages, float* v_scale, void* kidx_pages,
                                float* kidx_scale, const int32_t* page_table,
                                const int32_t* cu_new, const int32_t* seq_len, void* ws,
                                size_t ws_bytes, void* stream) {
  msa::NvtxRange nvtx_range("msa_paged_append_fp8");
  msa_status st = check_chunk(d, true, true, false);
  if (st != MSA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d->T > 0 && !all_aligned({k_new, v_new, k_idx_new, k_pages, k_scale, v_pages, v_scale,
                                kidx_pages, kidx_scale, page_table, cu_new, seq_len}))
    return MSA_ERR_INVALID_ARG;
  st = clear_status(ws, ws_bytes, s);
  if (st != MSA_OK || d->T == 0) return st;
  msa::CacheLaunch a{};
  a.c = chunk_seqs(d, cu_new, seq_len, page_table);
  a.x[0] = k_new;
  a.x[1] = v_new;
  a.x[2] = k_idx_new;
  a.codes[0] = k_pages;
  a.codes[1] = v_pages;
  a.codes[2] = kidx_pages;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.scale[2] = kidx_scale;
  a.H_kv = d->H_kv;
  a.d_h = d->d_h;
  a.d_idx = d->d_idx;
  a.status = ws != nullptr ? status_of(ws) : nullptr;
  return msa_from_cuda(msa::launch_paged_append(a, s));
}

msa_status msa_paged_gather_fp8(const msa_chunk_dims* d, const void* k_pages,
                                const float* k_scale, const void* v_pages, const float* v_scale,
                                const void* kidx_pages, const float* kidx_scale,
                                const int32_t* page_table, const int32_t* cu_rows,
                                const int32_t* start, void* k, void* v, void* k_idx, void* ws,
                                size_t ws_bytes, void* stream) {
  msa::NvtxRange nvtx_range("msa_paged_gather_fp8");
  msa_status st = check_chunk(d, true, true, false);
  if (st != MSA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d->T > 0 && !all_aligned({k_pages, k_scale, v_pages, v_scale, kidx_pages, kidx_scale,
                                page_table, cu_rows, start, k, v, k_idx}))
    return MSA_ERR_INVALID_ARG;
  st = clear_status(ws, ws_bytes, s);
  if (st != MSA_OK || d->T == 0) return st;
  msa::CacheLaunch a{};
  a.c = chunk_seqs(d, cu_rows, start, page_table);
  a.y[0] = k;
  a.y[1] = v;
  a.y[2] = k_idx;
  a.codes[0] = const_cast<void*>(k_pages);
  a.codes[1] = const_cast<void*>(v_pages);
  a.codes[2] = const_cast<void*>(kidx_pages);
  a.scale[0] = const_cast<float*>(k_scale);
  a.scale[1] = const_cast<float*>(v_scale);
  a.scale[2] = const_cast<float*>(kidx_scale);
  a.H_kv = d->H_kv;
  a.d_h = d->d_h;
  a.d_idx = d->d_idx;
  a.status = ws != nullptr ? status_of(ws) : nullptr;
  return msa_from_cuda(msa::launch_paged_gather(a, s));
}

// ------------------------------------------------------ selection of a chunk --
msa_status msa_paged_index_scores_fp8(const msa_chunk_dims* d, const void* q_idx,
                                      const void* kidx_pages, const float* kidx_scale,
                                      const int32_t* page_table, const int32_t* cu_new,
                                      const int32_t* seq_len, float* scores, void* ws,
                                      size_t ws_bytes, void* stream) {
  msa::NvtxRange nvtx_range("msa_paged_index_scores_fp8");
  msa_status st = check_chunk(d, false, true, false);
  if (st != MSA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d->T > 0 && !all_aligned({q_idx, kidx_pages, kidx_scale, page_table, cu_new, seq_len, scores}))
    return MSA_ERR_INVALID_ARG;
  st = clear_status(ws, ws_bytes, s);
  if (st != MSA_OK || d->T == 0) return st;
  msa::ScoreLaunch a{};
  a.c = chunk_seqs(d, cu_new, seq_len, page_table);
  a.q_idx = q_idx;
  a.pages = kidx_pages;
  a.scale = kidx_scale;
  a.out = scores;
  a.H_kv = d->H_kv;
  a.d_idx = d->d_idx;
  a.idx_scale = d->idx_scale > 0.0f ? d->idx_scale : 1.0f / sqrtf(static_cast<float>(d->d_idx));
  a.status = ws != nullptr ? status_of(ws) : nullptr;
  return msa_from_cuda(msa::launch_chunk_scores(a, s));
}

msa_status msa_block_topk(const msa_chunk_dims* d, const float* scores, const int32_t* pos,
                          int32_t* idx, void* stream) {
  msa::NvtxRange nvtx_range("msa_block_topk");
  msa_status st = check_chunk(d, false, false, false);
  if (st != MSA_OK) return st;
  if (d->k < 1) return MSA_ERR_INVALID_ARG;
  if (d->k > 32) return MSA_ERR_UNSUPPORTED;
  if (d->T == 0) return MSA_OK;
  if (!all_aligned({scores, pos, idx})) return MSA_ERR_INVALID_ARG;
  return msa_from_cuda(msa::launch_block_topk(scores, pos, idx, d->T, d->H_kv, d->max_pages,
                                              d->B_k, d->k,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

// ------------------------------------------------------ attention of a chunk --
size_t msa_paged_sparse_attn_fp8_workspace(const msa_chunk_dims* d) {
  if (check_chunk(d, true, false, true) != MSA_OK) return 0;
  return kStatusBytes +
         msa::chunk_attend_workspace_bytes(chunk_seqs(d, nullptr, nullptr, nullptr), d->H_q,
                                           d->H_kv, d->d_h, d->k);
}

msa_status msa_paged_sparse_attn_fp8(const msa_chunk_dims* d, const void* q, const int32_t* idx,
                                     const void* k_pages, const float* k_scale,
                                     const void* v_pages, const float* v_scale,
                                     const int32_t* page_table, const int32_t* cu_new,
                                     const int32_t* seq_len, void* o, float* lse, void* ws,
                                     size_t ws_bytes, void* stream) {
  msa::NvtxRange nvtx_range("msa_paged_sparse_attn_fp8");
  msa_status st = check_chunk(d, true, false, true);
  if (st != MSA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d->T == 0) return clear_status(ws, ws_bytes, s);
  if (!all_aligned({q, idx, k_pages, k_scale, v_pages, v_scale, page_table, cu_new, seq_len, o,
                    ws}) ||
      !aligned16(lse))
    return MSA_ERR_INVALID_ARG;
  if (ws_bytes < msa_paged_sparse_attn_fp8_workspace(d)) return MSA_ERR_WORKSPACE_TOO_SMALL;
  st = clear_status(ws, ws_bytes, s);
  if (st != MSA_OK) return st;
  msa::AttendLaunch a{};
  a.c = chunk_seqs(d, cu_new, seq_len, page_table);
  a.q = q;
  a.idx = idx;
  a.k_pages = k_pages;
  a.v_pages = v_pages;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.o = o;
  a.lse = lse;
  a.H_q = d->H_q;
  a.H_kv = d->H_kv;
  a.d_h = d->d_h;
  a.k = d->k;
  a.scale = d->attn_scale > 0.0f ? d->attn_scale : 1.0f / sqrtf(static_cast<float>(d->d_h));
  a.ws = static_cast<uint8_t*>(ws) + kStatusBytes;
  a.status = status_of(ws);
  return msa_from_cuda(msa::launch_chunk_attend(a, s));
}

// ------------------------------------------------------------ the whole step --
size_t msa_paged_chunk_fp8_workspace(const msa_chunk_dims* d) {
  if (check_chunk(d, true, true, true) != MSA_OK) return 0;
  return kStatusBytes + pos_bytes(d) + scores_bytes(d) +
         msa::chunk_attend_workspace_bytes(chunk_seqs(d, nullptr, nullptr, nullptr), d->H_q,
                                           d->H_kv, d->d_h, d->k);
}

msa_status msa_paged_chunk_fp8(const msa_chunk_dims* d, const void* q, const void* q_idx,
                               const void* k_new, const void* v_new, const void* k_idx_new,
                               void* k_pages, float* k_scale, void* v_pages, float* v_scale,
                               void* kidx_pages, float* kidx_scale, const int32_t* page_table,
                               const int32_t* cu_new, int32_t* seq_len, void* o, float* lse,
                               int32_t* idx_out, void* ws, size_t ws_bytes, void* stream) {
  msa::NvtxRange nvtx_range("msa_paged_chunk_fp8");
  msa_status st = check_chunk(d, true, true, true);
  if (st != MSA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d->T == 0) return clear_status(ws, ws_bytes, s);
  if (!all_aligned({q, q_idx, k_new, v_new, k_idx_new, k_pages, k_scale, v_pages, v_scale,
                    kidx_pages, kidx_scale, page_table, cu_new, seq_len, o, idx_out, ws}) ||
      !aligned16(lse))
    return MSA_ERR_INVALID_ARG;
  if (ws_bytes < msa_paged_chunk_fp8_workspace(d)) return MSA_ERR_WORKSPACE_TOO_SMALL;
  st = clear_status(ws, ws_bytes, s);
  if (st != MSA_OK) return st;
  uint8_t* at = static_cast<uint8_t*>(ws) + kStatusBytes;
  int32_t* pos = reinterpret_cast<int32_t*>(at);
  at += pos_bytes(d);
  float* scores = reinterpret_cast<float*>(at);
  at += scores_bytes(d);
  const msa::ChunkSeqs c = chunk_seqs(d, cu_new, seq_len, page_table);

  msa::CacheLaunch ca{};
  ca.c = c;
  ca.x[0] = k_new;
  ca.x[1] = v_new;
  ca.x[2] = k_idx_new;
  ca.codes[0] = k_pages;
  ca.codes[1] = v_pages;
  ca.codes[2] = kidx_pages;
  ca.scale[0] = k_scale;
  ca.scale[1] = v_scale;
  ca.scale[2] = kidx_scale;
  ca.H_kv = d->H_kv;
  ca.d_h = d->d_h;
  ca.d_idx = d->d_idx;
  ca.status = status_of(ws);
  st = msa_from_cuda(msa::launch_paged_append(ca, s));
  if (st != MSA_OK) return st;
  st = msa_from_cuda(msa::launch_chunk_positions(c, pos, s));
  if (st != MSA_OK) return st;

  msa::ScoreLaunch sa{};
  sa.c = c;
  sa.q_idx = q_idx;
  sa.pages = kidx_pages;
  sa.scale = kidx_scale;
  sa.out = scores;
  sa.H_kv = d->H_kv;
  sa.d_idx = d->d_idx;
  sa.idx_scale = d->idx_scale > 0.0f ? d->idx_scale : 1.0f / sqrtf(static_cast<float>(d->d_idx));
  sa.status = status_of(ws);
  st = msa_from_cuda(msa::launch_chunk_scores(sa, s));
  if (st != MSA_OK) return st;
  st = msa_from_cuda(msa::launch_block_topk(scores, pos, idx_out, d->T, d->H_kv, d->max_pages,
                                            d->B_k, d->k, s));
  if (st != MSA_OK) return st;

  msa::AttendLaunch aa{};
  aa.c = c;
  aa.q = q;
  aa.idx = idx_out;
  aa.k_pages = k_pages;
  aa.v_pages = v_pages;
  aa.k_scale = k_scale;
  aa.v_scale = v_scale;
  aa.o = o;
  aa.lse = lse;
  aa.H_q = d->H_q;
  aa.H_kv = d->H_kv;
  aa.d_h = d->d_h;
  aa.k = d->k;
  aa.scale = d->attn_scale > 0.0f ? d->attn_scale : 1.0f / sqrtf(static_cast<float>(d->d_h));
  aa.ws = at;
  aa.status = status_of(ws);
  st = msa_from_cuda(msa::launch_chunk_attend(aa, s));
  if (st != MSA_OK) return st;
  return msa_from_cuda(msa::launch_chunk_advance(c, seq_len, s));
}

}  // extern "C"
