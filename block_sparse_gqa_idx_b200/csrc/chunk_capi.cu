// chunk_capi.cu -- the extern "C" boundary of the operators that serve chunks
// of new tokens: argument validation, workspace sizing and launches.  As in
// msa_capi.cu, nothing is allocated here.
#include "capi_common.h"

namespace {

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

}  // extern "C"
