// chunk_launch.h -- launchers of the chunk operators (chunk_capi.cu calls them).
#pragma once
#include "chunk_common.cuh"

namespace msa {

// K, V and index-key rows of the chunk's tokens and their pages.
struct CacheLaunch {
  ChunkSeqs c;
  const void* x[3];  // append reads these bf16 rows
  void* y[3];        // gather writes these
  void* codes[3];
  float* scale[3];
  int H_kv, d_h, d_idx;
  DevStatus* status;  // or null
};
cudaError_t launch_paged_append(const CacheLaunch& a, cudaStream_t s);
cudaError_t launch_paged_gather(const CacheLaunch& a, cudaStream_t s);
cudaError_t launch_chunk_positions(const ChunkSeqs& c, int32_t* pos, cudaStream_t s);
cudaError_t launch_chunk_advance(const ChunkSeqs& c, int32_t* seq_len, cudaStream_t s);

// Block scores of the chunk's rows against the cached index keys.
struct ScoreLaunch {
  ChunkSeqs c;
  const void* q_idx;
  const void* pages;
  const float* scale;
  float* out;
  int H_kv, d_idx;
  float idx_scale;
  DevStatus* status;  // or null
};
cudaError_t launch_chunk_scores(const ScoreLaunch& a, cudaStream_t s);
// The selection of T x H_kv rows from n block scores each.
cudaError_t launch_block_topk(const float* scores, const int32_t* pos, int32_t* idx, int T,
                              int H_kv, int n, int B_k, int k, cudaStream_t s);

// Eq. 8 of the chunk's rows over their selected pages.
struct AttendLaunch {
  ChunkSeqs c;
  const void* q;
  const int32_t* idx;
  const void* k_pages;
  const void* v_pages;
  const float* k_scale;
  const float* v_scale;
  void* o;
  float* lse;  // or null
  int H_q, H_kv, d_h, k;
  float scale;
  void* ws;  // chunk_attend_workspace_bytes
  DevStatus* status;
};
size_t chunk_attend_workspace_bytes(const ChunkSeqs& c, int H_q, int H_kv, int d_h, int k);
cudaError_t launch_chunk_attend(const AttendLaunch& a, cudaStream_t s);
// The KV-outer form, for chunks of many rows (chunk_attn_kv.cu).
size_t chunk_attend_kv_workspace_bytes(int T, int S, int max_pages, int H_q, int H_kv, int d_h,
                                       int k);
cudaError_t launch_chunk_attend_kv(const AttendLaunch& a, cudaStream_t s);

}  // namespace msa
