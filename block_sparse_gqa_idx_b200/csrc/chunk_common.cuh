// chunk_common.cuh -- what the chunk operators share: which sequence and
// position a row of new tokens has, and where that position lives in the
// paged FP8 cache.
//
// A call has T rows of new tokens; sequence s owns rows cu[s] .. cu[s+1]-1
// and had seq_len[s] tokens cached before them, so row t sits at position
// seq_len[s] + t - cu[s].  Both arrays are device memory and are read by the
// kernels, never trusted: a row that no sequence holds, or whose sequence
// does not fit max_pages * B_k tokens, has position -1 and is skipped.
#pragma once
#include <cuda_fp8.h>

#include "msa_internal.h"

namespace msa {

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Two E4M3 codes -> an f16 pair (exact), one conversion instruction.
__device__ __forceinline__ uint32_t widen2(uint32_t c2) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c2 & 0xFFFFu), __NV_E4M3);
  return *reinterpret_cast<const uint32_t*>(&h);
}

struct ChunkSeqs {
  const int32_t* cu;       // [S + 1]
  const int32_t* seq_len;  // [S] tokens cached before the chunk
  const int32_t* table;    // [S, max_pages]
  int S, T, max_pages;
  int64_t n_pages;
  int B_k;
};

struct ChunkTok {
  int s;         // sequence
  int pos;       // position in it, -1 = skip the row
  bool too_long; // skipped because its sequence does not fit its pages
};

__device__ __forceinline__ ChunkTok chunk_tok(const ChunkSeqs& c, int t) {
  int lo = 0, hi = c.S;  // the last s with cu[s] <= t: skips empty sequences
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(c.cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  const int c0 = __ldg(c.cu + lo), c1 = __ldg(c.cu + lo + 1);
  if (t < c0 || t >= c1 || t >= c.T) return {lo, -1, false};
  const int64_t len = __ldg(c.seq_len + lo);
  const int64_t end = len + (static_cast<int64_t>(c1) - c0);
  if (len < 0 || end > static_cast<int64_t>(c.max_pages) * c.B_k) return {lo, -1, true};
  return {lo, static_cast<int>(len + t - c0), false};
}

// The page of block b of sequence s, or -1 when the table's entry is outside
// the pool.
__device__ __forceinline__ int64_t chunk_page(const ChunkSeqs& c, int s, int b) {
  const int32_t pg = __ldg(c.table + static_cast<int64_t>(s) * c.max_pages + b);
  return pg >= 0 && pg < c.n_pages ? pg : -1;
}

}  // namespace msa
