// chunk_index.cu -- the Index Branch for chunks of new tokens on the paged FP8
// cache: block scores of every row against the cached index keys (Eq. 6 and
// the block max-pool), then Eq. 7's selection from them.
//
//   M[t, r, b] = idx_scale * max over the keys j of block b of
//                <q_idx[t, r], e4m3(c_j)> * s_j      for b < own block of t
//   M[t, r, b] = -inf                                for the others
//
// Unlike the prefill's index kernel, which keeps each row's Top-k while it
// walks all earlier keys, a chunk writes its scores: a chunk has few rows, so
// the keys are split over the SMs and no CTA sees a whole row.  M is small
// beside the work (4 bytes per 2 * d_idx * B_k operations).
#include <cuda_fp8.h>

#include "chunk_launch.h"

namespace msa {
namespace {

struct ScoreParams {
  ChunkSeqs c;
  const __nv_bfloat16* q;  // [T, H_kv, d_idx]
  const uint8_t* pages;    // [n_pages, B_k, d_idx]
  const float* scale;      // [n_pages, B_k]
  float* out;              // [T, H_kv, max_pages]
  int H_kv;
  int tpt;                 // tokens per CTA column tile
  float idx_scale;
  DevStatus* status;
};

// Two E4M3 codes -> an f16 pair (exact), one conversion instruction.
__device__ __forceinline__ uint32_t widen2(uint32_t c2) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c2 & 0xFFFFu), __NV_E4M3);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Scores on mma.sync, straight from global memory.  MMA rows = 16 keys, whose
// codes widen to f16 in registers; columns = the (token, group) rows of the
// CTA's tpt tokens, NT tiles of 8.  The d axis is consumed in a per-thread
// order (thread t of a quad owns d in [t*D/4, (t+1)*D/4)), the same for keys
// and queries.  A query enters as f16 times a power of two that puts its
// largest magnitude in [2^13, 2^14): exact for every value within 2^-30 of
// it.  One warp scores one block at a time, the blocks strided over the grid's
// x; each key byte is read once per column tile.
template <int D, int BK, int NT>
__global__ void __launch_bounds__(256) chunk_scores_kernel(const ScoreParams p) {
  constexpr int DT = D / 4;     // codes per thread and key row
  constexpr int NMMA = D / 16;  // MMAs per 16-key tile
  constexpr int NU = DT / 16;   // 16-byte loads per thread and key row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int t_end = min(p.c.T, static_cast<int>(blockIdx.y + 1) * p.tpt);
  // the tile's tokens, one sequence's run at a time
  for (int ta = blockIdx.y * p.tpt; ta < t_end;) {
    const ChunkTok tok = chunk_tok(p.c, ta);
    if (tok.pos < 0) {
      if (tok.too_long && blockIdx.x == 0 && threadIdx.x == 0)
        report(p.status, DEV_ERR_CACHE_FULL, 120, tok.s, ta);
      ++ta;
      continue;
    }
    const int tb = min(t_end, __ldg(p.c.cu + tok.s + 1));
    const int ncol = (tb - ta) * p.H_kv;
    const int64_t row0 = static_cast<int64_t>(ta) * p.H_kv;
    uint32_t bq[NT][NMMA][2];
    float unscale[NT][2];  // of columns 2t, 2t + 1
    int own[NT][2];        // their tokens' own blocks (-1 past the columns)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int col = 8 * n + g;
      const __nv_bfloat16* qr = p.q + (row0 + (col < ncol ? col : 0)) * D;
      float qv[NMMA][4], amax = 0.f;
#pragma unroll
      for (int j = 0; j < NMMA; ++j) {
        const uint2 raw = __ldg(reinterpret_cast<const uint2*>(qr + t * DT + 4 * j));
        const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.x));
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw.y));
        qv[j][0] = a.x;
        qv[j][1] = a.y;
        qv[j][2] = b.x;
        qv[j][3] = b.y;
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(qv[j][e]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
      const int shift = amax > 0.f ? min(13 - ilogbf(amax), 126) : 0;
#pragma unroll
      for (int j = 0; j < NMMA; ++j) {
        const __half2 lo = __floats2half2_rn(ldexpf(qv[j][0], shift), ldexpf(qv[j][1], shift));
        const __half2 hi = __floats2half2_rn(ldexpf(qv[j][2], shift), ldexpf(qv[j][3], shift));
        bq[n][j][0] = *reinterpret_cast<const uint32_t*>(&lo);
        bq[n][j][1] = *reinterpret_cast<const uint32_t*>(&hi);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int sh = __shfl_sync(0xFFFFFFFFu, shift, (2 * t + e) * 4);
        unscale[n][e] = ldexpf(p.idx_scale, -sh);
        const int cc = 8 * n + 2 * t + e;
        own[n][e] = cc < ncol ? (tok.pos + cc / p.H_kv) / BK : -1;
      }
    }
    const int last = (tok.pos + tb - ta - 1) / BK;  // own block of the run's last token
    float* out = p.out + row0 * p.c.max_pages;
    for (int b = blockIdx.x * 8 + warp; b < p.c.max_pages; b += gridDim.x * 8) {
      float mx[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) mx[n][0] = mx[n][1] = -INFINITY;
      const int64_t pg = b < last ? chunk_page(p.c, tok.s, b) : -1;
      if (b < last && pg < 0 && lane == 0) report(p.status, DEV_ERR_BAD_INDEX, 121, tok.s, b);
      if (pg >= 0) {
        const uint8_t* kbase = p.pages + (pg * BK + g) * D + t * DT;
        const float* sbase = p.scale + pg * BK + g;
        // the block in halves: a half's codes are all loaded before its MMAs
        constexpr int HALF = BK / 32;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 cr[HALF][2][NU];
          float sc[HALF][2];
#pragma unroll
          for (int i = 0; i < HALF; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int key = (h * HALF + i) * 16 + 8 * e;
#pragma unroll
              for (int u = 0; u < NU; ++u)
                cr[i][e][u] = __ldg(reinterpret_cast<const uint4*>(kbase + key * D) + u);
              sc[i][e] = __ldg(sbase + key);
            }
#pragma unroll
          for (int i = 0; i < HALF; ++i) {
            float acc[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
            for (int j = 0; j < NMMA; ++j) {
              // k-slots 2t,2t+1 <- d0,d0+1 ; 2t+8,2t+9 <- d0+2,d0+3 (d0 = t*DT + 4j)
              const uint32_t w0 = reinterpret_cast<const uint32_t*>(cr[i][0])[j];
              const uint32_t w1 = reinterpret_cast<const uint32_t*>(cr[i][1])[j];
              const uint32_t a[4] = {widen2(w0), widen2(w1), widen2(w0 >> 16), widen2(w1 >> 16)};
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_f16_16816(acc[n], a, bq[n][j][0], bq[n][j][1]);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              mx[n][0] = fmax3(mx[n][0], (acc[n][0] * unscale[n][0]) * sc[i][0],
                               (acc[n][2] * unscale[n][0]) * sc[i][1]);
              mx[n][1] = fmax3(mx[n][1], (acc[n][1] * unscale[n][1]) * sc[i][0],
                               (acc[n][3] * unscale[n][1]) * sc[i][1]);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
              mx[n][e] = fmaxf(mx[n][e], __shfl_xor_sync(0xFFFFFFFFu, mx[n][e], o));
      }
      if (g == 0)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (own[n][e] >= 0)
              out[static_cast<int64_t>(8 * n + 2 * t + e) * p.c.max_pages + b] =
                  b < own[n][e] ? mx[n][e] : -INFINITY;
    }
    ta = tb;
  }
}

// ------------------------------------------------------------------- top-k --
struct TopkParams {
  const float* scores;  // [T, H_kv, n]
  const int32_t* pos;   // [T]
  int32_t* idx;         // [T, H_kv, k]
  int T, H_kv, n, B_k, k;
};

// The 32 lanes' values in descending order (bitonic network).
__device__ __forceinline__ float warp_sort_desc(float x, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int o = size >> 1; o > 0; o >>= 1) {
      const float y = __shfl_xor_sync(0xFFFFFFFFu, x, o);
      const bool want_max = ((lane & size) == 0) == ((lane & o) == 0);
      x = want_max ? fmaxf(x, y) : fminf(x, y);
    }
  return x;
}

// One warp per row.  The row's candidates (blocks before its own) are read
// once, NR * 32 of them at a time in registers.  The (k-1)-th largest of the 32
// lanes' maxima is a lower bound of the (k-1)-th largest candidate, so only
// the few candidates at or above it (and above what is kept already) enter the
// running list, which lane i holds the i-th best of; each entry costs a
// ballot and a shift.  Candidates come in ascending block order and a later
// one must be larger to pass an earlier one: ties keep the lower block.
// Scores of -inf and NaN are never chosen.
template <int NR>
__global__ void __launch_bounds__(256) block_topk_kernel(const TopkParams p) {
  griddep_wait();  // the scores may still be in flight
  const int lane = threadIdx.x & 31;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (row >= static_cast<int64_t>(p.T) * p.H_kv) return;
  const int t = static_cast<int>(row / p.H_kv);
  const int pos = __ldg(p.pos + t);
  if (pos < 0) return;
  const int own = pos / p.B_k;
  const int n = min(own, p.n);
  const int k1 = p.k - 1;
  const float* src = p.scores + row * p.n;
  float lv = -INFINITY;
  int li = -1;
  for (int base = 0; base < n && k1 > 0; base += NR * 32) {
    float x[NR], mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      const int b = base + 32 * j + lane;
      x[j] = b < n ? __ldg(src + b) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < NR; ++j) mx = fmaxf(mx, x[j]);
    const float floor_ = __shfl_sync(0xFFFFFFFFu, warp_sort_desc(mx, lane), k1 - 1);
    float worst = __shfl_sync(0xFFFFFFFFu, lv, k1 - 1);
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      unsigned todo = __ballot_sync(0xFFFFFFFFu, x[j] > worst && x[j] >= floor_);
      while (todo != 0) {
        const int from = __ffs(todo) - 1;
        const float v = __shfl_sync(0xFFFFFFFFu, x[j], from);
        const int at = __popc(__ballot_sync(0xFFFFFFFFu, lv >= v));
        const float uv = __shfl_up_sync(0xFFFFFFFFu, lv, 1);
        const int ui = __shfl_up_sync(0xFFFFFFFFu, li, 1);
        if (lane > at) {
          lv = uv;
          li = ui;
        } else if (lane == at) {
          lv = v;
          li = base + 32 * j + from;
        }
        worst = __shfl_sync(0xFFFFFFFFu, lv, k1 - 1);
        todo &= todo - 1;
        todo &= __ballot_sync(0xFFFFFFFFu, x[j] > worst);
      }
    }
  }
  // the kept blocks and the row's own, ascending, then -1
  const int kept = __popc(__ballot_sync(0xFFFFFFFFu, lane < k1 && li >= 0));
  const int mine = lane < kept ? li : (lane == kept ? own : 0x7FFFFFFF);
  int at = 0;
  for (int j = 0; j <= kept; ++j) at += __shfl_sync(0xFFFFFFFFu, mine, j) < mine ? 1 : 0;
  int32_t* dst = p.idx + row * p.k;
  if (lane <= kept) dst[at] = mine;
  else if (lane < p.k) dst[lane] = -1;
}

template <int D, int BK>
cudaError_t launch_scores_typed(const ScoreLaunch& a, cudaStream_t s) {
  ScoreParams p{};
  p.c = a.c;
  p.q = static_cast<const __nv_bfloat16*>(a.q_idx);
  p.pages = static_cast<const uint8_t*>(a.pages);
  p.scale = a.scale;
  p.out = a.out;
  p.H_kv = a.H_kv;
  p.idx_scale = a.idx_scale;
  p.status = a.status;
  const int sms = num_sms();
  // Columns per tile: 8 while there are no more tokens than sequences (single
  // tokens share no keys), else 32.
  const bool wide = a.c.T > a.c.S && a.c.T * a.H_kv > 8;
  p.tpt = (wide ? 32 : 8) / a.H_kv;
  const int tiles = (a.c.T + p.tpt - 1) / p.tpt;
  // about four CTAs per SM over all tiles, and no more than the blocks need
  int split = (4 * sms + tiles - 1) / tiles;
  const int most = (a.c.max_pages + 7) / 8;
  if (split > most) split = most;
  const dim3 grid(split, tiles);
  prof_begin("chunk_scores", s);
  if (wide) chunk_scores_kernel<D, BK, 4><<<grid, 256, 0, s>>>(p);
  else chunk_scores_kernel<D, BK, 1><<<grid, 256, 0, s>>>(p);
  prof_end(s);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_chunk_scores(const ScoreLaunch& a, cudaStream_t s) {
  if (a.d_idx == 64)
    return a.c.B_k == 128 ? launch_scores_typed<64, 128>(a, s) : launch_scores_typed<64, 64>(a, s);
  return a.c.B_k == 128 ? launch_scores_typed<128, 128>(a, s) : launch_scores_typed<128, 64>(a, s);
}

cudaError_t launch_block_topk(const float* scores, const int32_t* pos, int32_t* idx, int T,
                              int H_kv, int n, int B_k, int k, cudaStream_t s) {
  const TopkParams p{scores, pos, idx, T, H_kv, n, B_k, k};
  const int64_t threads = static_cast<int64_t>(T) * H_kv * 32;
  const dim3 grid(static_cast<unsigned>((threads + 255) / 256));
  prof_begin("block_topk", s);
  const cudaError_t e = n <= 256 ? launch_pdl(block_topk_kernel<8>, grid, dim3(256), 0, s, p)
                                 : launch_pdl(block_topk_kernel<32>, grid, dim3(256), 0, s, p);
  prof_end(s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace msa
