// paged_cache.cu -- the paged FP8 (E4M3) cache written by whole chunks of new
// tokens, and read back.
//
//   append  scale = amax / 448 of a row (1 for a zero row), code = E4M3 of
//           x / scale, to nearest even: the rule of the decode step's append
//   gather  bf16 of code * scale
//
// A CTA takes a few consecutive tokens: their pages are looked up once, by one
// thread each, and then all threads walk the tokens' rows in 16-code pieces (16
// bytes of codes, 32 of bf16): the gather's all three tensors' and two pieces at a
// time, the append's one tensor's (the grid's second axis) and one piece at a time.
// A row's maximum is a shuffle reduction over the d/16 lanes that hold it.
// The gather is bound by its bytes: 65536 tokens (H_kv = 4, d_h = 128, d_idx = 64;
// 217 MB) 43 us, 5.0 TB/s.  The append is not: 8192 tokens (27 MB) take 14.4 us, 1.9
// TB/s, 3.5 times their bytes.  Its instructions keep 57 % of the issue slots busy
// (a piece has 16 exact quotients and their conversions; the conversion pipe is at
// 47 %), each CTA begins with the look-ups, a chain of dependent loads, with
// nothing else in flight, and 1536 CTAs are 1.7 rounds of what the SMs hold.  A
// launch of few bytes is the latency of its look-ups, 4 us for 128 tokens.
#include "chunk_launch.h"

namespace msa {
namespace {

constexpr int kThreads = 256;

struct CacheParams {
  ChunkSeqs c;
  const __nv_bfloat16* x[3];  // K, V, index-key rows: append reads them
  __nv_bfloat16* y[3];        // ... gather writes them
  uint8_t* codes[3];
  float* scale[3];
  int H_kv, d_h, d_idx;
  DevStatus* status;
};

// The tokens' places: page * B_k + slot, or -1 (reported).
template <int TOK>
__device__ __forceinline__ void locate(const CacheParams& p, int64_t* place) {
  if (threadIdx.x < TOK) {
    const int t = blockIdx.x * TOK + threadIdx.x;
    int64_t at = -1;
    if (t < p.c.T) {
      const ChunkTok k = chunk_tok(p.c, t);
      if (k.pos >= 0) {
        const int b = k.pos / p.c.B_k;
        const int64_t pg = chunk_page(p.c, k.s, b);
        if (pg >= 0) at = pg * p.c.B_k + (k.pos - b * p.c.B_k);
        else report(p.status, DEV_ERR_BAD_INDEX, 111, k.s, b);
      } else if (k.too_long) {
        report(p.status, DEV_ERR_CACHE_FULL, 110, k.s, t);
      }
    }
    place[threadIdx.x] = at;
  }
  __syncthreads();
}

// Calls f(tensor, piece's index in the tokens' dense rows, in the cache's rows,
// pieces per row) for this thread's pieces of the CTA's tokens, U at a time so that
// their loads overlap; `on` false: nothing to do (shuffles still need the lane).
template <int TOK, int U, typename F>
__device__ __forceinline__ void for_pieces(const CacheParams& p, const int64_t* place, F f) {
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * TOK;
#pragma unroll
  for (int which = 0; which < 3; ++which) {
    if (gridDim.y > 1 && which != static_cast<int>(blockIdx.y)) continue;
    const int per_row = (which < 2 ? p.d_h : p.d_idx) / 16;
    const int per_tok = per_row * (which < 2 ? p.H_kv : 1);
    const int n = TOK * per_tok;
    for (int i0 = 0; i0 < n; i0 += U * blockDim.x) {
      int64_t dense[U], cached[U];
      bool on[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + j * blockDim.x + threadIdx.x;
        const int u = i / per_tok;
        const int64_t at = i < n ? place[u] : -1;
        on[j] = at >= 0;
        dense[j] = t0 * per_tok + i;
        cached[j] = at * per_tok + (i - u * per_tok);
      }
      f(which, per_row, dense, cached, on);
    }
  }
}

template <int TOK, int U>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const CacheParams p) {
  __shared__ int64_t place[TOK];
  locate<TOK>(p, place);
  for_pieces<TOK, U>(p, place, [&](int which, int per_row, const int64_t (&dense)[U],
                                   const int64_t (&cached)[U], const bool (&on)[U]) {
    uint4 raw[U][2];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint4* src = reinterpret_cast<const uint4*>(p.x[which]) + 2 * dense[j];
      raw[j][0] = on[j] ? __ldcs(src) : make_uint4(0, 0, 0, 0);
      raw[j][1] = on[j] ? __ldcs(src + 1) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      float v[16], amax = 0.f;
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(raw[j]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = __bfloat1622float2(h[e]);
        v[2 * e] = f.x;
        v[2 * e + 1] = f.y;
        amax = fmaxf(fmaxf(amax, fabsf(f.x)), fabsf(f.y));
      }
      for (int o = 1; o < per_row; o <<= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
      if (!on[j]) continue;
      const float sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(v[4 * e], sc), __fdiv_rn(v[4 * e + 1], sc)), __NV_SATFINITE,
            __NV_E4M3);
        const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(v[4 * e + 2], sc), __fdiv_rn(v[4 * e + 3], sc)), __NV_SATFINITE,
            __NV_E4M3);
        w[e] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
      }
      reinterpret_cast<uint4*>(p.codes[which])[cached[j]] = make_uint4(w[0], w[1], w[2], w[3]);
      if (cached[j] % per_row == 0) p.scale[which][cached[j] / per_row] = sc;
    }
  });
}

template <int TOK, int U>
__global__ void __launch_bounds__(kThreads) paged_gather_kernel(const CacheParams p) {
  __shared__ int64_t place[TOK];
  locate<TOK>(p, place);
  for_pieces<TOK, U>(p, place, [&](int which, int per_row, const int64_t (&dense)[U],
                                   const int64_t (&cached)[U], const bool (&on)[U]) {
    uint4 c[U];
    float sc[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      c[j] = on[j] ? __ldcs(reinterpret_cast<const uint4*>(p.codes[which]) + cached[j])
                   : make_uint4(0, 0, 0, 0);
      sc[j] = on[j] ? __ldg(p.scale[which] + cached[j] / per_row) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const uint32_t in[4] = {c[j].x, c[j].y, c[j].z, c[j].w};
      uint32_t out[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t h = widen2(in[e >> 1] >> (16 * (e & 1)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
        out[e] = pack_bf16(f.x * sc[j], f.y * sc[j]);
      }
      if (!on[j]) continue;
      uint4* dst = reinterpret_cast<uint4*>(p.y[which]) + 2 * dense[j];
      __stcs(dst, make_uint4(out[0], out[1], out[2], out[3]));
      __stcs(dst + 1, make_uint4(out[4], out[5], out[6], out[7]));
    }
  });
}

__global__ void __launch_bounds__(kThreads) chunk_positions_kernel(const ChunkSeqs c, int32_t* pos) {
  const int t = blockIdx.x * kThreads + threadIdx.x;
  if (t < c.T) pos[t] = chunk_tok(c, t).pos;
}

// seq_len[s] += the chunk's rows of s, where they fit (and were served).
__global__ void __launch_bounds__(kThreads) chunk_advance_kernel(const ChunkSeqs c, int32_t* seq_len) {
  const int s = blockIdx.x * kThreads + threadIdx.x;
  if (s >= c.S) return;
  const int c0 = c.cu[s], c1 = c.cu[s + 1];
  const int len = seq_len[s];
  if (c0 < 0 || c1 <= c0 || c1 > c.T || len < 0) return;
  if (static_cast<int64_t>(len) + (c1 - c0) <= static_cast<int64_t>(c.max_pages) * c.B_k)
    seq_len[s] = len + (c1 - c0);
}

CacheParams params_of(const CacheLaunch& a) {
  CacheParams p{};
  p.c = a.c;
  for (int j = 0; j < 3; ++j) {
    p.x[j] = static_cast<const __nv_bfloat16*>(a.x[j]);
    p.y[j] = static_cast<__nv_bfloat16*>(a.y[j]);
    p.codes[j] = static_cast<uint8_t*>(a.codes[j]);
    p.scale[j] = a.scale[j];
  }
  p.H_kv = a.H_kv;
  p.d_h = a.d_h;
  p.d_idx = a.d_idx;
  p.status = a.status;
  return p;
}

// Tokens per CTA: sixteen (all their rows share a look-up, and every thread has
// several pieces), or one token and one of the tensors while that would leave SMs
// without work.  One / sixteen, us: append 128 tokens 4.2 / 6.2, 512 6.1 / 6.2,
// 1024 8.2 / 6.2, 4096 17.1 / 10.3; gather 128 4.1 / 6.2, 1024 6.2 / 6.2, 4096
// 11.6 / 8.2.
bool few_tokens(int T) { return T < 4 * num_sms(); }

}  // namespace

cudaError_t launch_paged_append(const CacheLaunch& a, cudaStream_t s) {
  const CacheParams p = params_of(a);
  prof_begin("paged_append", s);
  if (few_tokens(a.c.T)) paged_append_kernel<1, 1><<<dim3(a.c.T, 3), 64, 0, s>>>(p);
  else paged_append_kernel<16, 1><<<dim3((a.c.T + 15) / 16, 3), kThreads, 0, s>>>(p);
  prof_end(s);
  return cudaGetLastError();
}

cudaError_t launch_paged_gather(const CacheLaunch& a, cudaStream_t s) {
  const CacheParams p = params_of(a);
  prof_begin("paged_gather", s);
  if (few_tokens(a.c.T)) paged_gather_kernel<1, 1><<<dim3(a.c.T, 3), 64, 0, s>>>(p);
  else paged_gather_kernel<16, 2><<<(a.c.T + 16 - 1) / 16, kThreads, 0, s>>>(p);
  prof_end(s);
  return cudaGetLastError();
}

cudaError_t launch_chunk_positions(const ChunkSeqs& c, int32_t* pos, cudaStream_t s) {
  prof_begin("chunk_positions", s);
  chunk_positions_kernel<<<(c.T + kThreads - 1) / kThreads, kThreads, 0, s>>>(c, pos);
  prof_end(s);
  return cudaGetLastError();
}

cudaError_t launch_chunk_advance(const ChunkSeqs& c, int32_t* seq_len, cudaStream_t s) {
  prof_begin("chunk_advance", s);
  chunk_advance_kernel<<<(c.S + kThreads - 1) / kThreads, kThreads, 0, s>>>(c, seq_len);
  prof_end(s);
  return cudaGetLastError();
}

}  // namespace msa
