// paged_cache.cu -- the paged FP8 (E4M3) cache written by whole chunks of new
// tokens, and read back.
//
//   append  scale = amax / 448 of a row (1 for a zero row), code = E4M3 of
//           x / scale, to nearest even: the rule of the decode step's append
//   gather  bf16 of code * scale
//
// Both are bound by the bytes they move.  A row (one head's d values of one
// token) belongs to d/8 lanes: 16 bytes of bf16 and 8 bytes of codes each, so
// the row maximum is a shuffle reduction and a row is read once.  The K, V and
// index-key rows are three ranges of one grid.
#include <cuda_fp8.h>

#include "chunk_common.cuh"

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
  int blocks_kv;  // CTAs of the K rows (and as many of the V rows)
  DevStatus* status;
};

// This thread's row: which tensor, which token and head, which 8 values.
struct CacheRow {
  int which, g, l, t, r, H, d;
};
__device__ __forceinline__ CacheRow row_of(const CacheParams& p) {
  CacheRow w;
  int b = blockIdx.x;
  w.which = b < p.blocks_kv ? 0 : (b < 2 * p.blocks_kv ? 1 : 2);
  b -= w.which * p.blocks_kv;
  w.H = w.which < 2 ? p.H_kv : 1;
  w.d = w.which < 2 ? p.d_h : p.d_idx;
  w.g = w.d / 8;
  const int64_t i = static_cast<int64_t>(b) * kThreads + threadIdx.x;
  const int64_t row = i / w.g;
  w.l = static_cast<int>(i - row * w.g);
  const int64_t t = row / w.H;
  w.t = t < p.c.T ? static_cast<int>(t) : p.c.T;  // T: past the rows
  w.r = static_cast<int>(row - t * w.H);
  return w;
}

// The row's place among its tensor's cached rows, or -1 (reported once a row).
__device__ __forceinline__ int64_t cached_row(const CacheParams& p, const CacheRow& w) {
  if (w.t >= p.c.T) return -1;
  const ChunkTok k = chunk_tok(p.c, w.t);
  if (k.pos < 0) {
    if (k.too_long && w.l == 0) report(p.status, DEV_ERR_CACHE_FULL, 110, k.s, w.t);
    return -1;
  }
  const int b = k.pos / p.c.B_k;
  const int64_t pg = chunk_page(p.c, k.s, b);
  if (pg < 0) {
    if (w.l == 0) report(p.status, DEV_ERR_BAD_INDEX, 111, k.s, b);
    return -1;
  }
  return (pg * p.c.B_k + (k.pos - b * p.c.B_k)) * w.H + w.r;
}

__global__ void __launch_bounds__(kThreads) paged_append_kernel(const CacheParams p) {
  const CacheRow w = row_of(p);
  uint4 raw = make_uint4(0, 0, 0, 0);
  if (w.t < p.c.T)
    raw = __ldg(reinterpret_cast<const uint4*>(p.x[w.which]) +
                (static_cast<int64_t>(w.t) * w.H + w.r) * w.g + w.l);
  const int64_t row = cached_row(p, w);
  float v[8], amax = 0.f;
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&raw);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __bfloat1622float2(h[e]);
    v[2 * e] = f.x;
    v[2 * e + 1] = f.y;
    amax = fmax3(amax, fabsf(f.x), fabsf(f.y));
  }
  for (int o = 1; o < w.g; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if (row < 0) return;
  const float sc = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
  uint32_t c[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(v[4 * j], sc), __fdiv_rn(v[4 * j + 1], sc)), __NV_SATFINITE,
        __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(
        make_float2(__fdiv_rn(v[4 * j + 2], sc), __fdiv_rn(v[4 * j + 3], sc)), __NV_SATFINITE,
        __NV_E4M3);
    c[j] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
  reinterpret_cast<uint2*>(p.codes[w.which])[row * w.g + w.l] = make_uint2(c[0], c[1]);
  if (w.l == 0) p.scale[w.which][row] = sc;
}

__global__ void __launch_bounds__(kThreads) paged_gather_kernel(const CacheParams p) {
  const CacheRow w = row_of(p);
  const int64_t row = cached_row(p, w);
  if (row < 0) return;
  const uint2 c = __ldg(reinterpret_cast<const uint2*>(p.codes[w.which]) + row * w.g + w.l);
  const float sc = __ldg(p.scale[w.which] + row);
  const uint32_t in[2] = {c.x, c.y};
  uint32_t out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((in[j >> 1] >> (16 * (j & 1))) & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    out[j] = pack_bf16(f.x * sc, f.y * sc);
  }
  __stcs(reinterpret_cast<uint4*>(p.y[w.which]) +
             (static_cast<int64_t>(w.t) * w.H + w.r) * w.g + w.l,
         make_uint4(out[0], out[1], out[2], out[3]));
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
  p.blocks_kv = static_cast<int>(
      (static_cast<int64_t>(a.c.T) * a.H_kv * (a.d_h / 8) + kThreads - 1) / kThreads);
  p.status = a.status;
  return p;
}

unsigned blocks_of(const CacheParams& p) {
  const int64_t idx = (static_cast<int64_t>(p.c.T) * (p.d_idx / 8) + kThreads - 1) / kThreads;
  return static_cast<unsigned>(2 * static_cast<int64_t>(p.blocks_kv) + idx);
}

}  // namespace

cudaError_t launch_paged_append(const CacheLaunch& a, cudaStream_t s) {
  const CacheParams p = params_of(a);
  prof_begin("paged_append", s);
  paged_append_kernel<<<blocks_of(p), kThreads, 0, s>>>(p);
  prof_end(s);
  return cudaGetLastError();
}

cudaError_t launch_paged_gather(const CacheLaunch& a, cudaStream_t s) {
  const CacheParams p = params_of(a);
  prof_begin("paged_gather", s);
  paged_gather_kernel<<<blocks_of(p), kThreads, 0, s>>>(p);
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
