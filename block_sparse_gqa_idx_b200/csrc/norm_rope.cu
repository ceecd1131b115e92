// norm_rope.cu -- RMS normalisation of every query and key head, then the
// position rotation, in one pass over the rows (forward), and its backward.
//
//   n = x / sqrt(mean(x^2) + eps),  y = R(pos) (w * n)
//   R rotates the pairs (j, j + rot/2) -- or (2j, 2j + 1), interleaved -- by
//   the angle pos * inv_freq[j], j < rot/2; dimensions rot .. d-1 pass through.
// Backward, with g = R(pos)^T dy:
//   dw = sum over rows of g * n,  dx = (w g - n mean(w g n)) / sqrt(mean(x^2) + eps)
//
// A row (one head of one token) is read once by d/8 lanes, 16 bytes each, and
// stays in registers: the mean is a shuffle reduction over those lanes and the
// partner of a rotated pair is one shuffle away.  The angle never loses its
// far positions: inv_freq is held as a fraction of a turn in 64-bit fixed
// point, so pos * turn modulo 2^64 is the exact fractional turn, and
// sincospi sees at most half a turn.  A token's cosines and sines are computed
// once per CTA and shared by all of its heads.
#include <math_constants.h>

#include "msa_internal.h"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct NRParams {
  const __nv_bfloat16* x[2];  // q, k
  const __nv_bfloat16* w[2];  // or null: no weight
  const __nv_bfloat16* dy[2];
  __nv_bfloat16* out[2];      // y forward, dx backward
  const int32_t* pos;
  float* part;                // backward: [grid][2][D] partial dw
  int T, H[2], half;          // half: rotated pairs
  float eps;
  uint64_t turn[64];          // inv_freq / (2 pi) in units of 2^-64 turns
};

struct Row8 {
  float v[8];
};

__device__ __forceinline__ Row8 unpack8(uint4 u) {
  Row8 r;
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __bfloat1622float2(h[e]);
    r.v[2 * e] = f.x;
    r.v[2 * e + 1] = f.y;
  }
  return r;
}
__device__ __forceinline__ uint4 pack8(const Row8& r) {
  return make_uint4(pack_bf16(r.v[0], r.v[1]), pack_bf16(r.v[2], r.v[3]),
                    pack_bf16(r.v[4], r.v[5]), pack_bf16(r.v[6], r.v[7]));
}

// Sum over the LPR lanes that hold one row.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// This lane's cosines and sines.  Pairs (j, j + half): lane l holds
// dimensions 8l .. 8l+7, which rotate with those of lane l -+ half/8; `sn` is
// then the sine with the sign of this side.  Interleaved: four pairs in the
// lane.  Dimensions that pass through get cos 1, sin 0.
template <int LPR, bool INTER>
struct Angles {
  float cs[INTER ? 4 : 8], sn[INTER ? 4 : 8];
  int partner;  // lane (within the warp) of the paired dimensions

  __device__ __forceinline__ void load(const float2* tab, int half, int lane) {
    const int l = lane % LPR;
    partner = lane;
    if constexpr (INTER) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = 4 * l + e;
        const float2 a = j < half ? tab[j] : make_float2(1.f, 0.f);
        cs[e] = a.x;
        sn[e] = a.y;
      }
    } else {
      const int hl = half / 8;
      const bool lo = l < hl, hi = !lo && l < 2 * hl;
      if (lo) partner = lane + hl;
      if (hi) partner = lane - hl;
      const int j0 = lo ? 8 * l : (hi ? 8 * (l - hl) : 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 a = lo || hi ? tab[j0 + e] : make_float2(1.f, 0.f);
        cs[e] = a.x;
        sn[e] = lo ? -a.y : a.y;
      }
    }
  }
  // y = R x (sgn = 1) or R^T x (sgn = -1)
  __device__ __forceinline__ Row8 turn(const Row8& x, float sgn) const {
    Row8 y;
    if constexpr (INTER) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float a = x.v[2 * e], b = x.v[2 * e + 1], s = sgn * sn[e];
        y.v[2 * e] = a * cs[e] - b * s;
        y.v[2 * e + 1] = b * cs[e] + a * s;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float other = __shfl_sync(0xFFFFFFFFu, x.v[e], partner);
        y.v[e] = x.v[e] * cs[e] + other * (sgn * sn[e]);
      }
    }
    return y;
  }
};

// cos and sin of the `half` angles of each of the CTA's tokens, into smem.
template <int TOK>
__device__ __forceinline__ void fill_table(const NRParams& p, int t0, float2 (*tab)[64]) {
  for (int i = threadIdx.x; i < TOK * p.half; i += kThreads) {
    const int u = i / p.half, j = i - u * p.half;
    if (t0 + u >= p.T) continue;
    const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(p.pos[t0 + u])) * p.turn[j];
    float s, c;  // frac as a signed fraction of half a turn
    sincospif(static_cast<float>(static_cast<int64_t>(frac)) * 0x1p-63f, &s, &c);
    tab[u][j] = make_float2(c, s);
  }
}

// TOK tokens per CTA, kWarps / TOK warps on each; a warp takes 32 / LPR rows
// at a time.  Rows of a token with pos < 0 (padding) are left untouched.
template <int D, bool INTER, int TOK>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NRParams p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, WPT = kWarps / TOK;
  __shared__ float2 tab[TOK][64];
  const int t0 = blockIdx.x * TOK;
  fill_table<TOK>(p, t0, tab);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u = warp / WPT, t = t0 + u;
  if (t >= p.T || p.pos[t] < 0) return;
  Angles<LPR, INTER> ang;
  ang.load(tab[u], p.half, lane);
  const int first = (warp % WPT) * RPW + lane / LPR, l = lane % LPR;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int H = p.H[which];
    Row8 w;
#pragma unroll
    for (int e = 0; e < 8; ++e) w.v[e] = 1.f;
    if (p.w[which] != nullptr) w = unpack8(reinterpret_cast<const uint4*>(p.w[which])[l]);
    const int64_t base = static_cast<int64_t>(t) * H;
    const uint4* src = reinterpret_cast<const uint4*>(p.x[which]);
    uint4* dst = reinterpret_cast<uint4*>(p.out[which]);
    // two rows in flight per lane; whole warps stay in the loop (shuffles)
    for (int h0 = 0; h0 < H; h0 += 2 * WPT * RPW) {
      uint4 raw[2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int h = h0 + b * WPT * RPW + first;
        raw[b] = h < H ? src[(base + h) * LPR + l] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int h = h0 + b * WPT * RPW + first;
        Row8 x = unpack8(raw[b]);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x.v[e], x.v[e], ss);
        const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x.v[e] = x.v[e] * r * w.v[e];
        const Row8 y = ang.turn(x, 1.f);
        if (h < H) dst[(base + h) * LPR + l] = pack8(y);
      }
    }
  }
}

// The backward: the same walk, tokens strided over a fixed grid so that each
// lane's share of dw stays in registers; a CTA's partial sums go to p.part and
// norm_rope_dw_kernel adds them in a fixed order (no atomics: the result does
// not depend on timing).  Rows of padding tokens get zero gradients.
template <int D, bool INTER, int TOK>
__global__ void __launch_bounds__(kThreads)
    norm_rope_bwd_kernel(const __grid_constant__ NRParams p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, WPT = kWarps / TOK;
  __shared__ float2 tab[TOK][64];
  __shared__ float red[kWarps * RPW][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u = warp / WPT;
  const int first = (warp % WPT) * RPW + lane / LPR, l = lane % LPR;
  float dw[2][8];
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[which][e] = 0.f;

  for (int t0 = blockIdx.x * TOK; t0 < p.T; t0 += gridDim.x * TOK) {
    __syncthreads();
    fill_table<TOK>(p, t0, tab);
    __syncthreads();
    const int t = t0 + u;
    if (t >= p.T) continue;
    if (p.pos[t] < 0) {
#pragma unroll
      for (int which = 0; which < 2; ++which)
        for (int i = (warp % WPT) * 32 + lane; i < p.H[which] * LPR; i += WPT * 32)
          reinterpret_cast<uint4*>(p.out[which])[static_cast<int64_t>(t) * p.H[which] * LPR + i] =
              make_uint4(0, 0, 0, 0);
      continue;
    }
    Angles<LPR, INTER> ang;
    ang.load(tab[u], p.half, lane);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const int H = p.H[which];
      Row8 w;
#pragma unroll
      for (int e = 0; e < 8; ++e) w.v[e] = 1.f;
      if (p.w[which] != nullptr) w = unpack8(reinterpret_cast<const uint4*>(p.w[which])[l]);
      const int64_t base = static_cast<int64_t>(t) * H;
      for (int h0 = 0; h0 < H; h0 += WPT * RPW) {
        const int h = h0 + first;
        const bool on = h < H;
        const int64_t at = (base + h) * LPR + l;
        const uint4 xr = on ? reinterpret_cast<const uint4*>(p.x[which])[at] : make_uint4(0, 0, 0, 0);
        const uint4 gr = on ? reinterpret_cast<const uint4*>(p.dy[which])[at] : make_uint4(0, 0, 0, 0);
        Row8 x = unpack8(xr);
        const Row8 g = ang.turn(unpack8(gr), -1.f);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x.v[e], x.v[e], ss);
        const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x.v[e] *= r;  // n
          dot = fmaf(w.v[e] * g.v[e], x.v[e], dot);
          dw[which][e] = fmaf(g.v[e], x.v[e], dw[which][e]);
        }
        const float mean = row_sum<LPR>(dot) * (1.f / D);
        Row8 dx;
#pragma unroll
        for (int e = 0; e < 8; ++e) dx.v[e] = r * (w.v[e] * g.v[e] - x.v[e] * mean);
        if (on) reinterpret_cast<uint4*>(p.out[which])[at] = pack8(dx);
      }
    }
  }
  if (p.part == nullptr) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) red[warp * RPW + lane / LPR][8 * l + e] = dw[which][e];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < kWarps * RPW; ++j) s += red[j][d];
      p.part[(static_cast<int64_t>(blockIdx.x) * 2 + which) * D + d] = s;
    }
  }
}

// dw[which][d] = sum over the n partial rows, 32 columns per CTA.
__global__ void __launch_bounds__(256) norm_rope_dw_kernel(const float* part, int n, int D,
                                                           float* dwq, float* dwk) {
  griddep_wait();
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;  // column of the [2][D] rows
  float s = 0.f;
#pragma unroll 8
  for (int j = warp; j < n; j += 8) s += part[static_cast<int64_t>(j) * 2 * D + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0) {
    s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += red[j][lane];
    float* dw = c < D ? dwq : dwk;
    if (dw != nullptr) dw[c < D ? c : c - D] = s;
  }
}

NRParams params_of(const NormRopeLaunch& a) {
  NRParams p{};
  p.x[0] = static_cast<const __nv_bfloat16*>(a.q);
  p.x[1] = static_cast<const __nv_bfloat16*>(a.k);
  p.w[0] = static_cast<const __nv_bfloat16*>(a.w_q);
  p.w[1] = static_cast<const __nv_bfloat16*>(a.w_k);
  p.dy[0] = static_cast<const __nv_bfloat16*>(a.dq_out);
  p.dy[1] = static_cast<const __nv_bfloat16*>(a.dk_out);
  p.out[0] = static_cast<__nv_bfloat16*>(a.q_out);
  p.out[1] = static_cast<__nv_bfloat16*>(a.k_out);
  p.pos = a.pos;
  p.T = a.T;
  p.H[0] = a.H_q;
  p.H[1] = a.H_k;
  p.half = a.rot / 2;
  p.eps = a.eps;
  for (int j = 0; j < p.half; ++j) {
    // inv_freq / (2 pi) modulo one turn, to 2^-64: 64 bits of mantissa
    long double turns = static_cast<long double>(a.inv_freq[j]) / 6.283185307179586476925286766559L;
    turns -= floorl(turns);
    const long double fixed = turns * 18446744073709551616.0L;
    p.turn[j] = fixed >= 18446744073709551615.0L ? 0 : static_cast<uint64_t>(fixed + 0.5L);
  }
  return p;
}

// Tokens per CTA: one while the tokens do not fill the SMs several times over
// (more warps on each token), else four (the cosines and sines of a token are
// then shared by two warps instead of eight).
bool few_tokens(int T) { return T < 8 * num_sms(); }

template <int D, bool INTER>
cudaError_t launch_fwd(const NormRopeLaunch& a, cudaStream_t s) {
  const NRParams p = params_of(a);
  prof_begin("norm_rope", s);
  if (few_tokens(a.T)) norm_rope_kernel<D, INTER, 1><<<a.T, kThreads, 0, s>>>(p);
  else norm_rope_kernel<D, INTER, 4><<<(a.T + 3) / 4, kThreads, 0, s>>>(p);
  prof_end(s);
  return cudaGetLastError();
}

int bwd_grid(int T) {
  const int tiles = few_tokens(T) ? T : (T + 3) / 4;
  const int most = num_sms() * 4;
  return tiles < most ? tiles : most;
}

template <int D, bool INTER>
cudaError_t launch_bwd(const NormRopeLaunch& a, cudaStream_t s) {
  NRParams p = params_of(a);
  p.part = a.dw_q != nullptr || a.dw_k != nullptr ? static_cast<float*>(a.ws) : nullptr;
  const int grid = bwd_grid(a.T);
  prof_begin("norm_rope_bwd", s);
  if (few_tokens(a.T)) norm_rope_bwd_kernel<D, INTER, 1><<<grid, kThreads, 0, s>>>(p);
  else norm_rope_bwd_kernel<D, INTER, 4><<<grid, kThreads, 0, s>>>(p);
  prof_end(s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.part == nullptr) return e;
  prof_begin("norm_rope_dw", s);
  e = launch_pdl(norm_rope_dw_kernel, dim3(2 * D / 32), dim3(256), 0, s,
                 static_cast<const float*>(p.part), grid, D, a.dw_q, a.dw_k);
  prof_end(s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t norm_rope_bwd_workspace_bytes(int T, int d) {
  return sizeof(float) * 2 * static_cast<size_t>(bwd_grid(T)) * d;
}

cudaError_t launch_norm_rope(const NormRopeLaunch& a, cudaStream_t s) {
  const bool bwd = a.dq_out != nullptr;
  auto go = [&](auto fwd_fn, auto bwd_fn) { return bwd ? bwd_fn(a, s) : fwd_fn(a, s); };
  switch (a.d * 2 + (a.interleaved ? 1 : 0)) {
    case 64: return go(launch_fwd<32, false>, launch_bwd<32, false>);
    case 65: return go(launch_fwd<32, true>, launch_bwd<32, true>);
    case 128: return go(launch_fwd<64, false>, launch_bwd<64, false>);
    case 129: return go(launch_fwd<64, true>, launch_bwd<64, true>);
    case 256: return go(launch_fwd<128, false>, launch_bwd<128, false>);
    case 257: return go(launch_fwd<128, true>, launch_bwd<128, true>);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace msa
