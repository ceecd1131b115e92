// norm_rope.cu -- RMS normalisation of every query and key head, then the
// position rotation, in one pass over the rows (forward), and its backward.
//
//   n = x / sqrt(mean(x^2) + eps),  y = R(pos) (w * n)
//   R rotates the pairs (j, j + rot/2) -- or (2j, 2j + 1), interleaved -- by
//   the angle pos * inv_freq[j], j < rot/2; dimensions rot .. d-1 pass through.
// Backward, with g = R(pos)^T dy:
//   dw = sum over rows of g * n,  dx = (w g - n mean(w g n)) / sqrt(mean(x^2) + eps)
//
// Both are bound by the bytes of the rows.  A row (one head of one token) is
// read once by d/8 lanes and stays in registers.  A lane holds four dimensions and
// the four that they rotate with (rows' halves are read as 8-byte pieces, whole
// 128-byte lines of a row together), so that turning needs no exchange and only
// the sums are shuffle reductions.  A warp takes the rows of one token, several
// loads in flight, and computes that token's cosines and sines itself while the
// first rows are on their way: no barrier.  The angle never loses its far
// positions: inv_freq is held as a fraction of a turn in 64-bit fixed point, so
// pos * turn modulo 2^64 is the exact fractional turn, and sincospi sees at most
// half a turn.
// 32768 tokens of 32 + 4 heads of 128: 107 us forward (5.6 TB/s), 186 us
// backward (4.9 TB/s, of it 11 for the weights' last sum).
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

// A lane's share of a row: dimensions d0 .. d0+3 and d1 .. d1+3.
struct Row8 {
  float v[8];
};
struct Raw8 {
  uint2 a, b;
};

__device__ __forceinline__ Row8 unpack8(const Raw8& u) {
  Row8 r;
  const uint32_t w[4] = {u.a.x, u.a.y, u.b.x, u.b.y};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[e]));
    r.v[2 * e] = f.x;
    r.v[2 * e + 1] = f.y;
  }
  return r;
}

// Sums over the LPR lanes that hold one row.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// Where a lane's dimensions are and the angles of its pairs: (d0 + e, d1 + e), or
// the neighbours of d0 .. d0+7 when interleaved.  The first rot/8 lanes of a row
// rotate; the others' dimensions follow behind rot and pass (cos 1, sin 0).
template <int LPR, bool INTER>
struct Lane {
  int d0, d1;
  float cs[4], sn[4];

  __device__ __forceinline__ Lane(int half, int l) {
    d0 = 8 * l;
    d1 = d0 + 4;
    if (!INTER && l < half / 4) {
      d0 = 4 * l;
      d1 = d0 + half;
    }
  }
  // The token's angles, by way of `tab` (the warp's own).
  __device__ __forceinline__ void angles(const NRParams& p, int pos, float2* tab, int lane) {
    for (int j = lane; j < p.half; j += 32) {
      const uint64_t frac = static_cast<uint64_t>(static_cast<int64_t>(pos)) * p.turn[j];
      float s, c;  // frac as a signed fraction of half a turn
      sincospif(static_cast<float>(static_cast<int64_t>(frac)) * 0x1p-63f, &s, &c);
      tab[j] = make_float2(c, s);
    }
    __syncwarp();
    const int j0 = 4 * (lane % LPR);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = j0 < p.half ? tab[j0 + e] : make_float2(1.f, 0.f);
      cs[e] = a.x;
      sn[e] = a.y;
    }
    __syncwarp();
  }
  // y = R x (sgn = 1) or R^T x (sgn = -1)
  __device__ __forceinline__ Row8 turn(const Row8& x, float sgn) const {
    Row8 y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = INTER ? 2 * e : e, j = INTER ? 2 * e + 1 : e + 4;
      const float a = x.v[i], b = x.v[j], s = sgn * sn[e];
      y.v[i] = a * cs[e] - b * s;
      y.v[j] = b * cs[e] + a * s;
    }
    return y;
  }
  template <int D>
  __device__ __forceinline__ Raw8 load(const __nv_bfloat16* x, int64_t row) const {
    const __nv_bfloat16* at = x + row * D;
    return {__ldcs(reinterpret_cast<const uint2*>(at + d0)),
            __ldcs(reinterpret_cast<const uint2*>(at + d1))};
  }
  __device__ __forceinline__ Row8 weight(const __nv_bfloat16* w) const {
    Row8 r;
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = 1.f;
    if (w != nullptr)
      r = unpack8({__ldg(reinterpret_cast<const uint2*>(w + d0)),
                   __ldg(reinterpret_cast<const uint2*>(w + d1))});
    return r;
  }
  template <int D>
  __device__ __forceinline__ void store(__nv_bfloat16* y, int64_t row, const Row8& r) const {
    __nv_bfloat16* at = y + row * D;
    *reinterpret_cast<uint2*>(at + d0) =
        make_uint2(pack_bf16(r.v[0], r.v[1]), pack_bf16(r.v[2], r.v[3]));
    *reinterpret_cast<uint2*>(at + d1) =
        make_uint2(pack_bf16(r.v[4], r.v[5]), pack_bf16(r.v[6], r.v[7]));
  }
};

// TOK tokens per CTA, kWarps / TOK warps on each; a warp takes 32 / LPR rows at a
// time.  Rows of a token with pos < 0 (padding) are left untouched.
template <int D, bool INTER, int TOK>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NRParams p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, WPT = kWarps / TOK;
  constexpr int U = TOK == 1 ? 1 : 4;  // loads in flight
  constexpr int STEP = WPT * RPW;
  __shared__ float2 tab[kWarps][64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * TOK + warp / WPT;
  if (t >= p.T) return;
  const int pos = __ldg(p.pos + t);
  if (pos < 0) return;
  Lane<LPR, INTER> ln(p.half, lane % LPR);
  const int first = (warp % WPT) * RPW + lane / LPR;
  bool have = false;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int H = p.H[which];
    const int64_t base = static_cast<int64_t>(t) * H;
    const Row8 w = ln.weight(p.w[which]);
    // whole warps stay in the loop (shuffles)
    for (int h0 = 0; h0 < H; h0 += U * STEP) {
      Raw8 raw[U];
#pragma unroll
      for (int b = 0; b < U; ++b) {
        const int h = h0 + b * STEP + first;
        raw[b] = ln.template load<D>(p.x[which], base + (h < H ? h : 0));
      }
      if (!have) {
        ln.angles(p, pos, tab[warp], lane);
        have = true;
      }
#pragma unroll
      for (int b = 0; b < U; ++b) {
        const int h = h0 + b * STEP + first;
        if (h0 + b * STEP >= H) break;
        Row8 x = unpack8(raw[b]);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x.v[e], x.v[e], ss);
        const float r = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < 8; ++e) x.v[e] = x.v[e] * r * w.v[e];
        const Row8 y = ln.turn(x, 1.f);
        if (h < H) ln.template store<D>(p.out[which], base + h, y);
      }
    }
  }
}

// The backward: the same walk, tokens strided over a fixed grid so that each
// lane's share of dw stays in registers; a CTA's partial sums go to p.part and
// norm_rope_dw_kernel adds them in a fixed order (no atomics: the result does
// not depend on timing).  Rows of padding tokens get zero gradients.
template <int D, bool INTER, int TOK>
__global__ void __launch_bounds__(kThreads, 3)
    norm_rope_bwd_kernel(const __grid_constant__ NRParams p) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, WPT = kWarps / TOK;
  constexpr int U = TOK == 1 ? 1 : 2;
  constexpr int STEP = WPT * RPW;
  __shared__ float2 tab[kWarps][64];
  __shared__ float red[kWarps * RPW][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int first = (warp % WPT) * RPW + lane / LPR;
  Lane<LPR, INTER> ln(p.half, lane % LPR);
  float dw[2][8];
#pragma unroll
  for (int which = 0; which < 2; ++which)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[which][e] = 0.f;

  for (int t = blockIdx.x * TOK + warp / WPT; t < p.T; t += gridDim.x * TOK) {
    const int pos = __ldg(p.pos + t);
    if (pos < 0) {
#pragma unroll
      for (int which = 0; which < 2; ++which)
        for (int i = (warp % WPT) * 32 + lane; i < p.H[which] * LPR; i += WPT * 32)
          reinterpret_cast<uint4*>(p.out[which])[static_cast<int64_t>(t) * p.H[which] * LPR + i] =
              make_uint4(0, 0, 0, 0);
      continue;
    }
    bool have = false;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const int H = p.H[which];
      const int64_t base = static_cast<int64_t>(t) * H;
      const Row8 w = ln.weight(p.w[which]);
      for (int h0 = 0; h0 < H; h0 += U * STEP) {
        Raw8 xr[U], gr[U];
#pragma unroll
        for (int b = 0; b < U; ++b) {
          const int h = h0 + b * STEP + first;
          const int64_t row = base + (h < H ? h : 0);
          xr[b] = ln.template load<D>(p.x[which], row);
          gr[b] = ln.template load<D>(p.dy[which], row);
        }
        if (!have) {
          ln.angles(p, pos, tab[warp], lane);
          have = true;
        }
#pragma unroll
        for (int b = 0; b < U; ++b) {
          const int h = h0 + b * STEP + first;
          if (h0 + b * STEP >= H) break;
          const bool on = h < H;
          const Row8 x = unpack8(xr[b]);
          Row8 g = ln.turn(unpack8(gr[b]), -1.f);
          float ss = 0.f, dot = 0.f;  // of x, and of w g with x
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ss = fmaf(x.v[e], x.v[e], ss);
            dot = fmaf(w.v[e] * g.v[e], x.v[e], dot);
          }
          ss = row_sum<LPR>(ss);
          dot = row_sum<LPR>(dot);
          const float r = rsqrtf(ss * (1.f / D) + p.eps);
          const float mean = dot * r * (1.f / D);
          Row8 dx;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float n = x.v[e] * r;
            if (on) dw[which][e] = fmaf(g.v[e], n, dw[which][e]);
            dx.v[e] = r * (w.v[e] * g.v[e] - n * mean);
          }
          if (on) ln.template store<D>(p.out[which], base + h, dx);
        }
      }
    }
  }
  if (p.part == nullptr) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e)
      red[warp * RPW + lane / LPR][(e < 4 ? ln.d0 : ln.d1 - 4) + e] = dw[which][e];
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
    long double turns = static_cast<long double>(a.inv_freq[j]) * 0.15915494309189533576888L;
    if (!(turns >= 0.0L && turns < 1.0L)) turns -= floorl(turns);
    const long double fixed = turns * 18446744073709551616.0L;
    p.turn[j] = fixed >= 18446744073709551615.0L ? 0 : static_cast<uint64_t>(fixed + 0.5L);
  }
  return p;
}

// Tokens per CTA: one while the tokens do not fill the SMs several times over
// (eight warps on each), else eight.
bool few_tokens(int T) { return T < 8 * num_sms(); }

template <int D, bool INTER>
cudaError_t launch_fwd(const NormRopeLaunch& a, cudaStream_t s) {
  const NRParams p = params_of(a);
  prof_begin("norm_rope", s);
  if (few_tokens(a.T)) norm_rope_kernel<D, INTER, 1><<<a.T, kThreads, 0, s>>>(p);
  else norm_rope_kernel<D, INTER, 8><<<(a.T + 7) / 8, kThreads, 0, s>>>(p);
  prof_end(s);
  return cudaGetLastError();
}

int bwd_grid(int T) {
  const int tiles = few_tokens(T) ? T : (T + 7) / 8;
  const int most = num_sms() * 3;
  return tiles < most ? tiles : most;
}

template <int D, bool INTER>
cudaError_t launch_bwd(const NormRopeLaunch& a, cudaStream_t s) {
  NRParams p = params_of(a);
  p.part = a.dw_q != nullptr || a.dw_k != nullptr ? static_cast<float*>(a.ws) : nullptr;
  const int grid = bwd_grid(a.T);
  prof_begin("norm_rope_bwd", s);
  if (few_tokens(a.T)) norm_rope_bwd_kernel<D, INTER, 1><<<grid, kThreads, 0, s>>>(p);
  else norm_rope_bwd_kernel<D, INTER, 8><<<grid, kThreads, 0, s>>>(p);
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
