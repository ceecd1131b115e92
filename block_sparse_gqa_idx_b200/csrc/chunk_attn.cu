// chunk_attn.cu -- Eq. 8 for a chunk of new tokens on the paged FP8 cache:
// exact softmax attention of every row's query heads over the keys j <= pos
// of its selected blocks.
//
//   S = (q e4m3(k_j)) ks_j scale,  O = sum_j softmax(S)_j vs_j e4m3(v_j)
//
// Query-outer kernel: one CTA per (row, group, split of the row's keys), four
// warps that walk the row's 16-key groups independently; no barrier until the
// warps' states are joined at the end.
//   * Each warp has its own ring of 16-key stages in shared memory, filled by
//     asynchronous copies two stages ahead.  (Four and five stages, and four CTAs
//     per SM, are slower, 34, 37 and 34 us against 32 in the case below: more reads
//     of 128 bytes in flight do not help the memory.)
//   * Codes go from there into MMA fragments, widened to f16 in registers (exact),
//     so the tensor cores see the raw codes; a key's scale multiplies its scores, a
//     value's scale its weight.
//   * Both products are transposed so that the 16-row side of the MMA is keys
//     (S^T = K Q^T) or dimensions (O^T = V^T P^T) and the 8-column side the
//     group's heads: no row is padding at G = 8.  V^T pairs keys: two keys'
//     code words are interleaved by byte permutes before widening.
//   * P^T is S^T's accumulator layout transposed: one movmatrix per 8 keys.
//   * A query enters as f16 times a power of two per head (exact, as in the
//     scores kernel).
//   * Weights are kept relative to the largest weight-times-scale so far
//     (ref_y), apart from the softmax's own maximum (ref_x): P fits f16 for
//     any value scales.  Both references move only when a score passes them
//     by more than 2^10, so a step costs one vote instead of two reductions.
// Single tokens of 48 sequences at 16K (H_q = 32, H_kv = 4, d_h = B_k = 128, k = 16;
// 104 MB): 28 us, and 4 for the join of two splits; 3.7 TB/s.
#include "chunk_launch.h"

namespace msa {
namespace {

constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr float kSlack = 10.f;  // log2 of how far a weight may pass its reference

struct AttendParams {
  ChunkSeqs c;
  const __nv_bfloat16* q;  // [T, H_q, D]
  const int32_t* idx;      // [T, H_kv, k]
  const uint8_t* kp;       // [n_pages, B_k, H_kv, D]
  const uint8_t* vp;
  const float* ks;         // [n_pages, B_k, H_kv]
  const float* vs;
  __nv_bfloat16* o;
  float* lse;              // or null
  int H_q, H_kv, G, k;
  int nsplit;
  float scale_log2;
  float* part_o;           // [T, H_kv, nsplit, G, D] normalised, when nsplit > 1
  float* part_lse;         // [T, H_kv, nsplit, G] log2 of the sum
  DevStatus* status;
};

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// 8x8 b16 transpose across the warp (row lane/4, columns 2 (lane%4), +1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// a in the log2 domain, relative to a reference that may be -inf (no key yet).
__device__ __forceinline__ float rel(float a, float ref) {
  return a - (ref == -INFINITY ? 0.f : ref);
}

template <int D, int BK, int NH>
struct Attend {
  static constexpr int DT = D / 4;    // K codes per thread and key
  static constexpr int NU = DT / 16;  // their 16-byte loads
  static constexpr int VB = D / 8;    // V codes per thread and key
  static constexpr int VW = VB / 4;   // their 4-byte words
  static constexpr int NK = D / 16;   // MMAs along d
  static constexpr int MT = D / 16;   // m-tiles of O^T

  struct Raw {  // 16 keys
    uint4 k[2][NU];     // keys g, g + 8
    uint32_t v[4][VW];  // keys 2t, 2t + 1, 2t + 8, 2t + 9
    float ks[2], vs[2]; // keys g, g + 8
    int j0;             // position of the first key
  };

  uint32_t bq[NH][NK][2];
  float un[NH][2];             // scale of the raw dots of heads 2t, 2t + 1 (log2 domain)
  float o[NH][MT][4];
  // sums; the references of scores and of weights (0 before the first key), and
  // what a score or weight must pass for them to move
  float l[NH][2], rx[NH][2], ry[NH][2], tx[NH][2], ty[NH][2];

  __device__ __forceinline__ void load_q(const AttendParams& p, int64_t row, int r, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      const int h = 8 * n + g;
      const __nv_bfloat16* qr = p.q + (row * p.H_q + r * p.G + (h < p.G ? h : 0)) * D;
      float qv[NK][4], amax = 0.f;
#pragma unroll
      for (int j = 0; j < NK; ++j) {
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
      const int shift = amax > 0.f && amax < INFINITY ? min(13 - ilogbf(amax), 126) : 0;
      const float up = pow2(shift);
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        bq[n][j][0] = pack_f16(qv[j][0] * up, qv[j][1] * up);
        bq[n][j][1] = pack_f16(qv[j][2] * up, qv[j][3] * up);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int sh = __shfl_sync(0xFFFFFFFFu, shift, (2 * t + e) * 4);
        un[n][e] = p.scale_log2 * pow2(-sh);
        l[n][e] = 0.f;
        rx[n][e] = ry[n][e] = 0.f;
        tx[n][e] = ty[n][e] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
    }
  }

  // A stage: 16 keys' K rows, V rows, K scales, V scales.  16-byte chunks of a row
  // are permuted so that a fragment load meets no bank twice.
  static constexpr int STAGE = 32 * D + 128;
  static __device__ __forceinline__ int chunk(int key, int c) {
    return key * D + 16 * (D == 128 ? c ^ (key & 7) : c ^ ((key >> 1) & 3));
  }
  // What a lane copies of every stage, from the stage's first row on.
  struct Share {
    int dst[2];     // in the stage: the copies' two permutations
    int64_t src;    // byte of the first copy
    int64_t rows;   // bytes from a copy to the next
    int64_t scale;  // element
  };
  static constexpr int C = D / 16;  // chunks per row
  static __device__ __forceinline__ Share share(const AttendParams& p, int lane) {
    const int key = lane / C, c = lane % C;
    const int64_t row = static_cast<int64_t>(p.H_kv) * D;
    Share h;
    h.dst[0] = chunk(key, c);
    h.dst[1] = chunk(key + 32 / C, c) - D * 32 / C;
    h.src = key * row + 16 * c;
    h.rows = row * (32 / C);
    h.scale = static_cast<int64_t>(lane & 15) * p.H_kv;
    return h;
  }
  static __device__ __forceinline__ void fill(const AttendParams& p, const Share& h, uint8_t* st,
                                              int64_t row0, int lane) {
    const int64_t at = row0 * D + h.src;
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
      uint8_t* dst = st + h.dst[i & 1] + i * (D * 32 / C);
      copy16(dst, p.kp + (at + i * h.rows));
      copy16(dst + 16 * D, p.vp + (at + i * h.rows));
    }
    copy4(st + 32 * D + 4 * lane, (lane < 16 ? p.ks : p.vs) + (row0 + h.scale));
  }
  static __device__ __forceinline__ void load(Raw& x, const uint8_t* st, int j0, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const float* sc = reinterpret_cast<const float*>(st + 32 * D);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int u = 0; u < NU; ++u)
        x.k[e][u] = *reinterpret_cast<const uint4*>(st + chunk(g + 8 * e, t * NU + u));
      x.ks[e] = sc[g + 8 * e];
      x.vs[e] = sc[16 + g + 8 * e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int key = 2 * t + (e & 1) + 8 * (e >> 1);
      const uint8_t* src = st + 16 * D + chunk(key, g * VB / 16) + g * VB % 16;
      if constexpr (VW == 4) {
        const uint4 w = *reinterpret_cast<const uint4*>(src);
        x.v[e][0] = w.x;
        x.v[e][1] = w.y;
        x.v[e][2] = w.z;
        x.v[e][3] = w.w;
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(src);
        x.v[e][0] = w.x;
        x.v[e][1] = w.y;
      }
    }
    x.j0 = j0;
  }

  __device__ __forceinline__ void step(Raw& x, int pos, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float s[NH][4];
#pragma unroll
    for (int n = 0; n < NH; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
    for (int j = 0; j < NK; ++j) {
      const uint32_t w0 = reinterpret_cast<const uint32_t*>(x.k[0])[j];
      const uint32_t w1 = reinterpret_cast<const uint32_t*>(x.k[1])[j];
      const uint32_t a[4] = {widen2(w0), widen2(w1), widen2(w0 >> 16), widen2(w1 >> 16)};
#pragma unroll
      for (int n = 0; n < NH; ++n) mma_f16_16816(s[n], a, bq[n][j][0], bq[n][j][1]);
    }
    const float lv[2] = {log2f(fabsf(x.vs[0])), log2f(fabsf(x.vs[1]))};
    const bool cut = x.j0 + 15 > pos;  // warp-uniform: some of these keys come after the row
    float y[NH][4];
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] *= un[n][e & 1] * x.ks[e >> 1];
        y[n][e] = s[n][e] + lv[e >> 1];
        if (cut && x.j0 + g + 8 * (e >> 1) > pos) s[n][e] = y[n][e] = -INFINITY;
      }
    if (cut) {  // a key that is not seen may hold anything, NaN codes too
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (x.j0 + 2 * t + (e & 1) + 8 * (e >> 1) > pos)
#pragma unroll
          for (int w = 0; w < VW; ++w) x.v[e][w] = 0u;
    }
    bool pass = false;
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        pass = pass || s[n][e] > tx[n][e & 1] || y[n][e] > ty[n][e & 1];
    if (__any_sync(0xFFFFFFFFu, pass)) {
#pragma unroll
      for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool nox = tx[n][e] == -INFINITY, noy = ty[n][e] == -INFINITY;
          float mx = fmax3(nox ? -INFINITY : rx[n][e], s[n][e], s[n][e + 2]);
          float my = fmax3(noy ? -INFINITY : ry[n][e], y[n][e], y[n][e + 2]);
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) {
            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, w));
            my = fmaxf(my, __shfl_xor_sync(0xFFFFFFFFu, my, w));
          }
          tx[n][e] = mx + kSlack;
          ty[n][e] = my + kSlack;
          mx = mx == -INFINITY ? 0.f : mx;
          my = my == -INFINITY ? 0.f : my;
          // (before the first key there is nothing in the sums to scale)
          l[n][e] *= nox ? 1.f : exp2f(rx[n][e] - mx);
          const float f = noy ? 1.f : exp2f(ry[n][e] - my);
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            o[n][i][e] *= f;
            o[n][i][e + 2] *= f;
          }
          rx[n][e] = mx;
          ry[n][e] = my;
        }
    }
    uint32_t pb[NH][2];
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        l[n][e & 1] += ex2_ftz(s[n][e] - rx[n][e & 1]);
        w[e] = copysignf(ex2_ftz(y[n][e] - ry[n][e & 1]), x.vs[e >> 1]);
      }
      pb[n][0] = transpose8(pack_f16(w[0], w[1]));
      pb[n][1] = transpose8(pack_f16(w[2], w[3]));
    }
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      const uint32_t lo01 = __byte_perm(x.v[0][w], x.v[1][w], 0x5140);
      const uint32_t lo23 = __byte_perm(x.v[2][w], x.v[3][w], 0x5140);
      const uint32_t hi01 = __byte_perm(x.v[0][w], x.v[1][w], 0x7362);
      const uint32_t hi23 = __byte_perm(x.v[2][w], x.v[3][w], 0x7362);
      const uint32_t a0[4] = {widen2(lo01), widen2(lo01 >> 16), widen2(lo23), widen2(lo23 >> 16)};
      const uint32_t a1[4] = {widen2(hi01), widen2(hi01 >> 16), widen2(hi23), widen2(hi23 >> 16)};
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        mma_f16_16816(o[n][2 * w], a0, pb[n][0], pb[n][1]);
        mma_f16_16816(o[n][2 * w + 1], a1, pb[n][0], pb[n][1]);
      }
    }
  }
};

template <int D, int NH>
constexpr int kHeld = D == 128 ? (NH == 1 ? 3 : 2) : (NH == 1 ? 4 : 3);  // CTAs per SM
template <int D, int BK, int NH>
__global__ void __launch_bounds__(kWarps * 32, kHeld<D, NH>) chunk_attend_kernel(const AttendParams p) {
  using A = Attend<D, BK, NH>;
  constexpr int HEADS = 8 * NH;
  constexpr int GPB = BK / 16;  // 16-key groups per block
  extern __shared__ __align__(128) uint8_t smem[];
  float (*so)[HEADS][D] = reinterpret_cast<float (*)[HEADS][D]>(smem);  // once the rings are done
  __shared__ float sl[kWarps][HEADS], sx[kWarps][HEADS], sy[kWarps][HEADS];
  __shared__ int2 slots[32];  // (page, block) of the row's usable slots
  __shared__ int n_full, n_own;  // other blocks, and the own one as often as it is listed

  const int sp = blockIdx.x % p.nsplit;
  const int64_t unit = blockIdx.x / p.nsplit;  // (row, group)
  const int row = static_cast<int>(unit / p.H_kv);
  const int r = static_cast<int>(unit - static_cast<int64_t>(row) * p.H_kv);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const ChunkTok tok = chunk_tok(p.c, row);
  if (tok.pos < 0) {
    if (tok.too_long && threadIdx.x == 0) report(p.status, DEV_ERR_CACHE_FULL, 130, tok.s, row);
    return;
  }
  if (warp == 0) {
    int b = lane < p.k ? __ldg(p.idx + unit * p.k + lane) : -1;
    if (b < -1 || b >= p.c.max_pages) {
      report(p.status, DEV_ERR_BAD_INDEX, 131, row, b);
      b = -1;
    }
    int64_t pg = -1;
    if (b >= 0 && b <= tok.pos / BK) {
      pg = chunk_page(p.c, tok.s, b);
      if (pg < 0) report(p.status, DEV_ERR_BAD_INDEX, 132, tok.s, b);
    }
    // the row's own block behind the others: the keys after the row are its last
    const bool last = pg >= 0 && b == tok.pos / BK;
    const unsigned use = __ballot_sync(0xFFFFFFFFu, pg >= 0 && !last);
    const unsigned end = __ballot_sync(0xFFFFFFFFu, last);
    const unsigned before = (1u << lane) - 1;
    if (pg >= 0)
      slots[last ? __popc(use) + __popc(end & before) : __popc(use & before)] =
          make_int2(static_cast<int>(pg), b);
    if (lane == 0) {
      n_full = __popc(use);
      n_own = __popc(end);
    }
  }
  A a;
  a.load_q(p, row, r, lane);
  __syncthreads();
  const int full = n_full * GPB, own = (tok.pos % BK) / 16 + 1;  // groups with keys of the row
  const int total = full + n_own * own;
  const int stride = p.nsplit * kWarps;
  uint8_t* ring = smem + warp * kStages * A::STAGE;
  const typename A::Share mine = A::share(p, lane);
  int ahead = sp * kWarps + warp;
  int j0[kStages - 1];  // first keys of the groups on their way
  auto fetch = [&](int stage) {
    int first = 0;
    if (ahead < total) {
      int slot = ahead / GPB, group = ahead % GPB;
      if (ahead >= full) {
        slot = (ahead - full) / own;
        group = ahead - full - slot * own;
        slot += n_full;
      }
      const int2 block = slots[slot];
      const int64_t key = static_cast<int64_t>(block.x) * BK + group * 16;
      A::fill(p, mine, ring + stage * A::STAGE, key * p.H_kv + r, lane);
      first = block.y * BK + group * 16;
    }
    ahead += stride;
    asm volatile("cp.async.commit_group;" ::: "memory");
    return first;
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) j0[s] = fetch(s);
  int stage = 0;
  for (int i = sp * kWarps + warp; i < total; i += stride) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();  // and all lanes have read the stage that is filled next
    const int now = j0[0];
#pragma unroll
    for (int s = 0; s + 2 < kStages; ++s) j0[s] = j0[s + 1];
    j0[kStages - 2] = fetch(stage == 0 ? kStages - 1 : stage - 1);
    typename A::Raw x;
    A::load(x, ring + stage * A::STAGE, now, lane);
    a.step(x, tok.pos, lane);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  __syncthreads();

  // join the four warps' states
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NH; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int h = 8 * n + 2 * t + e;
      float l = a.l[n][e];
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, w);
      if (g == 0) {
        sl[warp][h] = l;
        sx[warp][h] = a.tx[n][e] == -INFINITY ? -INFINITY : a.rx[n][e];
        sy[warp][h] = a.ty[n][e] == -INFINITY ? -INFINITY : a.ry[n][e];
      }
#pragma unroll
      for (int m = 0; m < A::MT; ++m)
        *reinterpret_cast<float2*>(&so[warp][h][g * A::VB + 2 * m]) =
            make_float2(a.o[n][m][e], a.o[n][m][e + 2]);
    }
  __syncthreads();
  for (int it = threadIdx.x; it < HEADS * (D / 8); it += kWarps * 32) {
    const int h = it / (D / 8), d = (it - h * (D / 8)) * 8;
    if (h >= p.G) break;
    float X = -INFINITY, Y = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      X = fmaxf(X, sx[w][h]);
      Y = fmaxf(Y, sy[w][h]);
    }
    float L = 0.f, acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      L += sl[w][h] * exp2f(rel(sx[w][h], X));
      const float f = exp2f(rel(sy[w][h], Y));
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(so[w][h][d + e], f, acc[e]);
    }
    // L is 0 only where no key was seen; a NaN goes through.  Y is -inf where
    // every value scale is zero: O is zero then.
    float lse2 = -INFINITY, norm = 0.f;
    if (L != 0.f) {
      lse2 = X + log2f(L);
      norm = Y == -INFINITY ? L * 0.f : exp2f(Y - X) / L;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= norm;
    if (p.nsplit == 1) {
      const int64_t at = static_cast<int64_t>(row) * p.H_q + r * p.G + h;
      *reinterpret_cast<uint4*>(p.o + at * D + d) =
          make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]),
                     pack_bf16(acc[4], acc[5]), pack_bf16(acc[6], acc[7]));
      if (d == 0 && p.lse != nullptr) p.lse[at] = lse2 * 0.6931471805599453f;
    } else {
      const int64_t at = (unit * p.nsplit + sp) * p.G + h;
      float4* dst = reinterpret_cast<float4*>(p.part_o + at * D + d);
      dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (d == 0) p.part_lse[at] = lse2;
    }
  }
}

// Join of a row's splits: one warp per (row, head), lane s weighs split s.
template <int D>
__global__ void __launch_bounds__(256) chunk_join_kernel(const AttendParams p) {
  griddep_wait();
  constexpr int PER = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (w >= static_cast<int64_t>(p.c.T) * p.H_q) return;
  const int row = static_cast<int>(w / p.H_q);
  const int head = static_cast<int>(w - static_cast<int64_t>(row) * p.H_q);
  if (chunk_tok(p.c, row).pos < 0) return;
  const int r = head / p.G, h = head - r * p.G;
  const int64_t base = (static_cast<int64_t>(row) * p.H_kv + r) * p.nsplit * p.G + h;
  const float z = lane < p.nsplit ? p.part_lse[base + static_cast<int64_t>(lane) * p.G] : -INFINITY;
  float m = z;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const float wt = exp2f(rel(z, m));
  float sum = wt;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  float acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  for (int s = 0; s < p.nsplit; ++s) {
    const float ws = __shfl_sync(0xFFFFFFFFu, wt, s);
    const float* src = p.part_o + (base + static_cast<int64_t>(s) * p.G) * D + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = fmaf(ws, src[e], acc[e]);
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat16* dst = p.o + w * D + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(dst + e) = __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && p.lse != nullptr)
    p.lse[w] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
}

// Splits of a row's keys: what ends first when a round of CTAs (as many as the SMs
// hold) takes a warp's share of the 16-key groups and about four groups' time to
// begin with, and a join costs as much again.  At least one group for every warp.
// 48 rows of four groups, k = 16, B_k = 128, on 148 SMs: two splits 35 us, three
// (a round and a third) 44, four 40, six 44.
int splits_of(int T, int H_q, int H_kv, int B_k, int d_h, int k) {
  const int64_t units = static_cast<int64_t>(T) * H_kv;
  const int64_t held = static_cast<int64_t>(num_sms()) *
                       (H_q / H_kv <= 8 ? (d_h == 128 ? kHeld<128, 1> : kHeld<64, 1>)
                                        : (d_h == 128 ? kHeld<128, 2> : kHeld<64, 2>));
  const int steps = k * B_k / 16 / kWarps;
  int best = 1;
  int64_t cost = 0;
  for (int n = 1; n <= 32 && n <= steps; ++n) {
    const int64_t c = (units * n + held - 1) / held * ((steps + n - 1) / n + 4) + (n > 1 ? 4 : 0);
    if (n == 1 || c < cost) {
      best = n;
      cost = c;
    }
  }
  return best;
}

template <int D, int BK, int NH>
cudaError_t launch_attend(const AttendParams& p, unsigned grid, cudaStream_t s) {
  constexpr int ring = kWarps * kStages * Attend<D, BK, NH>::STAGE;
  static_assert(ring >= kWarps * 8 * NH * D * 4 && kHeld<D, NH> * (ring + 2048) <= 227 * 1024,
                "the states to join, and the CTAs an SM holds");
  const cudaError_t e = cudaFuncSetAttribute(chunk_attend_kernel<D, BK, NH>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, ring);
  if (e != cudaSuccess) return e;
  chunk_attend_kernel<D, BK, NH><<<grid, kWarps * 32, ring, s>>>(p);
  return cudaGetLastError();
}

template <int D, int BK>
cudaError_t launch_direct(const AttendLaunch& a, cudaStream_t s) {
  AttendParams p{};
  p.c = a.c;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.idx = a.idx;
  p.kp = static_cast<const uint8_t*>(a.k_pages);
  p.vp = static_cast<const uint8_t*>(a.v_pages);
  p.ks = a.k_scale;
  p.vs = a.v_scale;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.H_q = a.H_q;
  p.H_kv = a.H_kv;
  p.G = a.H_q / a.H_kv;
  p.k = a.k;
  p.nsplit = splits_of(a.c.T, a.H_q, a.H_kv, a.c.B_k, D, a.k);
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.status = a.status;
  const int64_t units = static_cast<int64_t>(a.c.T) * a.H_kv;
  p.part_o = static_cast<float*>(a.ws);
  p.part_lse = reinterpret_cast<float*>(
      static_cast<uint8_t*>(a.ws) + align256(sizeof(float) * units * p.nsplit * p.G * D));
  const unsigned grid = static_cast<unsigned>(units * p.nsplit);
  prof_begin("chunk_attend", s);
  cudaError_t e = p.G <= 8 ? launch_attend<D, BK, 1>(p, grid, s) : launch_attend<D, BK, 2>(p, grid, s);
  prof_end(s);
  if (e != cudaSuccess || p.nsplit == 1) return e;
  const int64_t threads = static_cast<int64_t>(a.c.T) * a.H_q * 32;
  prof_begin("chunk_join", s);
  e = launch_pdl(chunk_join_kernel<D>, dim3(static_cast<unsigned>((threads + 255) / 256)),
                 dim3(256), 0, s, p);
  prof_end(s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Which form.  The query-outer kernel's time is the bytes of the selected pages as
// every row reads them (through L2).  The KV-outer form costs about 30 us of short
// kernels, and a tile for each page and up to 16 of the rows that chose it (8 when
// G = 16), full or not.  It pays from about 2^28 values on, and where sequences have
// many rows, so that rows share pages: 24 on average, as far as the host knows.
// Query-outer : KV-outer, us, with H_q = 32, H_kv = 4, d_h = B_k = 128, k = 16 unless
// said, and selections scattered over the context but for its first and last blocks:
//   size       one sequence at 9K / four at 9K / one at 61K: 128 rows 53 : 46 /
//              54 : 56 / 54 : 83, 256 rows (2^28) 93 : 51 / 95 : 74 / 95 : 87, 512 rows
//              151 : 76 / 153 : 107 / 152 : 127.  2^27 values are not enough: H_q = 8,
//              H_kv = 2, 256 rows 52 : 38 / 53 : 48 / 52 : 52, but at 128K 57 : 79, and
//              H_kv = 8, B_k = 64, k = 8, 256 rows at 9K / 61K 56 : 64 / 59 : 174.
//              (G = 16, one sequence at 9K: 64, 128, 256 rows 38 : 44, 69 : 53, 120 : 80.)
//   rows       single tokens of 64, 256, 512 sequences 45 : 188, 123 : 574, 195 : 1088.
//              64 chunks of 16, 24, 32 rows 296 : 461, 437 : 512, 578 : 543; one long
//              chunk beside 63 single tokens, as many rows 297 : 277, 437 : 314, 577 : 362.
//   context    one sequence at 128K / 1M: 256 rows 96 : 154 / 112 : 379, 1024 rows
//              293 : 220 / 331 : 775, 4096 rows 1190 : 462 / 1429 : 997.  Not in the rule:
//              only the device knows it, and a table may be far wider than it.
//   table      four sequences of 128 rows, 256, 1024, 8192 entries each: 152 : 87, 97, 106.
constexpr int64_t kShareRows = 24;
static bool kv_outer(const msa::ChunkSeqs& c, int H_q, int H_kv, int d_h, int k) {
  const int G = H_q / H_kv;
  if (16 % G != 0 || (G < 8 && H_q % 8 != 0)) return false;  // its MMA rows and TMA boxes
  if (static_cast<int64_t>(c.S) * c.max_pages * H_kv >= (int64_t(1) << 30)) return false;  // keys
  if (c.n_pages * c.B_k >= (int64_t(1) << 31)) return false;  // TMA row coordinates
  if (c.T < kShareRows * c.S) return false;
  return static_cast<int64_t>(c.T) * H_kv * k * c.B_k * d_h >= (int64_t(1) << 28);
}

size_t chunk_attend_workspace_bytes(const ChunkSeqs& c, int H_q, int H_kv, int d_h, int k) {
  if (c.T == 0) return 0;
  if (kv_outer(c, H_q, H_kv, d_h, k))
    return chunk_attend_kv_workspace_bytes(c.T, c.S, c.max_pages, H_q, H_kv, d_h, k);
  const int n = splits_of(c.T, H_q, H_kv, c.B_k, d_h, k);
  if (n == 1) return 0;
  const size_t rows = static_cast<size_t>(c.T) * H_q * n;
  return align256(sizeof(float) * rows * d_h) + align256(sizeof(float) * rows);
}

cudaError_t launch_chunk_attend(const AttendLaunch& a, cudaStream_t s) {
  if (kv_outer(a.c, a.H_q, a.H_kv, a.d_h, a.k)) return launch_chunk_attend_kv(a, s);
  if (a.d_h == 128)
    return a.c.B_k == 128 ? launch_direct<128, 128>(a, s) : launch_direct<128, 64>(a, s);
  return a.c.B_k == 128 ? launch_direct<64, 128>(a, s) : launch_direct<64, 64>(a, s);
}

}  // namespace msa
