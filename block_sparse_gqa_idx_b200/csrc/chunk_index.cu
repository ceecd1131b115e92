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

// Bulk (untiled) copy global -> shared, counted on an mbarrier.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
// D (TMEM) [+]= A B, E4M3 operands in shared memory, K = 32.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

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
      const int shift = amax > 0.f && amax < INFINITY ? min(13 - ilogbf(amax), 126) : 0;
      const float up = pow2(shift);
#pragma unroll
      for (int j = 0; j < NMMA; ++j) {
        const __half2 lo = __floats2half2_rn(qv[j][0] * up, qv[j][1] * up);
        const __half2 hi = __floats2half2_rn(qv[j][2] * up, qv[j][3] * up);
        bq[n][j][0] = *reinterpret_cast<const uint32_t*>(&lo);
        bq[n][j][1] = *reinterpret_cast<const uint32_t*>(&hi);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int sh = __shfl_sync(0xFFFFFFFFu, shift, (2 * t + e) * 4);
        unscale[n][e] = p.idx_scale * pow2(-sh);
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

// ---------------------------------------------- scores on tcgen05, many rows --
// For chunks with many rows: 256 rows (two UMMA M-tiles) against 128 keys at a
// time, both in FP8: the codes go from their page by TMA straight into the
// MMA's layout, and the queries are split into two E4M3 terms.  A row is scaled
// by a power of two that puts its largest magnitude in [224, 448]; hi =
// E4M3(x), lo = E4M3(x - hi) hold its 8 bits exactly down to 2^-10 of the
// largest, and every element to 2^-18 of it.  hi and lo accumulate into the
// same fp32 accumulators, so a tile costs what one bf16 product of the same
// shape would.
//   warp 0      page lookups, TMA of codes and of the keys' scales
//   warp 1      MMAs, TMEM (two stages x two M-tiles x 128 columns)
//   warps 4-7   the next unit's queries into hi and lo tiles
//   warps 8-15  epilogue: two groups of four take the even and the odd key
//               tiles; a thread has the same TMEM lane of both M-tiles, so a
//               key's scale, read from shared memory as a broadcast, serves
//               two rows; maxima wait in shared memory and leave eight tiles at
//               a time, a row's values side by side.
// A unit is (256 rows, CT key tiles); units are dealt out to one CTA per SM.
// Rows of several sequences in one unit are taken one sequence after another
// against the same query tiles.
constexpr int kTcThreads = 512;
constexpr int kRows = 256;   // rows per unit
constexpr int kKeys = 128;   // keys per tile
constexpr int kFlush = 8;    // tiles of a group between flushes

struct TcParams {
  ScoreParams s;
  int rows;     // T * H_kv
  int CT;       // key tiles per unit
  int nchunk;   // units per 256 rows
  int n_units;
};

template <int D, int BK>
struct TcShape {
  static constexpr int BPT = kKeys / BK;            // blocks per key tile
  static constexpr int A_BYTES = kRows * D;         // hi (or lo) of a unit's rows
  static constexpr int K_BYTES = kKeys * D;
  static constexpr int ST = D == 64 ? 6 : 3;        // key tiles in flight
  static constexpr uint32_t SWZ = D == 64 ? SW_64B : SW_128B;
  static constexpr int SBO = 8 * D;                 // 8 rows
  static constexpr int OUT = kFlush * BPT + 1;      // maxima per row (padded)
  static constexpr size_t SMEM = 1024 + 2 * 2 * A_BYTES + ST * (K_BYTES + kKeys * 4) +
                                 2 * kRows * OUT * 4 + 4 * kRows * 4 + ST * 4 +
                                 (2 * ST + 8) * 8 + 64;
  static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
};

// One sequence's rows of a unit.
struct TcItem {
  int s, ta;         // sequence, first token
  int pos;           // its position
  int own;           // the last token's own block
  int ra, rb;        // rows of the unit
  int k0, k1;        // key tiles to score
};

// Calls f for the items of unit u, in the same order in every role; stops when
// f returns false.  `tell`: report sequences that do not fit.
template <int BK, typename F>
__device__ __forceinline__ void for_items(const TcParams& p, int u, bool tell, F f) {
  constexpr int BPT = kKeys / BK;
  const ChunkSeqs& c = p.s.c;
  const int H = p.s.H_kv, m = u / p.nchunk, ch = u - m * p.nchunk;
  const int R0 = m * kRows, R1 = min(R0 + kRows, p.rows);
  const int t_end = (R1 - 1) / H + 1;
  for (int t = R0 / H; t < t_end;) {
    const ChunkTok tok = chunk_tok(c, t);
    if (tok.pos < 0) {
      if (tell && tok.too_long) report(p.s.status, DEV_ERR_CACHE_FULL, 202, tok.s, t);
      ++t;
      continue;
    }
    const int te = min(t_end, __ldg(c.cu + tok.s + 1));
    TcItem it;
    it.own = (tok.pos + te - t - 1) / BK;
    it.s = tok.s;
    it.ta = t;
    it.pos = tok.pos;
    it.ra = max(R0, t * H) - R0;
    it.rb = min(R1, te * H) - R0;
    it.k0 = ch * p.CT;
    it.k1 = max(it.k0, min(it.k0 + p.CT, (it.own + BPT - 1) / BPT));
    if (!f(it)) return;
    t = te;
  }
}

template <int D, int BK>
__global__ void __launch_bounds__(kTcThreads, 1)
    chunk_scores_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const TcParams p) {
  using SH = TcShape<D, BK>;
  constexpr int ST = SH::ST, BPT = SH::BPT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;                          // [2] hi, lo of a unit's rows
  uint8_t* sK = sA + 2 * 2 * SH::A_BYTES;      // [ST] codes
  float* sS = reinterpret_cast<float*>(sK + ST * SH::K_BYTES);  // [ST][128] scales
  float* sOut = sS + ST * kKeys;               // [2 groups][256][OUT] maxima
  float* sRow = sOut + 2 * kRows * SH::OUT;    // [2] what a row's dots are multiplied with
  int* sOwn = reinterpret_cast<int*>(sRow + 2 * kRows);  // [2 groups][256] own blocks
  int* sOk = sOwn + 2 * kRows;  // [ST] bit b: block b of the tile has a page
  uint64_t* bars = reinterpret_cast<uint64_t*>(
      (reinterpret_cast<uintptr_t>(sOk + ST) + 7) & ~static_cast<uintptr_t>(7));
  uint64_t* k_full = bars;             // [ST]
  uint64_t* k_empty = k_full + ST;     // [ST] MMAs done and scales read
  uint64_t* a_full = k_empty + ST;     // [2]
  uint64_t* a_empty = a_full + 2;      // [2] MMAs done and row factors read
  uint64_t* acc_full = a_empty + 2;    // [2]
  uint64_t* acc_empty = acc_full + 2;  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const ChunkSeqs& c = p.s.c;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int j = 0; j < ST; ++j) {
      mbar_init(&k_full[j], 1);
      mbar_init(&k_empty[j], 5);  // the MMAs' commit and the group's four warps
    }
    for (int j = 0; j < 2; ++j) {
      mbar_init(&a_full[j], 4);
      mbar_init(&a_empty[j], 9);  // the MMAs' commit and the eight epilogue warps
      mbar_init(&acc_full[j], 1);
      mbar_init(&acc_empty[j], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp == 0) {
    // -------------------------------------------------------- producer --
    // Lane l holds the page of block l of a batch of 32, the next batch on its
    // way; lane 0 waits and issues.
    if (lane == 0) prefetch_tmap(&tm_k);
    uint32_t g = 0;
    bool ok = true;
    for (int u = blockIdx.x; ok && u < p.n_units; u += gridDim.x)
      for_items<BK>(p, u, true, [&](const TcItem& it) {
        const int b0 = it.k0 * BPT, b1 = min(it.k1 * BPT, c.max_pages);
        auto fetch = [&](int b) {
          if (b >= b1) return -1;
          const int pg = static_cast<int>(chunk_page(c, it.s, b));
          if (pg < 0 && b < it.own) report(p.s.status, DEV_ERR_BAD_INDEX, 201, it.s, b);
          return pg;
        };
        int mine = fetch(b0 + lane), next = fetch(b0 + 32 + lane);
        for (int kt = it.k0; ok && kt < it.k1; ++kt, ++g) {
          const int at = (kt - it.k0) * BPT % 32;
          if (at == 0 && kt > it.k0) {
            mine = next;
            next = fetch(kt * BPT + 32 + lane);
          }
          int pg[BPT], have = 0;
#pragma unroll
          for (int j = 0; j < BPT; ++j) {
            pg[j] = __shfl_sync(0xFFFFFFFFu, mine, at + j);
            have |= pg[j] >= 0 ? 1 << j : 0;
          }
          const int st = g % ST;
          ok = mbar_wait(&k_empty[st], ((g / ST) & 1) ^ 1, abort_flag, p.s.status, 200);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (ok && lane == 0) {
            sOk[st] = have;
            mbar_arrive_expect_tx(&k_full[st], __popc(have) * (BK * D + BK * 4));
#pragma unroll
            for (int j = 0; j < BPT; ++j)
              if (pg[j] >= 0) {
                const int row = pg[j] * BK;
                tma_load_2d(sK + st * SH::K_BYTES + j * BK * D, &tm_k, &k_full[st], 0, row);
                bulk_load(sS + st * kKeys + j * BK, p.s.scale + row, BK * 4, &k_full[st]);
              }
          }
        }
        return ok;
      });
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA --
    if (lane == 0) {
      // kind::f8f6f4, E4M3 x E4M3 -> f32, both K-major
      constexpr uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(kKeys >> 3) << 17) | (128u >> 4 << 24);
      const uint64_t a_desc = umma_desc(smem_u32(sA), 16, SH::SBO, SH::SWZ);
      const uint64_t k_desc = umma_desc(smem_u32(sK), 16, SH::SBO, SH::SWZ);
      uint32_t g = 0, ua = 0;
      bool ok = true;
      for (int u = blockIdx.x; ok && u < p.n_units; u += gridDim.x, ++ua) {
        const int ab = ua & 1;
        ok = mbar_wait(&a_full[ab], (ua >> 1) & 1, abort_flag, p.s.status, 210);
        if (!ok) break;
        const uint64_t ad0 = a_desc + ab * (2 * SH::A_BYTES >> 4);
        for_items<BK>(p, u, false, [&](const TcItem& it) {
          for (int kt = it.k0; ok && kt < it.k1; ++kt, ++g) {
            const int st = g % ST, acc = g & 1;
            ok = mbar_wait(&k_full[st], (g / ST) & 1, abort_flag, p.s.status, 211) &&
                 mbar_wait(&acc_empty[acc], ((g >> 1) & 1) ^ 1, abort_flag, p.s.status, 212);
            if (!ok) break;
            tc_fence_after();
            const uint64_t kd = k_desc + st * (SH::K_BYTES >> 4);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int term = 0; term < 2; ++term)
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                  umma_f8(tmem_base + acc * 256 + mt * 128,
                          ad0 + ((term * SH::A_BYTES + mt * 128 * D + k * 32) >> 4),
                          kd + (k * 32 >> 4), idesc, (term | k) != 0);
            umma_commit(&k_empty[st]);
            umma_commit(&acc_full[acc]);
          }
          return ok;
        });
        umma_commit(&a_empty[ab]);
      }
      // the commits have arrived before the CTA ends
      for (uint32_t j = ua > 2 ? ua - 2 : 0; ok && j < ua; ++j)
        ok = mbar_wait(&a_empty[j & 1], (j >> 1) & 1, abort_flag, p.s.status, 213);
    }
  } else if (warp >= 4 && warp < 8) {
    // ---------------------------------------------------------- queries --
    // d/16 lanes per row, 16 values each
    constexpr int LPR = D / 16, RPP = 128 / LPR;  // lanes per row, rows per pass
    const int tid = threadIdx.x - 128, l = tid % LPR;
    uint32_t ua = 0;
    for (int u = blockIdx.x; u < p.n_units; u += gridDim.x, ++ua) {
      const int ab = ua & 1;
      if (!mbar_wait(&a_empty[ab], ((ua >> 1) & 1) ^ 1, abort_flag, p.s.status, 220)) break;
      uint8_t* hi = sA + ab * 2 * SH::A_BYTES;
      const int64_t R0 = static_cast<int64_t>(u / p.nchunk) * kRows;
#pragma unroll 1
      for (int r = tid / LPR; r < kRows; r += RPP) {
        const bool on = R0 + r < p.rows;
        const uint4* src = reinterpret_cast<const uint4*>(p.s.q + (R0 + (on ? r : 0)) * D) + 2 * l;
        const uint4 raw[2] = {__ldg(src), __ldg(src + 1)};
        float x[16], amax = 0.f;
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(raw);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 f = __bfloat1622float2(h[e]);
          x[2 * e] = f.x;
          x[2 * e + 1] = f.y;
          amax = fmax3(amax, fabsf(f.x), fabsf(f.y));
        }
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        int shift = 0;
        if (amax > 0.f && amax < INFINITY) {
          shift = min(8 - ilogbf(amax), 126);
          if (amax * pow2(shift) > 448.f) --shift;
        }
        const float up = pow2(shift);
        uint32_t ch[4], cl[4];
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t a = 0, b = 0;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 y = make_float2(x[4 * w + 2 * e] * up, x[4 * w + 2 * e + 1] * up);
            const __nv_fp8x2_storage_t c2 = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
            const uint32_t back = widen2(c2);
            const float2 z = __half22float2(*reinterpret_cast<const __half2*>(&back));
            const __nv_fp8x2_storage_t d2 =
                __nv_cvt_float2_to_fp8x2(make_float2(y.x - z.x, y.y - z.y), __NV_SATFINITE, __NV_E4M3);
            a |= static_cast<uint32_t>(c2) << (16 * e);
            b |= static_cast<uint32_t>(d2) << (16 * e);
          }
          ch[w] = a;
          cl[w] = b;
        }
        // 16-byte chunk l of the row, swizzled as TMA would
        const int chunk = D == 64 ? l ^ ((r >> 1) & 3) : l ^ (r & 7);
        *reinterpret_cast<uint4*>(hi + r * D + chunk * 16) = make_uint4(ch[0], ch[1], ch[2], ch[3]);
        *reinterpret_cast<uint4*>(hi + SH::A_BYTES + r * D + chunk * 16) =
            make_uint4(cl[0], cl[1], cl[2], cl[3]);
        if (l == 0) sRow[ab * kRows + r] = p.s.idx_scale * pow2(-shift);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&a_full[ab]);
    }
  } else if (warp >= 8) {
    // --------------------------------------------------------- epilogue --
    const int grp = (warp - 8) >> 2, quarter = warp & 3;
    const int tl = quarter * 32 + lane;  // TMEM lane; rows tl and tl + 128
    float* out_s = sOut + grp * kRows * SH::OUT;
    int* own_s = sOwn + grp * kRows;
    const int H = p.s.H_kv, max_pages = c.max_pages;
    uint32_t g = 0, ua = 0;
    // after a wait that gave up, a warp goes the same way without waiting, so
    // that the group's barriers still meet
    bool ok = true;
    for (int u = blockIdx.x; u < p.n_units; u += gridDim.x, ++ua) {
      const int ab = ua & 1;
      ok = ok && mbar_wait(&a_full[ab], (ua >> 1) & 1, abort_flag, p.s.status, 230);
      const float* row_f = sRow + ab * kRows;
      const int R0 = u / p.nchunk * kRows;
      const int b_end = min((u % p.nchunk + 1) * p.CT * BPT, max_pages);  // of this unit's blocks
      for_items<BK>(p, u, false, [&](const TcItem& it) {
        // the rows' own blocks, for the group's flushes
#pragma unroll
        for (int r = tl; r < kRows; r += 128) own_s[r] = (it.pos + (R0 + r) / H - it.ta) / BK;
        int held = 0, kt_first = 0;  // tiles of this group that wait in out_s: kt_first, + 2, ...
        auto flush = [&] {
          constexpr int NV = kFlush * BPT;  // a row's values, one lane each
          asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory");
          const int v = tl % NV;
          const int b = (kt_first + 2 * (v / BPT)) * BPT + v % BPT;
          if (v < held * BPT && b < b_end) {
            float* dst = p.s.out + static_cast<int64_t>(R0) * max_pages + b;
#pragma unroll 4
            for (int r = it.ra + tl / NV; r < it.rb; r += 128 / NV)
              dst[static_cast<int64_t>(r) * max_pages] =
                  b < own_s[r] ? out_s[r * SH::OUT + v] * row_f[r] : -INFINITY;
          }
          asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory");
          held = 0;
        };
        for (int kt = it.k0; kt < it.k1; ++kt, ++g) {
          if ((g & 1) != grp) continue;
          const int st = g % ST;
          ok = ok && mbar_wait(&k_full[st], (g / ST) & 1, abort_flag, p.s.status, 231) &&
               mbar_wait(&acc_full[grp], (g >> 1) & 1, abort_flag, p.s.status, 232);
          ok = __all_sync(0xFFFFFFFFu, ok);
          tc_fence_after();
          const uint32_t ta = tmem_base + grp * 256 + (static_cast<uint32_t>(quarter * 32) << 16);
          const float* sc = sS + st * kKeys;
          const int have = sOk[st];
          if (held == 0) kt_first = kt;
          float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 1
          for (int q = 0; q < kKeys / 32; ++q) {
            uint32_t a[32], b[32];
            tmem_ld32(ta + q * 32, a);
            tmem_ld32(ta + 128 + q * 32, b);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
              const float4 s4 = *reinterpret_cast<const float4*>(sc + q * 32 + j);
              const uint64_t s01 = f2_pack(s4.x, s4.y), s23 = f2_pack(s4.z, s4.w);
              auto pair = [](const uint32_t (&v)[32], int i) {
                return f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
              };
              const uint64_t x0 = f2_mul(pair(a, j), s01), x1 = f2_mul(pair(a, j + 2), s23);
              const uint64_t y0 = f2_mul(pair(b, j), s01), y1 = f2_mul(pair(b, j + 2), s23);
              m0 = fmax3(m0, f2_lo(x0), f2_hi(x0));
              m0 = fmax3(m0, f2_lo(x1), f2_hi(x1));
              m1 = fmax3(m1, f2_lo(y0), f2_hi(y0));
              m1 = fmax3(m1, f2_lo(y1), f2_hi(y1));
            }
            if ((q + 1) % (BK / 32) == 0) {  // a block is complete
              const int j = q / (BK / 32);
              const bool on = (have >> j) & 1;
              out_s[tl * SH::OUT + held * BPT + j] = on ? m0 : -INFINITY;
              out_s[(tl + 128) * SH::OUT + held * BPT + j] = on ? m1 : -INFINITY;
              m0 = m1 = -INFINITY;
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&acc_empty[grp]);
            mbar_arrive(&k_empty[st]);
          }
          if (++held == kFlush) flush();
        }
        if (held > 0) flush();
        // blocks that no row of the item scores
        const int b0 = max(it.k0, it.k1) * BPT;
        if (b0 < b_end)
          for (int r = it.ra + (warp - 8); r < it.rb; r += 8) {
            float* dst = p.s.out + (static_cast<int64_t>(R0) + r) * max_pages;
            for (int b = b0 + lane; b < b_end; b += 32) dst[b] = -INFINITY;
          }
        asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory");  // own_s is rewritten
        return true;
      });
      __syncwarp();
      if (lane == 0) mbar_arrive(&a_empty[ab]);
    }
  }

  // every MMA is done once the epilogue has read its accumulators
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
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

// Which form (see chunk_scores_tc_kernel).
bool scores_on_tc(const ScoreLaunch& a) {
  if (a.c.n_pages * a.c.B_k >= (int64_t(1) << 31)) return false;  // TMA row coordinates
  return static_cast<int64_t>(a.c.T) * a.H_kv >= 256;
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
  if (scores_on_tc(a)) {
    using SH = TcShape<D, BK>;
    TcParams t{};
    t.s = p;
    t.rows = a.c.T * a.H_kv;
    // about eight units per SM, of at least 16 key tiles, so that whole units
    // even out over the SMs
    const int m = (t.rows + kRows - 1) / kRows;
    const int tiles = (a.c.max_pages + SH::BPT - 1) / SH::BPT;
    const int want = (8 * sms + m - 1) / m;
    t.CT = (tiles + want - 1) / want;
    if (t.CT < 16) t.CT = 16;
    t.nchunk = (tiles + t.CT - 1) / t.CT;
    t.n_units = m * t.nchunk;
    CUtensorMap tk;
    // index keys as rows of D bytes (a map of 16-bit elements: only bytes move)
    const uint64_t dims[2] = {static_cast<uint64_t>(D) / 2, static_cast<uint64_t>(a.c.n_pages) * BK};
    const uint64_t strides[1] = {static_cast<uint64_t>(D)};
    const uint32_t box[2] = {static_cast<uint32_t>(D) / 2, static_cast<uint32_t>(BK)};
    if (!make_tmap_bf16(&tk, a.pages, 2, dims, strides, box, D)) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(chunk_scores_tc_kernel<D, BK>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(SH::SMEM));
    if (e != cudaSuccess) return e;
    prof_begin("chunk_scores_tc", s);
    chunk_scores_tc_kernel<D, BK><<<t.n_units < sms ? t.n_units : sms, kTcThreads, SH::SMEM, s>>>(tk, t);
    prof_end(s);
    return cudaGetLastError();
  }
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
