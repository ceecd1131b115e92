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
//
// Two forms, each with its own sequences of a batch (see kTcRows).  For single
// tokens the bound is the cache's bytes: 32 x 32.7K keys, d_idx = 64 (71 MB),
// 18.5 us, 3.8 TB/s; the rest is the launch, the look-ups and the last blocks of
// warps that have one more than others.  For long chunks it is latency: 4096 tokens
// of four groups x 61K keys take 232 us, 0.49 PFLOP/s (the tensor cores do twice
// that: two terms per query), with the tensor pipe at 27 to 31 %, the issue slots at
// 36 % and the shared-memory pipe at 51 % of their peaks.  The eight epilogue warps
// mostly wait: for each 32 columns of TMEM in turn (40 % of all stalled cycles),
// and at their groups' barriers around the writing of the maxima (20 %).
#include <cuda_fp8.h>

#include <climits>

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
  int tc_rows;             // sequences with this many rows are the tcgen05 kernel's
  float idx_scale;
  DevStatus* status;
};

// A sequence's rows of the call; n = 0 when it has none or does not fit.
struct SeqRows {
  int t0, n;  // first token, tokens
  int pos;    // the first token's position
};
__device__ __forceinline__ SeqRows seq_rows(const ScoreParams& p, int s, int code) {
  const int t0 = max(__ldg(p.c.cu + s), 0), t1 = min(__ldg(p.c.cu + s + 1), p.c.T);
  if (t1 <= t0) return {0, 0, 0};
  const int64_t len = __ldg(p.c.seq_len + s);
  if (len < 0 || len + t1 - t0 > static_cast<int64_t>(p.c.max_pages) * p.c.B_k) {
    if (code != 0) report(p.status, DEV_ERR_CACHE_FULL, code, s, t0);
    return {0, 0, 0};
  }
  return {t0, t1 - t0, static_cast<int>(len)};
}

// Work items dealt out by sequence: the block's threads count the items of a
// run of sequences each, and an item's sequence is found from the counts'
// prefix sums.  `pre` is [blockDim.x + 1] in shared memory; all threads call.
template <typename F>
__device__ __forceinline__ int64_t seq_scan(int S, int64_t* pre, F count) {
  const int per = (S + blockDim.x - 1) / blockDim.x, lane = threadIdx.x & 31;
  int64_t mine = 0;
  for (int j = 0; j < per; ++j) {
    const int s = threadIdx.x * per + j;
    if (s < S) mine += count(s);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, mine, o);
    if (lane >= o) mine += y;
  }
  pre[threadIdx.x + 1] = mine;
  __syncthreads();
  int64_t before = 0;  // the warps before this one
  for (int w = 0; w < (threadIdx.x >> 5); ++w) before += pre[32 * w + 32];
  __syncthreads();
  pre[threadIdx.x + 1] = mine + before;
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
  return pre[blockDim.x];
}
// Item u's sequence; u becomes the item's number within it.
template <typename F>
__device__ __forceinline__ int seq_find(int S, const int64_t* pre, int64_t& u, F count) {
  const int per = (S + blockDim.x - 1) / blockDim.x;
  int lo = 0, hi = blockDim.x;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= u) lo = mid;
    else hi = mid;
  }
  u -= pre[lo];
  if (per == 1) return lo;
  int s = lo * per;
  for (; s < S - 1; ++s) {
    const int64_t n = count(s);
    if (u < n) break;
    u -= n;
  }
  return s;
}

// Scores on mma.sync, straight from global memory, for sequences with few rows.
// MMA rows = 16 keys, whose codes widen to f16 in registers; columns = the
// (token, group) rows of one sequence's tokens, NT tiles of 8.  The d axis is
// consumed in a per-thread order (thread t of a quad owns d in [t*D/4,
// (t+1)*D/4)), the same for keys and queries.  A query enters as f16 times a
// power of two that puts its largest magnitude in [2^13, 2^14): exact for every
// value within 2^-30 of it.  One warp scores one block at a time; each key byte
// is read once per column tile.
template <int D, int BK, int NT>
__device__ __forceinline__ void scores_tile(const ScoreParams& p, int s, int ta, int tokens,
                                            int pos, int b_first, int b_step) {
  constexpr int DT = D / 4;     // codes per thread and key row
  constexpr int NMMA = D / 16;  // MMAs per 16-key tile
  constexpr int NU = DT / 16;   // 16-byte loads per thread and key row
  const int lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int ncol = tokens * p.H_kv;
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
      own[n][e] = cc < ncol ? (pos + cc / p.H_kv) / BK : -1;
    }
  }
  const int last = (pos + tokens - 1) / BK;  // own block of the last token
  float* out = p.out + row0 * p.c.max_pages;
  for (int b = b_first; b < p.c.max_pages; b += b_step) {
    float mx[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) mx[n][0] = mx[n][1] = -INFINITY;
    const int64_t pg = b < last ? chunk_page(p.c, s, b) : -1;
    if (b < last && pg < 0 && lane == 0) report(p.status, DEV_ERR_BAD_INDEX, 121, s, b);
    if (pg >= 0) {
      const uint8_t* kbase = p.pages + (pg * BK + g) * D + t * DT;
      const float* sbase = p.scale + pg * BK + g;
      // the block in parts: a part's codes are all loaded before its MMAs
      constexpr int PARTS = NT == 1 ? 4 : D / 32;
      constexpr int KT = BK / 16 / PARTS;  // 16-key tiles of a part
#pragma unroll 1
      for (int h = 0; h < PARTS; ++h) {
        uint4 cr[KT][2][NU];
        float sc[KT][2];
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = (h * KT + i) * 16 + 8 * e;
#pragma unroll
            for (int u = 0; u < NU; ++u)
              cr[i][e][u] = __ldg(reinterpret_cast<const uint4*>(kbase + key * D) + u);
            sc[i][e] = __ldg(sbase + key);
          }
#pragma unroll
        for (int i = 0; i < KT; ++i) {
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
}

// Units are (a column tile of one sequence, a share of the blocks), dealt out
// to the grid; a tile's blocks are split so that the units fill it.
template <int D, int NT>
constexpr int kHeld = NT == 1 ? 4 : D == 64 ? 2 : 1;  // CTAs per SM
template <int D, int BK, int NT>
__global__ void __launch_bounds__(256, kHeld<D, NT>) chunk_scores_kernel(const ScoreParams p) {
  __shared__ int64_t pre[257];
  griddep_wait();
  const int tpt = 8 * NT / p.H_kv, code = blockIdx.x == 0 ? 120 : 0;
  const auto count_of = [&](const SeqRows& r) {
    return static_cast<int64_t>(r.n) * p.H_kv < p.tc_rows ? (r.n + tpt - 1) / tpt : 0;
  };
  const auto count = [&](int s) { return count_of(seq_rows(p, s, 0)); };
  // (no more than T unless cu is not a sequence of offsets)
  const int tiles = static_cast<int>(min(
      seq_scan(p.c.S, pre, [&](int s) { return count_of(seq_rows(p, s, code)); }),
      static_cast<int64_t>(p.c.T)));
  if (tiles == 0) return;
  const int grid = gridDim.x;
  int split = grid / tiles;
  if (split < 4) split = min((p.c.max_pages + 31) / 32, (4 * grid + tiles - 1) / tiles);
  split = max(1, min(split, (p.c.max_pages + 7) / 8));
  const int warp = threadIdx.x >> 5;
  for (int64_t u = blockIdx.x; u < static_cast<int64_t>(tiles) * split; u += grid) {
    int64_t tile = u / split;
    const int x = static_cast<int>(u - tile * split);
    const int s = seq_find(p.c.S, pre, tile, count);
    const SeqRows r = seq_rows(p, s, 0);
    const int first = static_cast<int>(tile) * tpt, n = min(tpt, r.n - first);
    if (NT == 1 || n * p.H_kv <= 8)
      scores_tile<D, BK, 1>(p, s, r.t0 + first, n, r.pos + first, x * 8 + warp, split * 8);
    else
      scores_tile<D, BK, NT>(p, s, r.t0 + first, n, r.pos + first, x * 8 + warp, split * 8);
  }
}

// ---------------------------------------------- scores on tcgen05, many rows --
// For chunks with many rows: 256 rows (two UMMA M-tiles) against 128 keys at a
// time, both in FP8: the codes go from their page by TMA straight into the
// MMA's layout, and the queries are split into two E4M3 terms.  A row is scaled
// by a power of two that puts its largest magnitude in [224, 448]; hi =
// E4M3(x), lo = E4M3(x - hi) hold its 8 bits exactly down to 2^-10 of the
// largest, and every element to 2^-10 / 224 of it.  hi and lo accumulate into the
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
// A unit is (256 rows of one sequence, CT key tiles); units are dealt out to one
// CTA per SM, about eight to each so that whole units even out.
constexpr int kTcThreads = 512;
constexpr int kRows = 256;   // rows per unit
constexpr int kKeys = 128;   // keys per tile
constexpr int kFlush = 8;    // tiles of a group between flushes

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
                                 (2 * ST + 9) * 8 + 64 + (kTcThreads + 1) * 8;
  static_assert(SMEM <= 227 * 1024, "shared memory of one CTA");
};

struct TcUnit {
  int s;
  int64_t row0;      // first row of the call
  int rows;          // rows of the unit
  int first;         // the unit's first row within its sequence
  int pos;           // position of the sequence's first row
  int own;           // the last row's own block
  int k0, k1;        // key tiles to score
  int b_end;         // end of the blocks that the unit writes
};

// How the call's units are laid out: the same in every role.
template <int BK>
struct TcPlan {
  static constexpr int BPT = kKeys / BK;
  const ScoreParams& p;
  const int64_t* pre;
  int CT;
  int64_t units;

  __device__ __forceinline__ bool has(const SeqRows& r) const {
    return static_cast<int64_t>(r.n) * p.H_kv >= p.tc_rows;
  }
  __device__ __forceinline__ int tiles_m(const SeqRows& r) const {
    return static_cast<int>((static_cast<int64_t>(r.n) * p.H_kv + kRows - 1) / kRows);
  }
  __device__ __forceinline__ int tiles_k(const SeqRows& r) const {  // at least one
    return max(1, ((r.pos + r.n - 1) / BK + BPT - 1) / BPT);
  }
  __device__ __forceinline__ int64_t count(const SeqRows& r) const {
    return has(r) ? static_cast<int64_t>(tiles_m(r)) * ((tiles_k(r) + CT - 1) / CT) : 0;
  }
  __device__ __forceinline__ TcPlan(const ScoreParams& p_, int64_t* pre_) : p(p_), pre(pre_) {
    const int code = blockIdx.x == 0 ? 202 : 0;
    const int64_t visits = seq_scan(p.c.S, pre_, [&](int s) {
      const SeqRows r = seq_rows(p, s, code);
      return has(r) ? static_cast<int64_t>(tiles_m(r)) * tiles_k(r) : 0;
    });
    // eight units per SM, of at least 16 key tiles where there is that much work
    const int64_t g = gridDim.x, one = (visits + g - 1) / g, eight = (visits + 8 * g - 1) / (8 * g);
    CT = static_cast<int>(max(eight, min(one, static_cast<int64_t>(16))));
    CT = max(CT, 1);
    __syncthreads();
    units = seq_scan(p.c.S, pre_, [&](int s) { return count(seq_rows(p, s, 0)); });
  }
  __device__ __forceinline__ TcUnit unit(int64_t u) const {
    TcUnit it;
    it.s = seq_find(p.c.S, pre, u, [&](int s) { return count(seq_rows(p, s, 0)); });
    const SeqRows r = seq_rows(p, it.s, 0);
    const int kt = tiles_k(r), nc = (kt + CT - 1) / CT;
    const int m = static_cast<int>(u / nc), ch = static_cast<int>(u - static_cast<int64_t>(m) * nc);
    it.first = m * kRows;
    it.rows = min(kRows, r.n * p.H_kv - it.first);
    it.row0 = static_cast<int64_t>(r.t0) * p.H_kv + it.first;
    it.pos = r.pos;
    it.own = (r.pos + (it.first + it.rows - 1) / p.H_kv) / BK;
    it.k0 = ch * CT;
    it.k1 = max(it.k0, min(it.k0 + CT, (it.own + BPT - 1) / BPT));
    it.b_end = ch == nc - 1 ? p.c.max_pages : min((it.k0 + CT) * BPT, p.c.max_pages);
    return it;
  }
};

template <int D, int BK>
__global__ void __launch_bounds__(kTcThreads, 1)
    chunk_scores_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const ScoreParams p) {
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
  uint64_t* fin = acc_empty + 2;       // every MMA of the CTA finished
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int64_t* pre = reinterpret_cast<int64_t*>(tmem_slot + 2);  // [threads + 1]
  const ChunkSeqs& c = p.c;

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
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const TcPlan<BK> plan(p, pre);

  if (warp == 0) {
    // -------------------------------------------------------- producer --
    // Lane l holds the page of block l of a batch of 32, the next batch on its
    // way; lane 0 waits and issues.
    if (lane == 0) prefetch_tmap(&tm_k);
    uint32_t g = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; ok && u < plan.units; u += gridDim.x) {
        const TcUnit it = plan.unit(u);
        const int b0 = it.k0 * BPT, b1 = min(it.k1 * BPT, c.max_pages);
        auto fetch = [&](int b) {
          if (b >= b1) return -1;
          const int pg = static_cast<int>(chunk_page(c, it.s, b));
          if (pg < 0 && b < it.own) report(p.status, DEV_ERR_BAD_INDEX, 201, it.s, b);
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
          ok = mbar_wait_warp(&k_empty[st], ((g / ST) & 1) ^ 1, abort_flag, p.status, 200);
          if (!ok) break;
          if (lane == 0) {
            sOk[st] = have;
            mbar_arrive_expect_tx(&k_full[st], __popc(have) * (BK * D + BK * 4));
#pragma unroll
            for (int j = 0; j < BPT; ++j)
              if (pg[j] >= 0) {
                const int row = pg[j] * BK;
                tma_load_2d(sK + st * SH::K_BYTES + j * BK * D, &tm_k, &k_full[st], 0, row);
                bulk_load(sS + st * kKeys + j * BK, p.scale + row, BK * 4, &k_full[st]);
              }
          }
        }
    }
    // nothing is still on its way into this CTA's shared memory when it ends, not
    // even after a wait that gave up
    for (uint32_t j = g > ST ? g - ST : 0; j < g; ++j)
      mbar_wait(&k_full[j % ST], (j / ST) & 1, nullptr, p.status, 203);
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA --
    if (lane == 0) {
      // kind::f8f6f4, E4M3 x E4M3 -> f32, both K-major
      constexpr uint32_t idesc = (1u << 4) | (static_cast<uint32_t>(kKeys >> 3) << 17) | (128u >> 4 << 24);
      const uint64_t a_desc = umma_desc(smem_u32(sA), 16, SH::SBO, SH::SWZ);
      const uint64_t k_desc = umma_desc(smem_u32(sK), 16, SH::SBO, SH::SWZ);
      uint32_t g = 0, ua = 0;
      bool ok = true;
      for (int64_t u = blockIdx.x; ok && u < plan.units; u += gridDim.x, ++ua) {
        const int ab = ua & 1;
        const TcUnit it = plan.unit(u);
        ok = mbar_wait(&a_full[ab], (ua >> 1) & 1, abort_flag, p.status, 210);
        if (!ok) break;
        const uint64_t ad0 = a_desc + ab * (2 * SH::A_BYTES >> 4);
          for (int kt = it.k0; ok && kt < it.k1; ++kt, ++g) {
            const int st = g % ST, acc = g & 1;
            ok = mbar_wait(&k_full[st], (g / ST) & 1, abort_flag, p.status, 211) &&
                 mbar_wait(&acc_empty[acc], ((g >> 1) & 1) ^ 1, abort_flag, p.status, 212);
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
        umma_commit(&a_empty[ab]);
      }
      // every MMA is done before TMEM is released, and every commit has arrived
      // before the CTA ends, after a wait that gave up too
      umma_commit(fin);
      mbar_wait(fin, 0, nullptr, p.status, 213);
    }
  } else if (warp >= 4 && warp < 8) {
    // ---------------------------------------------------------- queries --
    // d/16 lanes per row, 16 values each
    constexpr int LPR = D / 16, RPP = 128 / LPR;  // lanes per row, rows per pass
    const int tid = threadIdx.x - 128, l = tid % LPR;
    uint32_t ua = 0;
    for (int64_t u = blockIdx.x; u < plan.units; u += gridDim.x, ++ua) {
      const int ab = ua & 1;
      const TcUnit it = plan.unit(u);
      if (!mbar_wait_warp(&a_empty[ab], ((ua >> 1) & 1) ^ 1, abort_flag, p.status, 220)) break;
      uint8_t* hi = sA + ab * 2 * SH::A_BYTES;
      constexpr int NP = 4;  // passes whose rows are loaded together
#pragma unroll 1
      for (int r0 = tid / LPR; r0 < kRows; r0 += NP * RPP) {
        uint4 raw[NP][2];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int r = r0 + i * RPP;
          const uint4* src =
              reinterpret_cast<const uint4*>(p.q + (it.row0 + (r < it.rows ? r : 0)) * D) + 2 * l;
          raw[i][0] = __ldg(src);
          raw[i][1] = __ldg(src + 1);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
        const int r = r0 + i * RPP;
        float x[16], amax = 0.f;
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(raw[i]);
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
        if (l == 0) sRow[ab * kRows + r] = p.idx_scale * pow2(-shift);
      }
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
    const int H = p.H_kv, max_pages = c.max_pages;
    uint32_t g = 0, ua = 0;
    // after a wait that gave up, a warp goes the same way without waiting, so
    // that the group's barriers still meet
    bool ok = true;
    for (int64_t u = blockIdx.x; u < plan.units; u += gridDim.x, ++ua) {
      const int ab = ua & 1;
      const TcUnit it = plan.unit(u);
      ok = ok && mbar_wait_warp(&a_full[ab], (ua >> 1) & 1, abort_flag, p.status, 230);
      const float* row_f = sRow + ab * kRows;
      const int b_end = it.b_end;
      float* out_g = p.out + it.row0 * max_pages;
        // the rows' own blocks, for the group's flushes
#pragma unroll
        for (int r = tl; r < kRows; r += 128) own_s[r] = (it.pos + (it.first + r) / H) / BK;
        int held = 0, kt_first = 0;  // tiles of this group that wait in out_s: kt_first, + 2, ...
        auto flush = [&] {
          constexpr int NV = kFlush * BPT;  // a row's values, one lane each
          asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory");
          const int v = tl % NV;
          const int b = (kt_first + 2 * (v / BPT)) * BPT + v % BPT;
          if (v < held * BPT && b < b_end) {
            float* dst = out_g + b;
#pragma unroll 4
            for (int r = tl / NV; r < it.rows; r += 128 / NV)
              dst[static_cast<int64_t>(r) * max_pages] =
                  b < own_s[r] ? out_s[r * SH::OUT + v] * row_f[r] : -INFINITY;
          }
          asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory");
          held = 0;
        };
        for (int kt = it.k0; kt < it.k1; ++kt, ++g) {
          if ((g & 1) != grp) continue;
          const int st = g % ST;
          ok = ok && mbar_wait_warp(&k_full[st], (g / ST) & 1, abort_flag, p.status, 231) &&
               mbar_wait_warp(&acc_full[grp], (g >> 1) & 1, abort_flag, p.status, 232);
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
          for (int r = warp - 8; r < it.rows; r += 8) {
            float* dst = out_g + static_cast<int64_t>(r) * max_pages;
            for (int b = b0 + lane; b < b_end; b += 32) dst[b] = -INFINITY;
          }
        asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory");  // own_s is rewritten
      __syncwarp();
      if (lane == 0) mbar_arrive(&a_empty[ab]);
    }
  }

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

// A score and its block as one number: larger scores first, of equal ones the
// lower block (-0 counts as 0).
__device__ __forceinline__ uint64_t topk_key(float x, int block) {
  const uint32_t u = __float_as_uint(x + 0.f);
  const uint32_t o = u & 0x80000000u ? ~u : u | 0x80000000u;
  return (static_cast<uint64_t>(o) << 32) | ~static_cast<uint32_t>(block);
}
__device__ __forceinline__ void topk_unkey(uint64_t key, float& x, int& block) {
  const uint32_t o = static_cast<uint32_t>(key >> 32);
  x = __uint_as_float(o & 0x80000000u ? o & 0x7FFFFFFFu : ~o);
  block = static_cast<int>(~static_cast<uint32_t>(key));
}

// One warp per row.  The row's candidates (blocks before its own) are read
// once, NR * 32 of them at a time in registers.  The (k-1)-th largest of the 32
// lanes' maxima is a lower bound of the (k-1)-th largest candidate, so only
// the few candidates at or above it (and above what is kept already) can enter:
// about 22 of 1024 at k = 16.  They are gathered (each lane's behind those of the
// lanes before it) and ranked with the kept ones by counting the larger ones; lane
// i then holds the i-th best.  More than kGather of them (many equal scores) enter
// the list one after another instead, each by a ballot and a shift: in ascending
// block order, and a later one must be larger to pass an earlier one, so that ties
// keep the lower block here too.  Scores of -inf and NaN are never chosen.
// The bound is instructions, about 800 a row of 1024 blocks (issue slots 68 % busy):
// 16384 such rows (67 MB) take 22.9 us, 128 rows of 257 4.8.
constexpr int kGather = 64;
constexpr int kTopkWarps = 2;  // rows per CTA

template <int NR>
__global__ void __launch_bounds__(32 * kTopkWarps, 32 / kTopkWarps) block_topk_kernel(const TopkParams p) {
  constexpr int kList = kGather + 32;  // candidates and kept ones
  __shared__ alignas(16) uint64_t lists[kTopkWarps][kList + 32];
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
    const float* at = src + base + lane;
    const int left = n - base - lane;
#pragma unroll
    for (int j = 0; j < NR; ++j) x[j] = 32 * j < left ? __ldg(at + 32 * j) : -INFINITY;
#pragma unroll
    for (int j = 0; j < NR; ++j) mx = fmaxf(mx, x[j]);
    const float floor_ = __shfl_sync(0xFFFFFFFFu, warp_sort_desc(mx, lane), k1 - 1);
    float worst = __shfl_sync(0xFFFFFFFFu, lv, k1 - 1);
    // what enters is above this: not below floor_, and above worst
    const float lim = floor_ > worst ? nextafterf(floor_, -INFINITY) : worst;
    unsigned in = 0;  // bit j: candidate j of this lane enters
#pragma unroll
    for (int j = 0; j < NR; ++j)
      if (x[j] > lim) in |= 1u << j;
    const int mine = __popc(in);
    int upto = mine;  // the candidates of this lane and the ones before
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    const int count = __shfl_sync(0xFFFFFFFFu, upto, 31);
    if (count <= kGather) {
      uint64_t* list = lists[threadIdx.x >> 5];
      const int held = __popc(__ballot_sync(0xFFFFFFFFu, lane < k1 && li >= 0));
      __syncwarp();
      float2* to = reinterpret_cast<float2*>(list) + upto - mine;
      for (; in != 0; in &= in - 1) {  // few: read again rather than picked from registers
        const int j = __ffs(in) - 1;
        *to++ = make_float2(__ldg(at + 32 * j), __int_as_float(base + 32 * j + lane));
      }
      if (lane < held) reinterpret_cast<float2*>(list)[count + lane] = make_float2(lv, __int_as_float(li));
      __syncwarp();
      const int all = count + held;
      uint64_t key[kList / 32];
      int rank[kList / 32];
#pragma unroll
      for (int c = 0; c < kList / 32; ++c) {
        rank[c] = 0;
        if (c * 32 + lane < all) {
          const float2 e = reinterpret_cast<const float2*>(list)[c * 32 + lane];
          key[c] = topk_key(e.x, __float_as_int(e.y));
          list[c * 32 + lane] = key[c];
        }
      }
      __syncwarp();
      if (all <= 32) {
        // two at a time; behind the last one key 0, which is larger than none
        if (lane == 0) list[all] = 0;
        __syncwarp();
#pragma unroll 4
        for (int j = 0; j < all; j += 2) {
          const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(list + j);
          rank[0] += two.x > key[0] ? 1 : 0;
          rank[0] += two.y > key[0] ? 1 : 0;
        }
      } else {
        for (int j = 0; j < all; ++j) {
          const uint64_t other = list[j];
#pragma unroll
          for (int c = 0; c < kList / 32; ++c) rank[c] += other > key[c] ? 1 : 0;
        }
      }
#pragma unroll
      for (int c = 0; c < kList / 32; ++c)
        if (c * 32 + lane < all && rank[c] < 32) list[kList + rank[c]] = key[c];
      __syncwarp();
      lv = -INFINITY;
      li = -1;
      if (lane < min(all, k1)) topk_unkey(list[kList + lane], lv, li);
      continue;
    }
#pragma unroll 1
    for (int j = 0; j < NR; ++j) {
      const float xj = 32 * j < left ? __ldg(at + 32 * j) : -INFINITY;
      unsigned todo = __ballot_sync(0xFFFFFFFFu, xj > worst && xj > lim);
      while (todo != 0) {
        const int from = __ffs(todo) - 1;
        const float v = __shfl_sync(0xFFFFFFFFu, xj, from);
        const int to = __popc(__ballot_sync(0xFFFFFFFFu, lv >= v));
        const float uv = __shfl_up_sync(0xFFFFFFFFu, lv, 1);
        const int ui = __shfl_up_sync(0xFFFFFFFFu, li, 1);
        if (lane > to) {
          lv = uv;
          li = ui;
        } else if (lane == to) {
          lv = v;
          li = base + 32 * j + from;
        }
        worst = __shfl_sync(0xFFFFFFFFu, lv, k1 - 1);
        todo &= todo - 1;
        todo &= __ballot_sync(0xFFFFFFFFu, xj > worst);
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

// A sequence's rows go to the tcgen05 kernel from this many on, each form taking
// its own sequences of a batch, so that single tokens beside a long chunk cost
// what they cost alone.  Rows in one sequence, mma.sync / tcgen05 in us:
//            d_idx 64, 9K keys   61K keys     d_idx 128, 9K keys   61K keys
//    256        10.3 / 16.6     16.5 / 18.6      12.4 / 21.0      24.0 / 24.7
//    512        12.4 / 16.5     24.7 / 18.9      12.4 / 19.7      34.9 / 22.6
//   1024        12.4 / 18.5     37.0 / 26.7      20.6 / 20.6      63.6 / 28.8
//   2048        20.6 / 24.7     67.7 / 47.9      34.9 / 22.6     135.7 / 51.7
constexpr int kTcRows = 512;

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
  const int64_t rows = static_cast<int64_t>(a.c.T) * a.H_kv;
  const int sms = num_sms();
  // TMA row coordinates are 32 bits
  const bool tc = rows >= kTcRows && a.c.n_pages * BK < (int64_t(1) << 31);
  p.tc_rows = tc ? kTcRows : INT_MAX;
  if (tc) {
    using SH = TcShape<D, BK>;
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
    chunk_scores_tc_kernel<D, BK><<<sms, kTcThreads, SH::SMEM, s>>>(tk, p);
    prof_end(s);
    e = cudaGetLastError();
    // The other form follows for one sequence too: the call's rows may be padding
    // for the most part.
    if (e != cudaSuccess) return e;
  }
  // Columns per tile: 8 while there are no more tokens than sequences (single
  // tokens share no keys, and fewer registers let twice as many warps load), else
  // up to 32.  The grid is what the SMs hold, fewer when tokens x blocks are.
  const bool wide = a.c.T > a.c.S && rows > 8;
  const int64_t most = static_cast<int64_t>(a.c.T) * ((a.c.max_pages + 7) / 8);
  const int64_t held = (wide ? kHeld<D, 4> : kHeld<D, 1>) * sms;
  const dim3 grid(static_cast<unsigned>(most < held ? most : held));
  prof_begin("chunk_scores", s);
  const cudaError_t e =
      wide ? launch_pdl(chunk_scores_kernel<D, BK, 4>, grid, dim3(256), 0, s, p)
           : launch_pdl(chunk_scores_kernel<D, BK, 1>, grid, dim3(256), 0, s, p);
  prof_end(s);
  return e != cudaSuccess ? e : cudaGetLastError();
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
  const dim3 block(32 * kTopkWarps), grid(static_cast<unsigned>((threads + block.x - 1) / block.x));
  prof_begin("block_topk", s);
  const cudaError_t e = n <= 256 ? launch_pdl(block_topk_kernel<8>, grid, block, 0, s, p)
                                 : launch_pdl(block_topk_kernel<32>, grid, block, 0, s, p);
  prof_end(s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace msa
