// chunk_attn_kv.cu -- Eq. 8 for chunks with many rows on the paged FP8 cache,
// KV-outer on tcgen05: each selected page is read once for all the rows of
// the chunk that chose it.
//
//   1. tables: per row its sequence's offsets, per block its page, first key
//      and number of keys;
//   2. inverse index (inv_index.cu): per (group, block) the selection slots
//      that chose it, cut into tiles of Tq rows x the group's heads = 128 MMA
//      rows;
//   3. tiles: S = Q K^T and O = P V for one page and one gathered tile, an
//      fp16 partial of O, its LSE and its factor per slot;
//   4. merge: the LSE-weighted sum of each row's partials.
//
// The tile kernel has the prefill's structure (sparse_attn.cu: gathered Q tiles
// by TMA, S and O in TMEM, P taken from TMEM) with the operands made from E4M3
// codes: a TMA ring brings a page's codes, a warpgroup widens K to bf16 (the
// queries' type) and V to f16, both exact, into the MMA's tiles; a key's scale
// multiplies its column of S in the softmax, a value's scale its weight.  The
// weights go to the tensor cores relative to the page's largest value scale,
// or to the row's largest weight-times-scale where a page's scales are far
// apart, so that f16 holds them (11 bits; a bf16 P would hold 8); that factor
// over the row's sum is kept beside the LSE and applied by the merge, and a
// partial stays within 128 * 448 < 65504.
//
// 4096 rows of two sequences at 61K cached tokens (H_q = 32, H_kv = 4, d_h =
// B_k = 128, k = 16; 137 GFLOP): 355 us in the tile kernel, of 465 in all (the
// query-outer kernel: 1122); the merge reads its 537 MB of partials in 88.
// What bounds the tiles is the MMAs beside the softmax's TMEM reads: S and O
// take 1200 and 1500 clocks a tile in place, 512 each at the peak rate.
#include <climits>
#include <type_traits>

#include <cuda_fp8.h>

#include "attn_common.cuh"
#include "chunk_launch.h"

namespace msa {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

struct KVParams {
  int q4d;  // 1: one 4-D TMA box per gathered row ([d-chunk][head] rows, 8 heads)
  int H_kv, kk, G, R;
  int B;             // S * max_pages: blocks, numbered s * max_pages + b
  int q0;            // first row of the chunk window
  const int4* blk;   // [B] {page, first key as a row number, keys, 0}
  const float* ks;
  const float* vs;
  float scale_log2;
  ChunkBufs c;
  float* part_f;     // [slots, G] largest weight over the sum of weights
  DevStatus* status;
};

constexpr int kThreads = 896;  // 28 warps of at most 72 registers
constexpr int kIR = 8;         // tile-info ring depth
constexpr int kNS = 2;         // S/P and O buffers in TMEM
constexpr int kNKV = 2;        // K/V slots
constexpr int kRaw = 3;        // raw ring: 64 keys of K or V each
template <int D_H, int B_K>
struct KVShape {
  static constexpr int Q_BYTES = kRowsPerTile * D_H * 2;
  static constexpr int K_BYTES = B_K * D_H * 2;
  static constexpr int KV_BYTES = 2 * K_BYTES;
  // what the Q ring may take of the 227 KB: minus alignment slack, the scales,
  // the tile-info ring and the barriers
  static constexpr int RAW_BYTES = 64 * D_H;     // codes of 64 keys
  static constexpr int CPP = B_K / 64;           // such pieces of a page's K (or V)
  static constexpr int SCALES_PAD = 2 * B_K + 32;  // floats per K/V slot: scales, unit, even
  static constexpr int BUDGET = 227 * 1024 - 1024 - kNKV * SCALES_PAD * 4 - kRaw * RAW_BYTES - 2048;
  static constexpr int QS_FIT = (BUDGET - kNKV * KV_BYTES) / Q_BYTES;
  static constexpr int QS = QS_FIT > 4 ? 4 : QS_FIT;
  static_assert(QS >= 2, "two Q stages must fit");
  static constexpr int DCH = D_H / 64;
  static constexpr uint32_t TM_S = 0, TM_O = kNS * 128;
  static constexpr int PPK = D_H / 16;             // 16-code pieces per key
  static constexpr int NP = 64 * PPK / 128;        // pieces per thread of 64 keys
  static constexpr int KPP = 128 / PPK;            // keys per pass of the warpgroup
};

constexpr int kMaxTq = 16;
constexpr float kEven = 16.f;  // value scales of a page this close need no row maximum

struct TileInfo {
  int r, len, gen;
  int jb;  // the block's first key, numbered as the rows are
  uint32_t slot[kMaxTq];
  int qi[kMaxTq];
};

// Instruction descriptor of kind::f16 with f16 A/B and f32 accumulation.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t e4m3x2_bf16x2(uint32_t c2) {
  const uint32_t h = widen2(c2);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16(f.x, f.y);
}
// Byte masks (0xFF) of the NaN codes of four (0x7F and 0xFF).
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
}

// 16-lane TMEM access (layouts as .x8 in msa_common.cuh): 32 columns of S, 16
// of P.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_16x128b_x4(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

template <int D_H, int B_K>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_tile_kernel(const __grid_constant__ CUtensorMap tm_q,
                      const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const KVParams p) {
  using SH = KVShape<D_H, B_K>;
  constexpr int QS = SH::QS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;                         // [QS] gathered Q tiles
  uint8_t* sKV = sQ + QS * SH::Q_BYTES;       // [kNKV] K (bf16), then V (f16)
  // per slot: key scales, value scales, the value scales' unit and whether
  // they are even
  float* sSc = reinterpret_cast<float*>(sKV + kNKV * SH::KV_BYTES);  // [kNKV][SCALES_PAD]
  uint8_t* sRaw = reinterpret_cast<uint8_t*>(sSc + kNKV * SH::SCALES_PAD);  // [kRaw] 64 keys' codes
  TileInfo* info = reinterpret_cast<TileInfo*>(sRaw + kRaw * SH::RAW_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(info + kIR);
  uint64_t* q_full = bars;               // [QS] gathered Q landed
  uint64_t* q_empty = q_full + QS;       // [QS] S of the stage's tile computed
  uint64_t* raw_full = q_empty + QS;     // [kRaw] codes landed
  uint64_t* raw_empty = raw_full + kRaw; // [kRaw] codes read
  uint64_t* sc_full = raw_empty + kRaw;  // [kNKV] slot free, its scales written
  uint64_t* kv_full = sc_full + kNKV;    // [kNKV] page widened
  uint64_t* kv_empty = kv_full + kNKV;   // [kNKV] last O = P V of the page's run finished
  uint64_t* i_full = kv_empty + kNKV;    // [kIR] tile info written
  uint64_t* i_empty = i_full + kIR;      // [kIR] the tile's epilogue and softmax are done
  uint64_t* s_full = i_empty + kIR;      // [kNS] S in TMEM
  uint64_t* p_full = s_full + kNS;       // [kNS] P in TMEM
  uint64_t* o_full = p_full + kNS;       // [kNS] O in TMEM
  uint64_t* o_empty = o_full + kNS;      // [kNS] O read
  uint64_t* fin = o_empty + kNS;         // every MMA of the CTA finished
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(fin + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* gen_keys = abort_flag + 1;  // [kNKV] keys of the slot's page, 0 = no more pages

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < QS; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int j = 0; j < kRaw; ++j) {
      mbar_init(&raw_full[j], 1);
      mbar_init(&raw_empty[j], 4);  // the four widening warps
    }
    for (int j = 0; j < kNKV; ++j) {
      mbar_init(&sc_full[j], 1);
      mbar_init(&kv_full[j], 4);  // the four widening warps
      mbar_init(&kv_empty[j], 1);
    }
    for (int j = 0; j < kIR; ++j) {
      mbar_init(&i_full[j], 1);
      mbar_init(&i_empty[j], 12);  // the four epilogue and the tile's eight softmax warps
    }
    for (int s = 0; s < kNS; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 8);   // the tile's eight softmax warps
      mbar_init(&o_full[s], 1);
      mbar_init(&o_empty[s], 4);
    }
    mbar_init(fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();  // the tiles' records
  const int n_tiles = p.c.n_tiles[0];
  // The CTA's tiles: segments of L consecutive tiles, dealt out in turn, so
  // that every CTA gets its share of the lists where a page serves few tiles
  // (and costs more than they do).  18000 tiles: contiguous ranges 377 us,
  // segments of 4, 8, 12, 16, 31: 432, 376, 360, 361, 398.
  const int grid = gridDim.x, cta = blockIdx.x;
  const int share = (n_tiles + grid - 1) / grid;
  const int quarter_share = (share + 3) / 4;
  const int L = share < 16 ? (share > 0 ? share : 1)
                           : (quarter_share < 8 ? 8 : (quarter_share > 12 ? 12 : quarter_share));
  int my_tiles = 0;
  for (int64_t t = static_cast<int64_t>(cta) * L; t < n_tiles; t += static_cast<int64_t>(grid) * L)
    my_tiles += n_tiles - t < L ? static_cast<int>(n_tiles - t) : L;
  auto tile_of = [&](int n) { return (n / L * grid + cta) * L + n % L; };
  const int per_q = p.H_kv * p.kk;
  const int wg = warp >> 2;

  // Generation g of this CTA: the g-th run of its tiles with one key (within
  // a segment), which needs one page.  The run that starts at tile n ends here:
  auto run_end = [&](int n, int4 meta) {
    const int seg = (n / L + 1) * L;
    const int end = n + meta.w - tile_of(n);
    return end < seg ? end : seg;
  };
  auto page_of = [&](int4 meta) { return p.blk[meta.x % p.B]; };
  auto group_of = [&](int4 meta) { return (meta.x / p.B) % p.H_kv; };

  if (wg == 6) {
    // ---------------------------------------------------------- widening --
    // 64 keys of K or V at a time from the raw ring into the operand tiles.
    const int tid = threadIdx.x - 768;
    const int key0 = tid / SH::PPK, piece = tid % SH::PPK;
    // (row, 16-byte chunk) of a 128-byte-swizzled tile of 64-element boxes
    auto put = [&](uint8_t* base, int key, int half, uint4 w) {
      const int d = piece * 16 + half * 8;
      *reinterpret_cast<uint4*>(base + (d >> 6) * B_K * 128 + key * 128 +
                                ((((d >> 3) & 7) ^ (key & 7)) << 4)) = w;
    };
    int ring = 0;
    bool ok = true;
    for (int gen = 0; ok; ++gen) {
      const int slot = gen % kNKV;
      if (!mbar_wait_warp(&sc_full[slot], (gen / kNKV) & 1, abort_flag, p.status, 151)) break;
      const int keys = gen_keys[slot];
      if (keys == 0) break;  // no more generations
      uint8_t* sK = sKV + slot * SH::KV_BYTES;
      float* sc = sSc + slot * SH::SCALES_PAD;
#pragma unroll 1
      for (int c = 0; ok && c < 2 * SH::CPP; ++c, ++ring) {
        const int rs = ring % kRaw;
        ok = mbar_wait_warp(&raw_full[rs], (ring / kRaw) & 1, abort_flag, p.status, 153);
        if (!ok) break;
        const uint8_t* src = sRaw + rs * SH::RAW_BYTES + tid * 16;
        uint4 w[SH::NP];
#pragma unroll
        for (int i = 0; i < SH::NP; ++i)
          w[i] = *reinterpret_cast<const uint4*>(src + i * 128 * 16);
        __syncwarp();
        if (lane == 0) mbar_arrive(&raw_empty[rs]);
        const bool is_v = c >= SH::CPP;
        const int first = (is_v ? c - SH::CPP : c) * 64 + key0;
        if (!is_v) {
#pragma unroll
          for (int i = 0; i < SH::NP; ++i) {
            const int key = first + i * SH::KPP;
            put(sK, key, 0, make_uint4(e4m3x2_bf16x2(w[i].x), e4m3x2_bf16x2(w[i].x >> 16),
                                       e4m3x2_bf16x2(w[i].y), e4m3x2_bf16x2(w[i].y >> 16)));
            put(sK, key, 1, make_uint4(e4m3x2_bf16x2(w[i].z), e4m3x2_bf16x2(w[i].z >> 16),
                                       e4m3x2_bf16x2(w[i].w), e4m3x2_bf16x2(w[i].w >> 16)));
          }
        } else {
#pragma unroll
          for (int i = 0; i < SH::NP; ++i) {
            const int key = first + i * SH::KPP;
            uint4 x = w[i];
            // What lies behind the sequence is zeroed.  A NaN value must not
            // reach the rows that do not see it (0 * NaN): its code becomes 0
            // and its row's scale NaN, which the rows that see it multiply with.
            if (key >= keys) x = make_uint4(0, 0, 0, 0);
            const uint4 bad =
                make_uint4(nan_bytes(x.x), nan_bytes(x.y), nan_bytes(x.z), nan_bytes(x.w));
            if ((bad.x | bad.y | bad.z | bad.w) != 0u) {
              x = make_uint4(x.x & ~bad.x, x.y & ~bad.y, x.z & ~bad.z, x.w & ~bad.w);
              sc[B_K + key] = __int_as_float(0x7FC00000);
            }
            put(sK + SH::K_BYTES, key, 0,
                make_uint4(widen2(x.x), widen2(x.x >> 16), widen2(x.y),
                           widen2(x.y >> 16)));
            put(sK + SH::K_BYTES, key, 1,
                make_uint4(widen2(x.z), widen2(x.z >> 16), widen2(x.w),
                           widen2(x.w >> 16)));
          }
        }
      }
      if (!ok) break;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&kv_full[slot]);
    }
  } else if (wg == 1) {
    if (warp == 4) {
      // ----------------------------------------------------- TMA producer --
      if (lane == 0) prefetch_tmap(&tm_q);
      auto meta_of = [&](int n) -> int4 {
        return n < my_tiles ? p.c.tile_meta[tile_of(n)] : make_int4(-1, 0, 0, 0);
      };
      // a tile's record two tiles ahead, its slots one tile ahead
      int4 meta_next = meta_of(0), meta_next2 = meta_of(1);
      uint32_t next_slot = 0;
      if (my_tiles > 0 && lane < meta_next.z) next_slot = p.c.entries[meta_next.y + lane];
      int kv_key = -1, gen = -1, sent = 0;
      for (int n = 0; n < my_tiles; ++n) {
        const int key = meta_next.x, len = meta_next.z;
        const uint32_t myslot = next_slot;
        const int r = (key / p.B) % p.H_kv;
        meta_next = meta_next2;
        next_slot = (n + 1 < my_tiles && lane < meta_next.z) ? p.c.entries[meta_next.y + lane] : 0u;
        meta_next2 = meta_of(n + 2);
        if (key != kv_key || n % L == 0) {
          kv_key = key;
          ++gen;
        }
        const int is = n % kIR, qs = n % QS;
        const int i = p.q0 + static_cast<int>(myslot / per_q);
        if (!mbar_wait_warp(&i_empty[is], ((n / kIR) & 1) ^ 1, abort_flag, p.status, 150)) break;
        TileInfo& ti = info[is];
        if (lane < len) {
          ti.slot[lane] = myslot;
          ti.qi[lane] = i;
        }
        if (lane == 0) {
          ti.r = r;
          ti.len = len;
          ti.gen = gen;
          ti.jb = p.blk[key % p.B].y;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_full[is]);
        if (!mbar_wait_warp(&q_empty[qs], ((n / QS) & 1) ^ 1, abort_flag, p.status, 152)) break;
        if (lane == 0) mbar_arrive_expect_tx(&q_full[qs], len * p.R * D_H * 2);
        __syncwarp();
        const int h0 = p.G >= 8 ? r * p.G : (r * p.G / 8) * 8;
        if (lane < len) {
          uint8_t* dst = sQ + qs * SH::Q_BYTES;
          if (p.q4d) {
            // row-major: [row][d-chunk][8 heads x 128 B]
            tma_load_4d(dst + lane * 8 * D_H * 2, &tm_q, &q_full[qs], 0, h0, 0, i);
          } else {
            // chunk-major: [d-chunk][rows x 128 B]
#pragma unroll
            for (int c = 0; c < SH::DCH; ++c)
              tma_load_3d(dst + c * kRowsPerTile * 128 + lane * p.R * 128, &tm_q, &q_full[qs],
                          c * 64, h0, i);
          }
        }
        ++sent;
      }
      // nothing is still on its way into this CTA's shared memory when it ends,
      // not even after a wait that gave up (so below for the pages)
      for (int j = sent > QS ? sent - QS : 0; j < sent; ++j)
        mbar_wait(&q_full[j % QS], (j / QS) & 1, nullptr, p.status, 156);
    } else if (warp == 6) {
      // ------------------------------------------- raw pages (TMA), ahead --
      if (lane == 0) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        int ring = 0;
        bool ok = true;
        for (int n = 0; ok && n < my_tiles;) {
          const int4 meta = p.c.tile_meta[tile_of(n)];
          const int row = page_of(meta).x * B_K, r = group_of(meta);
          for (int c = 0; ok && c < 2 * SH::CPP; ++c, ++ring) {
            const int rs = ring % kRaw;
            ok = mbar_wait(&raw_empty[rs], ((ring / kRaw) & 1) ^ 1, abort_flag, p.status, 154);
            if (!ok) break;
            mbar_arrive_expect_tx(&raw_full[rs], SH::RAW_BYTES);
            const bool is_v = c >= SH::CPP;
            tma_load_3d(sRaw + rs * SH::RAW_BYTES, is_v ? &tm_v : &tm_k, &raw_full[rs], 0, r,
                        row + (is_v ? c - SH::CPP : c) * 64);
          }
          n = run_end(n, meta);
        }
        for (int j = ring > kRaw ? ring - kRaw : 0; j < ring; ++j)
          mbar_wait(&raw_full[j % kRaw], (j / kRaw) & 1, nullptr, p.status, 157);
      }
    } else if (warp == 7) {
      // ------------------------------------------------------ page scales --
      // Lane l: keys l, l + 32, ...; a generation's scales load while the one
      // before waits for its slot.
      constexpr int KPL = B_K / 32;
      float ks[KPL], vs[KPL];
      int keys = 0;
      auto fetch = [&](int n) {  // the generation that starts at tile n; its successor's first tile
        keys = 0;
        if (n >= my_tiles) return n;
        const int4 meta = p.c.tile_meta[tile_of(n)];
        const int4 b = page_of(meta);
        keys = b.z;
        const int64_t row = static_cast<int64_t>(b.x) * B_K * p.H_kv + group_of(meta);
#pragma unroll
        for (int j = 0; j < KPL; ++j) {
          const int key = lane + 32 * j;
          const bool on = key < keys;
          ks[j] = on ? __ldg(p.ks + row + static_cast<int64_t>(key) * p.H_kv) : 0.f;
          vs[j] = on ? __ldg(p.vs + row + static_cast<int64_t>(key) * p.H_kv) : 0.f;
        }
        return run_end(n, meta);
      };
      int next = fetch(0);
      for (int gen = 0;; ++gen) {
        const int slot = gen % kNKV;
        if (gen >= kNKV &&
            !mbar_wait_warp(&kv_empty[slot], ((gen / kNKV) - 1) & 1, abort_flag, p.status, 155))
          break;
        // Value scales within kEven of one another (the usual page) are
        // stored relative to the largest: the softmax's weights times them
        // are f16 values as they are.  Others are left for it to normalise.
        float hi = 0.f, lo = INFINITY;
#pragma unroll
        for (int j = 0; j < KPL; ++j) {
          hi = fmaxf(hi, fabsf(vs[j]));
          if (lane + 32 * j < keys) lo = fminf(lo, fabsf(vs[j]));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
          lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
        }
        const bool even = hi > 0.f && hi < INFINITY && lo * kEven >= hi;
        float* sc = sSc + slot * SH::SCALES_PAD;
#pragma unroll
        for (int j = 0; j < KPL; ++j) {
          sc[lane + 32 * j] = ks[j] * p.scale_log2;
          sc[B_K + lane + 32 * j] = even ? __fdividef(vs[j], hi) : vs[j];
        }
        if (lane == 0) {
          *reinterpret_cast<float2*>(sc + 2 * B_K) = make_float2(even ? hi : 1.f, even ? 1.f : 0.f);
          gen_keys[slot] = keys;
        }
        const bool more = keys != 0;  // 0: the end, which the widening warps read
        __syncwarp();
        if (lane == 0) mbar_arrive(&sc_full[slot]);
        if (!more) break;
        next = fetch(next);
      }
    } else if (warp == 5 && lane == 0) {
      // ------------------------------------------------------ MMA issuer --
      // the next tiles' S before O(n) when their rows and pages are there, else
      // after (a page may wait for O(n) to free its slot)
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, B_K, 0, 0);
      constexpr uint32_t idesc_o = idesc_f16_f32(128, D_H, 0, 1);
      // one descriptor of each operand: a stage, chunk or K step is an offset
      // of its address field (16-byte units; the field never carries over, the
      // operands lie below 256 KB)
      const uint64_t q_desc = umma_desc(smem_u32(sQ), 16, p.q4d ? 8 * D_H * 2 : 1024, SW_128B);
      const uint32_t q_cstep = (p.q4d ? 8 * 128 : kRowsPerTile * 128) >> 4;
      const uint64_t k_desc = umma_desc(smem_u32(sKV), 16, 1024, SW_128B);
      const uint64_t v_desc = umma_desc(smem_u32(sKV + SH::K_BYTES), B_K * 128, 1024, SW_128B);
      int kv_ready = -1;
      auto prep = [&](int n, int* gen) -> bool {
        if (!mbar_wait(&i_full[n % kIR], (n / kIR) & 1, abort_flag, p.status, 160)) return false;
        *gen = info[n % kIR].gen;
        return true;
      };
      auto s_ready = [&](int n, int gen) -> bool {
        return mbar_test_wait(&q_full[n % QS], (n / QS) & 1) &&
               (gen <= kv_ready || mbar_test_wait(&kv_full[gen % kNKV], (gen / kNKV) & 1));
      };
      auto issue_s = [&](int n, int gen) -> bool {
        if (!mbar_wait(&q_full[n % QS], (n / QS) & 1, abort_flag, p.status, 161)) return false;
        if (gen > kv_ready) {
          if (!mbar_wait(&kv_full[gen % kNKV], (gen / kNKV) & 1, abort_flag, p.status, 162))
            return false;
          kv_ready = gen;
        }
        tc_fence_after();
        const uint64_t qd = q_desc + (n % QS) * (SH::Q_BYTES >> 4);
        const uint64_t kd = k_desc + (gen % kNKV) * (SH::KV_BYTES >> 4);
        const uint32_t tS = tmem_base + (n % kNS) * 128 + SH::TM_S;
#pragma unroll
        for (int c = 0; c < SH::DCH; ++c)
#pragma unroll
          for (int s = 0; s < 4; ++s)
            umma_bf16(tS, qd + c * q_cstep + s * 2, kd + (c * B_K * 128 + s * 32) / 16, idesc_s,
                      (c | s) != 0);
        umma_commit(&s_full[n % kNS]);
        umma_commit(&q_empty[n % QS]);
        return true;
      };
      auto issue_o = [&](int m, int gen, bool last_of_gen) -> bool {
        if (!mbar_wait(&p_full[m % kNS], (m / kNS) & 1, abort_flag, p.status, 163)) return false;
        if (!mbar_wait(&o_empty[m % kNS], ((m / kNS) & 1) ^ 1, abort_flag, p.status, 164))
          return false;
        tc_fence_after();
        const uint64_t vd = v_desc + (gen % kNKV) * (SH::KV_BYTES >> 4);
        const uint32_t tP = tmem_base + (m % kNS) * 128 + SH::TM_S;
        const uint32_t tO = tmem_base + SH::TM_O + (m % kNS) * 128;
#pragma unroll
        for (int k = 0; k < B_K / 16; ++k)  // V: MN-major; 16 keys = two 8-key groups = 2048 B
          umma_bf16_ts(tO, tP + k * 8, vd + k * 2048 / 16, idesc_o, k != 0);
        umma_commit(&o_full[m % kNS]);
        if (last_of_gen) umma_commit(&kv_empty[gen % kNKV]);
        return true;
      };
      // S(n + 1) takes the buffer of tile n - 1, whose O was issued before it
      int g0 = 0, g1 = 0;  // generations of tiles n, n + 1
      bool ok = my_tiles > 0 && prep(0, &g0) && issue_s(0, g0);
      for (int n = 0; ok && n < my_tiles; ++n) {
        const bool more = n + 1 < my_tiles;
        if (more) ok = prep(n + 1, &g1);
        if (!ok) break;
        const bool ahead = more && s_ready(n + 1, g1);
        if (ahead) ok = issue_s(n + 1, g1);
        ok = ok && issue_o(n, g0, !more || g1 != g0);
        if (ok && more && !ahead) ok = issue_s(n + 1, g1);
        g0 = g1;
      }
      // every MMA of this CTA must be done before TMEM is released
      umma_commit(fin);
      mbar_wait(fin, 0, nullptr, p.status, 169);
    }
  } else if (wg == 0) {
    // -------------------------------------------------------- epilogue --
    const int row = warp * 32 + lane;
    const int q_local = row / p.R;
    const int hrow = row - q_local * p.R;
    for (int n = 0; n < my_tiles; ++n) {
      const int is = n % kIR;
      if (!mbar_wait_warp(&i_full[is], (n / kIR) & 1, abort_flag, p.status, 170)) break;
      if (!mbar_wait_warp(&o_full[n % kNS], (n / kNS) & 1, abort_flag, p.status, 171)) break;
      tc_fence_after();
      const TileInfo& ti = info[is];
      const int goff = p.G >= 8 ? 0 : (ti.r * p.G) % 8;  // group's first head in the box
      const bool useful = q_local < ti.len && hrow >= goff && hrow < goff + p.G;
      const int g = hrow - goff;
      const uint32_t slot = useful ? ti.slot[q_local] : 0u;
      // partial layout [slot][d/8][g][8]
      __half* dst = p.c.part_o + static_cast<int64_t>(slot) * p.G * D_H + g * 8;
      const uint32_t tO =
          tmem_base + SH::TM_O + (n % kNS) * 128 + (static_cast<uint32_t>(warp * 32) << 16);
#pragma unroll 1
      for (int c = 0; c < D_H / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(tO + c * 32, v);
        tmem_wait_ld();
        if (c == D_H / 32 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_empty[n % kNS]);
        }
        if (useful) {
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __half2 h = __floats2half2_rn(__uint_as_float(v[j + 2 * e]),
                                                  __uint_as_float(v[j + 2 * e + 1]));
              w[e] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(dst + (c * 4 + j / 8) * p.G * 8) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&i_empty[is]);
    }
  } else {
    // ---------------------------------------------------------- softmax --
    // Two teams of eight warps take the even and the odd tiles.  Warps w and
    // w + 4 of a team share TMEM lane quarter w % 4, 16 lanes each; a thread
    // holds rows A and B = A + 8 x the keys 8r + 2c, 8r + 2c + 1 of 32 keys
    // at a time (c = lane % 4, r = 0 .. 3), so a scale serves two rows and a
    // row's reductions are two shuffles.  S is read twice, for the maximum and
    // for the weights, 32 keys ahead: the loops are short, so that the teams'
    // code stays in the instruction caches, and 72 registers are enough for
    // 16 warps (straight-line code over a row's keys with half the warps: 410
    // us on 18000 tiles, this 349 when they were compared; there ncu counts 4.4
    // warps per issue that wait for instructions, here 1.1).
    const int team = (warp - 8) >> 3;
    const int lane0 = (warp & 3) * 32 + ((warp >> 2) & 1) * 16;
    const int cq = lane & 3;
    const int rowA = lane0 + (lane >> 2), rowB = rowA + 8;
    const int qA = rowA / p.R, qB = rowB / p.R;
    for (int n = team; n < my_tiles; n += 2) {
      const int is = n % kIR, st = n % kNS;
      if (!mbar_wait_warp(&i_full[is], (n / kIR) & 1, abort_flag, p.status, 180)) break;
      const TileInfo& ti = info[is];
      const int jb = ti.jb + 2 * cq;
      const int iA = qA < ti.len ? ti.qi[qA] - jb : INT_MAX, iB = qB < ti.len ? ti.qi[qB] - jb : INT_MAX;
      // a row's own block: keys past the row (warp-uniform)
      const bool cut = __any_sync(0xFFFFFFFFu, (iA < iB ? iA : iB) < B_K);
      // page scales: they stay until the page's last O = P V is done
      const float* sc = sSc + (ti.gen % kNKV) * SH::SCALES_PAD;
      if (!mbar_wait_warp(&s_full[st], (n / kNS) & 1, abort_flag, p.status, 181)) break;
      tc_fence_after();
      const uint32_t tS = tmem_base + st * 128 + SH::TM_S + (static_cast<uint32_t>(lane0) << 16);
      const float unit = sc[2 * B_K];
      const bool even = sc[2 * B_K + 1] != 0.f;
      sc += 2 * cq;
      // body(c, v): keys 32 c .. of the two rows, the next 32 on their way
      auto sweep = [&](auto body) {
        uint32_t a[16], b[16];
        tmem_ld_16x256b_x4(tS, a);
#pragma unroll 1
        for (int c = 0; c < B_K / 32; c += 2) {
          tmem_wait_ld();
          tmem_ld_16x256b_x4(tS + 32 * (c + 1), b);
          body(c, a);
          tmem_wait_ld();
          if (c + 2 < B_K / 32) tmem_ld_16x256b_x4(tS + 32 * (c + 2), a);
          body(c + 1, b);
        }
      };
      auto pair = [](const uint32_t (&v)[16], int i) {
        return f2_pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
      };
      float mA = -INFINITY, mB = -INFINITY, fA = unit, fB = unit;
      uint64_t lA2 = f2_pack(0.f, 0.f), lB2 = lA2;
      // The usual tile has no key to mask and an even page: its loops carry
      // neither test.
      auto softmax = [&](auto special) {
        constexpr bool kSpecial = decltype(special)::value;
        const bool mask = kSpecial && cut;
        sweep([&](int c, const uint32_t (&v)[16]) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float2 k2 = *reinterpret_cast<const float2*>(sc + 32 * c + 8 * r);
            const uint64_t kk = f2_pack(k2.x, k2.y);
            uint64_t a = f2_mul(pair(v, 4 * r), kk), b = f2_mul(pair(v, 4 * r + 2), kk);
            if (mask) {
              const int j = 32 * c + 8 * r;
              a = f2_pack(j <= iA ? f2_lo(a) : -INFINITY, j < iA ? f2_hi(a) : -INFINITY);
              b = f2_pack(j <= iB ? f2_lo(b) : -INFINITY, j < iB ? f2_hi(b) : -INFINITY);
            }
            mA = fmax3(mA, f2_lo(a), f2_hi(a));
            mB = fmax3(mB, f2_lo(b), f2_hi(b));
          }
        });
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          mA = fmaxf(mA, __shfl_xor_sync(0xFFFFFFFFu, mA, o));
          mB = fmaxf(mB, __shfl_xor_sync(0xFFFFFFFFu, mB, o));
        }
        // the weights of keys j, j + 1 of a row: S is scaled again (one fma)
        auto weights = [&](uint64_t s2, uint64_t kk, uint64_t nm, int j, int i) {
          const uint64_t x = f2_fma(s2, kk, nm);
          float e0 = ex2_ftz(f2_lo(x)), e1 = ex2_ftz(f2_hi(x));
          if (mask) {
            e0 = j <= i ? e0 : 0.f;
            e1 = j < i ? e1 : 0.f;
          }
          return f2_pack(e0, e1);
        };
        // times their value scales; 0 * NaN of a key that the row does not see is 0
        auto scaled = [&](uint64_t e, uint64_t vv, int j, int i) {
          uint64_t w = f2_mul(e, vv);
          if (mask) w = f2_pack(j <= i ? f2_lo(w) : 0.f, j < i ? f2_hi(w) : 0.f);
          return w;
        };
        const uint64_t nmA = f2_pack(-mA, -mA), nmB = f2_pack(-mB, -mB);
        uint64_t uA = f2_pack(1.f, 1.f), uB = uA;
        if (kSpecial && !even) {  // the rows' largest weights times scales
          fA = fB = 0.f;
          sweep([&](int c, const uint32_t (&v)[16]) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int j = 32 * c + 8 * r;
              const float2 k2 = *reinterpret_cast<const float2*>(sc + j);
              const float2 v2 = *reinterpret_cast<const float2*>(sc + B_K + j);
              const uint64_t kk = f2_pack(k2.x, k2.y), vv = f2_pack(v2.x, v2.y);
              const uint64_t a = scaled(weights(pair(v, 4 * r), kk, nmA, j, iA), vv, j, iA);
              const uint64_t b = scaled(weights(pair(v, 4 * r + 2), kk, nmB, j, iB), vv, j, iB);
              fA = fmax3(fA, fabsf(f2_lo(a)), fabsf(f2_hi(a)));
              fB = fmax3(fB, fabsf(f2_lo(b)), fabsf(f2_hi(b)));
            }
          });
#pragma unroll
          for (int o = 1; o < 4; o <<= 1) {
            fA = fmaxf(fA, __shfl_xor_sync(0xFFFFFFFFu, fA, o));
            fB = fmaxf(fB, __shfl_xor_sync(0xFFFFFFFFu, fB, o));
          }
          const float a = fA > 0.f ? 1.f / fA : 0.f, b = fB > 0.f ? 1.f / fB : 0.f;
          uA = f2_pack(a, a);
          uB = f2_pack(b, b);
        }
        sweep([&](int c, const uint32_t (&v)[16]) {
          uint32_t pk[8];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int j = 32 * c + 8 * r;
            const float2 k2 = *reinterpret_cast<const float2*>(sc + j);
            const float2 v2 = *reinterpret_cast<const float2*>(sc + B_K + j);
            const uint64_t kk = f2_pack(k2.x, k2.y), vv = f2_pack(v2.x, v2.y);
            const uint64_t ea = weights(pair(v, 4 * r), kk, nmA, j, iA);
            const uint64_t eb = weights(pair(v, 4 * r + 2), kk, nmB, j, iB);
            lA2 = f2_add(lA2, ea);
            lB2 = f2_add(lB2, eb);
            uint64_t wa = scaled(ea, vv, j, iA), wb = scaled(eb, vv, j, iB);
            if (kSpecial && !even) {
              wa = f2_mul(wa, uA);
              wb = f2_mul(wb, uB);
            }
            const __half2 ha = __floats2half2_rn(f2_lo(wa), f2_hi(wa));
            const __half2 hb = __floats2half2_rn(f2_lo(wb), f2_hi(wb));
            pk[2 * r] = *reinterpret_cast<const uint32_t*>(&ha);
            pk[2 * r + 1] = *reinterpret_cast<const uint32_t*>(&hb);
          }
          tmem_st_16x128b_x4(tS + 16 * c, pk);  // over S that was read
        });
      };
      if (cut || !even) softmax(std::true_type{});
      else softmax(std::false_type{});
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[st]);
      // off the way to O: the rows' LSEs and factors
      float lA = f2_lo(lA2) + f2_hi(lA2), lB = f2_lo(lB2) + f2_hi(lB2);
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        lA += __shfl_xor_sync(0xFFFFFFFFu, lA, o);
        lB += __shfl_xor_sync(0xFFFFFFFFu, lB, o);
      }
      if (cq < 2) {  // lane 0 of the four writes row A, lane 1 row B
        const int q = cq == 0 ? qA : qB;
        const int h = (cq == 0 ? rowA : rowB) - q * p.R - (p.G >= 8 ? 0 : (ti.r * p.G) % 8);
        if (q < ti.len && h >= 0 && h < p.G) {
          const int64_t at = static_cast<int64_t>(ti.slot[q]) * p.G + h;
          const float l = cq == 0 ? lA : lB;
          p.c.part_lse[at] = (cq == 0 ? mA : mB) + __log2f(l);
          p.part_f[at] = __fdividef(cq == 0 ? fA : fB, l);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&i_empty[is]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// Row t: {t - position, its sequence's first block}, or a first key so late
// that the row has no block (skipped rows).  Block g = s * max_pages + b:
// {page or -1, first key as a row number, keys that exist, 0}.  Also the start
// values: no entries per key, no LSE per slot.
__global__ void __launch_bounds__(256) chunk_tables_kernel(const ChunkSeqs c, int2* qinfo, int4* blk,
                                                           int32_t* counts, int64_t nkeys,
                                                           float4* lse, int64_t n_lse4,
                                                           DevStatus* status) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const float inf = INFINITY;
  for (int64_t j = i; j < n_lse4; j += static_cast<int64_t>(gridDim.x) * blockDim.x)
    lse[j] = make_float4(-inf, -inf, -inf, -inf);
  if (i < nkeys) counts[i] = 0;
  if (i < c.T) {
    const int t = static_cast<int>(i);
    const ChunkTok k = chunk_tok(c, t);
    if (k.too_long) report(status, DEV_ERR_CACHE_FULL, 140, k.s, t);
    qinfo[t] = k.pos >= 0 ? make_int2(t - k.pos, k.s * c.max_pages) : make_int2(t + 2 * c.B_k, 0);
  }
  const int64_t B = static_cast<int64_t>(c.S) * c.max_pages;
  if (i < B) {
    const int s = static_cast<int>(i / c.max_pages);
    const int b = static_cast<int>(i - static_cast<int64_t>(s) * c.max_pages);
    // of the sequence's rows in the chunk: where they start and how many keys
    // there are with them.  A sequence without rows here has no entries.
    const int c0 = c.cu[s], c1 = c.cu[s + 1], len = c.seq_len[s];
    int4 rec = make_int4(-1, 0, 0, 0);
    if (c0 >= 0 && c1 > c0 && c1 <= c.T && len >= 0) {
      const int64_t end = static_cast<int64_t>(len) + (c1 - c0);
      const int64_t left = end - static_cast<int64_t>(b) * c.B_k;
      if (end <= static_cast<int64_t>(c.max_pages) * c.B_k && left > 0) {
        const int64_t pg = chunk_page(c, s, b);
        rec = make_int4(static_cast<int>(pg), c0 - len + b * c.B_k,
                        static_cast<int>(left < c.B_k ? left : c.B_k), 0);
      }
    }
    blk[i] = rec;
  }
}

// The inverse index of few keys (up to kFewKeys; more go through
// inv_index.cu's multi-CTA scan), in three short kernels:
//   rank   every selection's key and its place in the key's list, by counting:
//          a warp takes one (group, slot) of 32 consecutive rows, which mostly
//          agree on the hot blocks (the first one, their own), so that those
//          cost one atomic a warp;
//   scan   one CTA: where each key's list and its tiles start;
//   place  the selections to their places, and the tiles' records.
constexpr int64_t kFewKeys = 32768;
constexpr int kPlaceRows = 32;  // rows per CTA of rank

// `rank`: {key or -1, place}, a CTA's selections as [group, slot][row].
__global__ void __launch_bounds__(1024) chunk_rank_kernel(const InvParams p, int2* rank) {
  extern __shared__ int32_t sel[];  // [kPlaceRows][H_kv * k]
  griddep_wait();
  const int per_q = p.H_kv * p.kk;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kPlaceRows;
  const int rows = static_cast<int>(p.nq - row0 < kPlaceRows ? p.nq - row0 : kPlaceRows);
  const int32_t* src = p.idx + (p.q0 + row0) * per_q;
  for (int i = threadIdx.x; i < rows * per_q; i += blockDim.x) sel[i] = __ldg(src + i);
  const int lane = threadIdx.x & 31;
  const int t = static_cast<int>(p.q0 + row0) + lane;
  const int2 sq = lane < rows ? __ldg(p.qinfo + t) : make_int2(INT_MAX, 0);
  const int own = lane < rows && t >= sq.x ? (t - sq.x) / p.B_k : -1;
  __syncthreads();
  for (int c = threadIdx.x >> 5; c < per_q; c += blockDim.x >> 5) {
    // a skipped row's entries were never written: they are not looked at
    const int b = own >= 0 ? sel[lane * per_q + c] : -1;
    int key = -1;
    if (b < -1 || b >= p.B_seq) {
      report(p.status, DEV_ERR_BAD_INDEX, 141, t, b);
    } else if (b >= 0 && b <= own) {
      if (__ldg(&p.blk[sq.y + b].x) >= 0) key = c / p.kk * static_cast<int>(p.B) + sq.y + b;
      else report(p.status, DEV_ERR_BAD_INDEX, 142, t, b);
    }
    const unsigned peers = __match_any_sync(0xFFFFFFFFu, key);
    const int leader = __ffs(peers) - 1;
    int base = 0;
    if (lane == leader && key >= 0) base = atomicAdd(&p.c.counts[key], __popc(peers));
    base = __shfl_sync(0xFFFFFFFFu, base, leader);
    rank[(static_cast<int64_t>(blockIdx.x) * per_q + c) * 32 + lane] =
        make_int2(key, base + __popc(peers & ((1u << lane) - 1)));
  }
}

__global__ void __launch_bounds__(1024) chunk_scan_kernel(const InvParams p, int nkeys) {
  griddep_wait();
  __shared__ int2 ws[32];
  __shared__ int2 carry;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  if (threadIdx.x == 0) carry = make_int2(0, 0);
  __syncthreads();
  for (int base = 0; base < nkeys; base += 4096) {
    const int k0 = base + threadIdx.x * 4;
    int cnt[4], a = 0, b = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      cnt[j] = k0 + j < nkeys ? p.c.counts[k0 + j] : 0;
      a += cnt[j];
      b += (cnt[j] + p.Tq - 1) / p.Tq;
    }
    int x = a, y = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, x, o), v = __shfl_up_sync(0xFFFFFFFFu, y, o);
      if (lane >= o) {
        x += u;
        y += v;
      }
    }
    if (lane == 31) ws[w] = make_int2(x, y);
    __syncthreads();
    if (w == 0) {
      int2 t = ws[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, t.x, o), v = __shfl_up_sync(0xFFFFFFFFu, t.y, o);
        if (lane >= o) {
          t.x += u;
          t.y += v;
        }
      }
      ws[lane] = t;
    }
    __syncthreads();
    int run_a = carry.x + x - a + (w > 0 ? ws[w - 1].x : 0);
    int run_b = carry.y + y - b + (w > 0 ? ws[w - 1].y : 0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k0 + j < nkeys) {
        p.c.offsets[k0 + j] = run_a;
        p.c.tile_off[k0 + j] = run_b;
        run_a += cnt[j];
        run_b += (cnt[j] + p.Tq - 1) / p.Tq;
      }
    __syncthreads();
    if (threadIdx.x == 0) {
      carry.x += ws[31].x;
      carry.y += ws[31].y;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    p.c.offsets[nkeys] = carry.x;
    p.c.tile_off[nkeys] = carry.y;
    p.c.n_tiles[0] = carry.y;
  }
}

// A thread per selection and, for the records, a thread per key; the tiles of a
// long list are written by the key's warp.
__global__ void __launch_bounds__(256) chunk_place_kernel(const InvParams p, const int2* rank,
                                                         int64_t n_rank, int nkeys) {
  griddep_wait();
  constexpr int kOwn = 4;  // records that a key's thread writes itself
  const int per_q = p.H_kv * p.kk;
  const int lane = threadIdx.x & 31;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i < n_rank) {
    const int2 k = __ldg(rank + i);
    if (k.x >= 0) {
      const int64_t col = i >> 5, block = col / per_q;
      const int64_t e = (block * kPlaceRows + (i & 31)) * per_q + (col - block * per_q);
      p.c.entries[p.c.offsets[k.x] + k.y] = static_cast<uint32_t>(e);
    }
  }
  const int64_t threads = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t k0 = i - lane; k0 < nkeys; k0 += threads) {  // whole warps
    const int key = static_cast<int>(k0) + lane;
    int t0 = 0, t1 = 0, first = 0, end = 0;
    if (key < nkeys) {
      t0 = p.c.tile_off[key];
      t1 = p.c.tile_off[key + 1];
      first = p.c.offsets[key];
      end = p.c.offsets[key + 1];
    }
    auto put = [&](int key_, int t, int at, int end_, int t1_) {
      p.c.tile_meta[t] = make_int4(key_, at, end_ - at < p.Tq ? end_ - at : p.Tq, t1_);
    };
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
      if (t0 + j < t1) put(key, t0 + j, first + j * p.Tq, end, t1);
    unsigned more = __ballot_sync(0xFFFFFFFFu, t1 - t0 > kOwn);
    for (; more != 0; more &= more - 1) {
      const int src = __ffs(more) - 1;
      const int a = __shfl_sync(0xFFFFFFFFu, t0, src), b = __shfl_sync(0xFFFFFFFFu, t1, src);
      const int f = __shfl_sync(0xFFFFFFFFu, first, src), z = __shfl_sync(0xFFFFFFFFu, end, src);
      for (int j = kOwn + lane; a + j < b; j += 32)
        put(static_cast<int>(k0) + src, a + j, f + j * p.Tq, z, b);
    }
  }
}

struct MergeParams {
  __nv_bfloat16* o;
  float* lse;
  int q0, nq;
  int H_q, H_kv, kk;
  const int2* qinfo;
  const __half* part_o;
  const float* part_lse;
  const float* part_f;
};

// Merge: one thread per 8 consecutive outputs of a head, the G * D / 8 threads
// of a (row, group) in the partials' order [d/8][g].  The first slots' partials
// (16 bytes each, coalesced) are on their way while the slots' LSEs become
// weights: the R lanes of a warp that share a head take R slots at a time, their
// maximum and sum are shuffles, and a slot's weight comes from its lane when its
// partial is due.  No barrier: with the weights in shared memory, made once per
// CTA, the 537 MB of the case above took 129 us, this 88 (6.1 TB/s).
template <int D, int G>
__global__ void __launch_bounds__(256) chunk_merge_kernel(const MergeParams p) {
  griddep_wait();
  constexpr int NB = 8;  // slots in flight
  constexpr int PER_UNIT = G * D / 8;
  constexpr int LANES = PER_UNIT < 32 ? PER_UNIT : 32;  // of a unit in one warp
  constexpr int R = LANES / G;
  constexpr int NJ = (32 + R - 1) / R;  // slots per lane
  const int lane = threadIdx.x & 31, el = lane % LANES;
  const int u = threadIdx.x / PER_UNIT, e = threadIdx.x - u * PER_UNIT;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (blockDim.x / PER_UNIT) + u;
  const bool on = unit < static_cast<int64_t>(p.nq) * p.H_kv;
  constexpr int64_t stride = static_cast<int64_t>(G) * D;
  const int64_t slot0 = (on ? unit : 0) * p.kk;
  const __half* base = p.part_o + slot0 * stride + e * 8;
  uint4 x[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
    x[j] = j < p.kk ? __ldcs(reinterpret_cast<const uint4*>(base + j * stride))
                    : make_uint4(0, 0, 0, 0);
  const int g = e % G;
  float z[NJ], w[NJ];
  float m = -INFINITY, l = 0.f;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int s = j * R + el / G;
    z[j] = -INFINITY;  // -inf: an unused slot, the rest of it was never written
    w[j] = 0.f;
    if (s < p.kk) {
      const int64_t at = (slot0 + s) * G + g;
      z[j] = p.part_lse[at];
      w[j] = p.part_f[at];
    }
    m = fmaxf(m, z[j]);
  }
#pragma unroll
  for (int o = G; o < LANES; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  const float ms = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const float t = exp2f(z[j] - ms);
    l += t;
    w[j] = z[j] == -INFINITY ? 0.f : t * w[j];
  }
#pragma unroll
  for (int o = G; o < LANES; o <<= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
#pragma unroll
  for (int s0 = 0; s0 < 32; s0 += NB) {
    if (s0 >= p.kk) break;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const int s = s0 + j;
      const float ws = __shfl_sync(0xFFFFFFFFu, w[s / R], lane - el + s % R * G + g);
      const __half2* h = reinterpret_cast<const __half2*>(&x[j]);
      if (ws != 0.f)  // nothing of an unused slot
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 v = __half22float2(h[q]);
          acc[2 * q] = fmaf(ws, v.x, acc[2 * q]);
          acc[2 * q + 1] = fmaf(ws, v.y, acc[2 * q + 1]);
        }
      if (s + NB < p.kk)
        x[j] = __ldcs(reinterpret_cast<const uint4*>(base + (s + NB) * stride));
    }
  }
  if (!on) return;
  const int il = static_cast<int>(unit / p.H_kv);
  const int r = static_cast<int>(unit - static_cast<int64_t>(il) * p.H_kv);
  const int t = p.q0 + il;
  if (t < __ldg(&p.qinfo[t].x)) return;  // a skipped row
  const int d0 = e / G * 8;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t head = static_cast<int64_t>(t) * p.H_q + r * G + g;
  *reinterpret_cast<uint4*>(p.o + head * D + d0) =
      make_uint4(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv),
                 pack_bf16(acc[4] * inv, acc[5] * inv), pack_bf16(acc[6] * inv, acc[7] * inv));
  if (p.lse != nullptr && d0 == 0) p.lse[head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <int D>
auto merge_kernel(int G) {
  switch (G) {
    case 1: return chunk_merge_kernel<D, 1>;
    case 2: return chunk_merge_kernel<D, 2>;
    case 4: return chunk_merge_kernel<D, 4>;
    case 8: return chunk_merge_kernel<D, 8>;
    default: return chunk_merge_kernel<D, 16>;  // the form takes divisors of 16
  }
}

struct KVBufs {
  ChunkBufs c;
  int2* rank;
  float* part_f;
  int2* qinfo;
  int4* blk;
};

KVBufs carve_kv(void* ws, int T, int64_t B, int H_q, int H_kv, int d_h, int kk, int64_t Nc,
                size_t* total) {
  KVBufs b;
  size_t off = 0;
  b.c = carve(ws, Nc, H_q, H_kv, d_h, kk, inv_nkeys(Nc, kWindow, H_kv, B), &off);
  uint8_t* p = static_cast<uint8_t*>(ws);
  auto take = [&](size_t bytes) {
    uint8_t* r = p ? p + off : nullptr;
    off += align256(bytes);
    return r;
  };
  b.rank = reinterpret_cast<int2*>(take(sizeof(int2) * (Nc + kPlaceRows) * H_kv * kk));
  b.part_f = reinterpret_cast<float*>(take(sizeof(float) * Nc * kk * H_q));
  b.qinfo = reinterpret_cast<int2*>(take(sizeof(int2) * T));
  b.blk = reinterpret_cast<int4*>(take(sizeof(int4) * B));
  *total = off;
  return b;
}

// Rows per window: bounds the partials.
int64_t window_of(int T) { return T < kMaxChunk ? T : kMaxChunk; }

template <int D_H, int B_K>
size_t tile_smem() {
  using SH = KVShape<D_H, B_K>;
  return 1024 + SH::QS * SH::Q_BYTES + kNKV * SH::KV_BYTES + kNKV * SH::SCALES_PAD * 4 + kRaw * SH::RAW_BYTES +
         kIR * sizeof(TileInfo) + (2 * SH::QS + 2 * kRaw + 3 * kNKV + 2 * kIR + 4 * kNS + 1) * 8 + 16;
}

template <int D_H, int B_K>
cudaError_t launch_typed(const AttendLaunch& a, cudaStream_t stream) {
  static_assert(sizeof(TileInfo) * kIR + (8 + 2 * kRaw + 3 * kNKV + 2 * kIR + 4 * kNS + 1) * 8 + 16 <= 2048,
                "tile info and barriers fit what the Q ring leaves them");
  const int T = a.c.T;
  const int G = a.H_q / a.H_kv;
  const int R = rows_per_query(G);
  const int64_t B = static_cast<int64_t>(a.c.S) * a.c.max_pages;
  const int64_t Nc = window_of(T);
  size_t need = 0;
  const KVBufs b = carve_kv(a.ws, T, B, a.H_q, a.H_kv, a.d_h, a.k, Nc, &need);

  CUtensorMap tq;
  int q4d = 0;
  if (R == 8) {
    const uint64_t dims[4] = {64, static_cast<uint64_t>(a.H_q), static_cast<uint64_t>(D_H / 64),
                              static_cast<uint64_t>(T)};
    const uint64_t strides[3] = {static_cast<uint64_t>(D_H) * 2, 128,
                                 static_cast<uint64_t>(a.H_q) * D_H * 2};
    const uint32_t box[4] = {64, 8, static_cast<uint32_t>(D_H / 64), 1};
    q4d = make_tmap_bf16(&tq, a.q, 4, dims, strides, box, 128) ? 1 : 0;
  }
  if (!q4d) {
    const uint64_t dims[3] = {static_cast<uint64_t>(D_H), static_cast<uint64_t>(a.H_q),
                              static_cast<uint64_t>(T)};
    const uint64_t strides[2] = {static_cast<uint64_t>(D_H) * 2,
                                 static_cast<uint64_t>(a.H_q) * D_H * 2};
    const uint32_t box[3] = {64, static_cast<uint32_t>(R), 1};
    if (!make_tmap_bf16(&tq, a.q, 3, dims, strides, box, 128)) return cudaErrorInvalidValue;
  }
  // pages as rows of D_H bytes (maps of 16-bit elements: only bytes move)
  CUtensorMap tk, tv;
  {
    const uint64_t dims[3] = {static_cast<uint64_t>(D_H) / 2, static_cast<uint64_t>(a.H_kv),
                              static_cast<uint64_t>(a.c.n_pages) * B_K};
    const uint64_t strides[2] = {static_cast<uint64_t>(D_H), static_cast<uint64_t>(a.H_kv) * D_H};
    const uint32_t box[3] = {static_cast<uint32_t>(D_H) / 2, 1, 64};
    if (!make_tmap_bf16(&tk, a.k_pages, 3, dims, strides, box, 0)) return cudaErrorInvalidValue;
    if (!make_tmap_bf16(&tv, a.v_pages, 3, dims, strides, box, 0)) return cudaErrorInvalidValue;
  }
  const size_t smem = tile_smem<D_H, B_K>();
  cudaError_t e = cudaFuncSetAttribute(chunk_tile_kernel<D_H, B_K>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int sms = num_sms();
  for (int64_t q0 = 0; q0 < T; q0 += Nc) {
    const int64_t nq = T - q0 < Nc ? T - q0 : Nc;
    const int64_t nkeys = inv_nkeys(nq, kWindow, a.H_kv, B);
    int64_t work = nkeys > T ? nkeys : T;
    if (B > work) work = B;
    const int64_t n_lse4 = (nq * a.k * a.H_q + 3) / 4;  // the buffer is padded to 256 bytes
    if (work < 256 * sms) work = 256 * sms;
    prof_begin("chunk_tables", stream);
    chunk_tables_kernel<<<static_cast<unsigned>((work + 255) / 256), 256, 0, stream>>>(
        a.c, b.qinfo, b.blk, b.c.counts, nkeys, reinterpret_cast<float4*>(b.c.part_lse), n_lse4,
        a.status);
    prof_end(stream);
    InvParams ip{};
    ip.idx = a.idx;
    ip.q0 = q0;
    ip.nq = nq;
    ip.H_kv = a.H_kv;
    ip.B_k = a.c.B_k;
    ip.kk = a.k;
    ip.B = B;
    ip.qinfo = b.qinfo;
    ip.blk = b.blk;
    ip.B_seq = a.c.max_pages;
    ip.Tq = kRowsPerTile / R;
    ip.Cw = kWindow;
    ip.W = static_cast<int>((nq + kWindow - 1) / kWindow);
    ip.c = b.c;
    ip.status = a.status;
    if (nkeys <= kFewKeys) {
      const unsigned blocks = static_cast<unsigned>((nq + kPlaceRows - 1) / kPlaceRows);
      const size_t rows = sizeof(int32_t) * kPlaceRows * a.H_kv * a.k;  // at most 32 KB
      prof_begin("chunk_rank", stream);
      e = launch_pdl(chunk_rank_kernel, dim3(blocks), dim3(1024), rows, stream, ip, b.rank);
      prof_end(stream);
      if (e != cudaSuccess) return e;
      prof_begin("chunk_scan", stream);
      e = launch_pdl(chunk_scan_kernel, dim3(1), dim3(1024), 0, stream, ip, static_cast<int>(nkeys));
      prof_end(stream);
      if (e != cudaSuccess) return e;
      prof_begin("chunk_place", stream);
      const int64_t n_rank = static_cast<int64_t>(blocks) * kPlaceRows * a.H_kv * a.k;
      e = launch_pdl(chunk_place_kernel, dim3(static_cast<unsigned>((n_rank + 255) / 256)), dim3(256), 0,
                     stream, ip, static_cast<const int2*>(b.rank), n_rank, static_cast<int>(nkeys));
      prof_end(stream);
      if (e != cudaSuccess) return e;
    } else {
      size_t hist_bytes = 0;
      int hist_grid = 0;
      e = inv_setup(a.H_kv * B, sms, &hist_bytes, &hist_grid);
      if (e != cudaSuccess) return e;
      launch_inv_index(ip, hist_bytes, hist_grid, sms, stream);
    }

    KVParams kp{};
    kp.q4d = q4d;
    kp.H_kv = a.H_kv;
    kp.kk = a.k;
    kp.G = G;
    kp.R = R;
    kp.B = static_cast<int>(B);
    kp.q0 = static_cast<int>(q0);
    kp.blk = b.blk;
    kp.ks = a.k_scale;
    kp.vs = a.v_scale;
    kp.scale_log2 = a.scale * 1.4426950408889634f;
    kp.c = b.c;
    kp.part_f = b.part_f;
    kp.status = a.status;
    prof_begin("chunk_tile", stream);
    e = launch_pdl(chunk_tile_kernel<D_H, B_K>, dim3(sms), dim3(kThreads), smem, stream, tq, tk, tv,
                   kp);
    prof_end(stream);
    if (e != cudaSuccess) return e;

    MergeParams mp{};
    mp.o = static_cast<__nv_bfloat16*>(a.o);
    mp.lse = a.lse;
    mp.q0 = static_cast<int>(q0);
    mp.nq = static_cast<int>(nq);
    mp.H_q = a.H_q;
    mp.H_kv = a.H_kv;
    mp.kk = a.k;
    mp.qinfo = b.qinfo;
    mp.part_o = b.c.part_o;
    mp.part_lse = b.c.part_lse;
    mp.part_f = b.part_f;
    const int per_unit = G * D_H / 8;  // 8 .. 256 threads
    const int block = per_unit > 128 ? per_unit : 128;
    const int64_t units = block / per_unit;
    prof_begin("chunk_merge", stream);
    e = launch_pdl(merge_kernel<D_H>(G),
                   dim3(static_cast<unsigned>((nq * a.H_kv + units - 1) / units)), dim3(block), 0,
                   stream, mp);
    prof_end(stream);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace

size_t chunk_attend_kv_workspace_bytes(int T, int S, int max_pages, int H_q, int H_kv, int d_h,
                                       int k) {
  size_t total = 0;
  carve_kv(nullptr, T, static_cast<int64_t>(S) * max_pages, H_q, H_kv, d_h, k, window_of(T), &total);
  return total;
}

cudaError_t launch_chunk_attend_kv(const AttendLaunch& a, cudaStream_t s) {
  if (a.d_h == 128)
    return a.c.B_k == 128 ? launch_typed<128, 128>(a, s) : launch_typed<128, 64>(a, s);
  return a.c.B_k == 128 ? launch_typed<64, 128>(a, s) : launch_typed<64, 64>(a, s);
}

}  // namespace msa
