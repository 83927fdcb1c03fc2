// fa_decode.cuh -- attention of one new token per sequence over the paged cache.
//
// Per sequence b and cache head h, with the G = Hq / H query heads that share it as
// the columns of Q^T and the visible positions as rows:
//   S^T = K Q^T,  P = 2^(c S - m) (c = scale * log2 e, m the running maximum),
//   O^T = V^T P,  l = sum_j P_j,  o = O / l,  lse = (m + log2 l) ln 2.
// Nearly all of the work is reading K and V once: 4 G d operations for 4 d bytes (bf16)
// of a position and head.  So keys are the M axis of the tensor instructions and heads
// the N axis: K and V go from memory to shared memory by TMA and from there to the
// tensor core, and no thread ever holds an element of them.  A thread's work is one
// key's G scores.
//
// Work split.  A tile is 128 positions of one (sequence, cache head, block of at most GB
// query heads).  All tiles, in that order, are dealt out evenly: CTA c of nc takes tiles
// [T c / nc, T (c + 1) / nc), so SMs finish together whatever the lengths, and a sequence
// is split over the cache's length exactly where a CTA's share ends.  A CTA walks its
// share as segments (runs of one item's tiles); an item held by one CTA is written out
// whole, the others leave (m, l, O) per segment in the workspace and fa_decode_join_kernel
// adds them up in a fixed order.
//
// Precision.  N is at least 16 in an M = 128 instruction, so for G <= 8 half of it is
// idle; the idle columns carry the low part of the operand that has to be rounded:
// * bf16: P = hi + lo, both bf16 (16 significant bits), as 2 GB columns of O^T;
// * e4m3: codes are multiplied as they are (kind::f8f6f4), the factor of K goes into the
//   score, that of V into the weight.  q (8 bits, scaled by a power of two per head) is
//   hi + lo / 16 in e4m3, exact to 2^-20 of the head's largest element; weights are
//   hi + mid / 16 + lo / 256, 12 bits and not less than 2^-22 of the largest weight.
// The columns' sums meet again in fp32.
#pragma once

#include <cstdint>

#include "fa_cache.cuh"
#include "ptx.cuh"

namespace fa {

constexpr int kDecodeMaxCtas = 192;  // workspace slots; the grid never exceeds it

struct DecodeParams {
  CacheView c;
  const uint16_t *q;  // [B, Hq, d]
  uint16_t *o;        // [B, Hq, d]
  float *lse;         // [B, Hq] or null
  int Hq, G;          // query heads, and query heads per cache head
  int nblk;           // blocks of GB query heads per cache head
  int window;         // 0: all positions
  float scale_log2;   // scale * log2(e)
  int4 *meta;         // [kDecodeMaxCtas] item whose parts start at CTA c: {b, item, parts, -}; parts 0: none
  float2 *part_ml;    // [2 * kDecodeMaxCtas][GB] (m, l) of a part
  float *part_o;      // [2 * kDecodeMaxCtas][GB][d]
};

template <int D, bool E4M3, int GB>
struct DecodeCfg {
  static constexpr int kElem = E4M3 ? 1 : 2;
  static constexpr int kRowBytes = D * kElem;
  static constexpr int kPanelRow = kRowBytes < 128 ? kRowBytes : 128;  // bytes of a row in one swizzled panel
  static constexpr int kPanels = kRowBytes / kPanelRow;
  static constexpr int kPanelBytes = 128 * kPanelRow;
  static constexpr int kTileBytes = 128 * kRowBytes;
  static constexpr int kQCols = E4M3 ? 2 * GB : (GB < 16 ? 16 : GB);
  static constexpr int kOParts = E4M3 ? 3 : 2;
  static constexpr int kOCols = (kOParts * GB + 15) / 16 * 16;
  static constexpr int kQBytes = kQCols * kRowBytes;
  static constexpr int kPBytes = kOCols * 128 * kElem;
  static constexpr int kScStages = 8;  // ring of the keys' factors (e4m3)
  // A score may exceed the running reference by kGrow (log2) before the reference moves;
  // e4m3 weights leave room for it below 448.
  static constexpr float kGrow = E4M3 ? 3.f : 8.f;
  static constexpr float kWeight = 32.f;  // e4m3: a weight of 1 is code value 32, 2^kGrow is 256

  static constexpr int kPOff = 0;
  static constexpr int kQOff = kPOff + 2 * kPBytes;
  static constexpr int kScOff = kQOff + 2 * kQBytes;
  static constexpr int kMiscOff = kScOff + (E4M3 ? kScStages * 1024 : 0);
  // float: xmax[2][GB][4], lpart[2][4][GB], mref[2][GB], qscale[2][GB], vmax[2][4], vref[2] (+2)
  static constexpr int kMiscFloats = 2 * GB * 4 + 2 * 4 * GB + 2 * GB + 2 * GB + 8 + 4;
  static constexpr int kBarOff = kMiscOff + kMiscFloats * 4;
  static constexpr int kFixedBars = 22 + 2 * kScStages;
  static constexpr int kTailBytes = kFixedBars * 8 + 16 * 4;  // then the ring's barriers
  static constexpr int kRingBudget = 232448 - 1024 - (kBarOff + kTailBytes);
  static constexpr int kSlotCost = kTileBytes + 16;
  static constexpr int kSlots = kRingBudget / kSlotCost > 24 ? 24 : kRingBudget / kSlotCost;
  static constexpr int kRingOff = (kBarOff + kTailBytes + kSlots * 16 + 1023) / 1024 * 1024;
  static constexpr int kSmemBytes = kRingOff + kSlots * kTileBytes;
  static constexpr int kTmemUse = 2 * (kQCols + kOCols);
  static constexpr int kTmemCols = kTmemUse <= 64 ? 64 : kTmemUse <= 128 ? 128 : kTmemUse <= 256 ? 256 : 512;
  static_assert(kPBytes % 1024 == 0 && kQBytes % 1024 == 0, "swizzled buffers start on 1024 bytes");
  static_assert(kSmemBytes <= 232448 && kSlots >= 4, "shared memory budget");
  static_assert(kTmemUse <= 512, "tensor memory budget");
};

constexpr int kDecodeThreads = 384;
// Warps 0-3 softmax, 4-7 epilogue (each on the tensor memory lanes of its number mod 4).
enum : int { kDecProducer = 8, kDecIssuer = 9, kDecQ = 10, kDecScales = 11 };

enum DecodeTag : int {
  kTagDFull = 1, kTagDEmpty = 2, kTagDQ = 3, kTagDQEmpty = 4, kTagDS = 5, kTagDSEmpty = 6, kTagDP = 7, kTagDPEmpty = 8,
  kTagDO = 9, kTagDOEmpty = 10, kTagDStat = 11, kTagDSc = 12, kTagDScEmpty = 13
};

// 4-D tiled load (x = feature, y = row of the page, z = head, w = page).
__device__ __forceinline__ void tma_load_4d(const CUtensorMap *m, uint64_t *bar, void *dst, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// make_sdesc with a 64-byte swizzle (mode 4): rows of 64 bytes, groups of 8 rows 512 bytes apart.
__device__ __forceinline__ uint64_t make_sdesc64(uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  return (make_sdesc(saddr, lbo_bytes, sbo_bytes) & ~(7ull << 61)) | (4ull << 61);
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t *r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Barrier `id` over `n` threads that also returns whether any of them passed true.
__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t n, bool mine) {
  __syncwarp();
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\tbar.red.or.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"(mine ? 1u : 0u)
      : "memory");
  return r != 0;
}

// 4-byte asynchronous copy global -> shared; zeros if !valid.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float *src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
// Arrive on `bar` once this thread's earlier cp.async copies have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Reduce v[0..N) over the warp's lanes, leaving column lane / (32 / N) in v[0]: halves of
// the columns change hands first, so N columns take N + log2(32 / N) - 1 shuffles.
template <int N, class F>
__device__ __forceinline__ void reduce_columns(float (&v)[N], F f) {
  const int lane = threadIdx.x & 31;
  int bit = 16;
#pragma unroll
  for (int w = N / 2; w >= 1; w /= 2) {
    const bool up = (lane & bit) != 0;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float keep = up ? v[i + w] : v[i], give = up ? v[i] : v[i + w];
      v[i] = f(keep, __shfl_xor_sync(0xffffffffu, give, bit));
    }
    bit >>= 1;
  }
  for (; bit >= 1; bit >>= 1) v[0] = f(v[0], __shfl_xor_sync(0xffffffffu, v[0], bit));
}

// A walk over this CTA's tiles, run by a whole warp.  Lane i holds the length of sequence
// base + i, so that moving on to another sequence costs a load once in 32.
struct DecodeWalk {
  int b, x, off, rem;        // sequence, item of it, tile of the item, tiles left to this CTA
  int len, first, tile0, n;  // b's length, first visible position, its tile, and the item's tiles
  int base, lane_len;

  __device__ __forceinline__ void window32(const DecodeParams &p, int at) {
    base = at;
    const int i = at + static_cast<int>(lane_id());
    lane_len = i < p.c.B ? cache_len(p.c, i, kKernelDecode) : 0;
  }
  __device__ __forceinline__ void sequence(const DecodeParams &p) {
    len = __shfl_sync(0xffffffffu, lane_len, b - base);
    first = p.window > 0 ? max(0, len - p.window) : 0;
    tile0 = first >> 7;
    n = ((len + 127) >> 7) - tile0;
  }
  __device__ __forceinline__ void start(const DecodeParams &p, int b0, int x0, int off0, int tiles) {
    b = b0;
    x = x0;
    off = off0;
    rem = tiles;
    base = lane_len = len = first = tile0 = n = 0;
    if (rem > 0) {
      window32(p, b);
      sequence(p);
    }
  }
  // Tiles of the current segment: the item's tiles from `off` on, as far as the share goes.
  __device__ __forceinline__ int run() const { return min(n - off, rem); }
  // Past `k` tiles of the current item, to the next item if they were its last.
  __device__ __forceinline__ void advance(const DecodeParams &p, int k) {
    rem -= k;
    off += k;
    if (rem <= 0 || off < n) return;
    off = 0;
    if (++x < p.c.H * p.nblk) return;
    x = 0;
    for (;;) {
      const uint32_t later = __ballot_sync(0xffffffffu, lane_len > 0 && base + static_cast<int>(lane_id()) > b);
      if (later) {
        b = base + __ffs(later) - 1;
        break;
      }
      if (base + 32 >= p.c.B) {  // not reached while tiles are left
        rem = 0;
        return;
      }
      b = base + 31;
      window32(p, base + 32);
    }
    sequence(p);
  }
};

template <int D, bool E4M3, int GB>
__global__ void __launch_bounds__(kDecodeThreads, 1)
    fa_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ DecodeParams p) {
  using C = DecodeCfg<D, E4M3, GB>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
  uint64_t *bar_q = bars + 0;         // [2] Q of a segment is in shared memory
  uint64_t *bar_q_empty = bars + 2;   // [2] ... and read for the last time
  uint64_t *bar_s = bars + 4;         // [2] S^T of a tile is in tensor memory
  uint64_t *bar_s_empty = bars + 6;   // [2]
  uint64_t *bar_p = bars + 8;         // [2] P of a tile is in shared memory (V's masked rows are zero, O is rescaled)
  uint64_t *bar_p_empty = bars + 10;  // [2] the tile's V^T P has completed
  uint64_t *bar_o = bars + 12;        // [2] a segment's last V^T P has completed
  uint64_t *bar_o_empty = bars + 14;  // [2] the epilogue has read O and the segment's sums
  uint64_t *bar_stat = bars + 16;     // [2] the segment's m and l are in shared memory
  uint64_t *bar_drain = bars + 18;    // abort path: the issuer's MMAs completed
  uint64_t *bar_sc = bars + 20;       // [kScStages] the keys' factors
  uint64_t *bar_sc_empty = bar_sc + C::kScStages;
  int *words = reinterpret_cast<int *>(bars + C::kFixedBars);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(words);
  volatile int *abort_flag = words + 1;
  int *share = words + 2;  // b, x, off, tiles of this CTA's share, then T, nc and "do nothing"
  uint64_t *bar_full = reinterpret_cast<uint64_t *>(words + 16);  // [kSlots]
  uint64_t *bar_empty = bar_full + C::kSlots;                     // [kSlots]
  float *xmax = reinterpret_cast<float *>(smem + C::kMiscOff);    // [2][GB][4]
  float *lpart = xmax + 2 * GB * 4;                               // [2][4][GB]
  float *mstat = lpart + 2 * 4 * GB;                              // [2][GB]
  float *qscale = mstat + 2 * GB;                                 // [2][GB]
  float *vmaxw = qscale + 2 * GB;                                 // [2][4]
  float *vstat = vmaxw + 8;                                       // [2]
  uint8_t *ring = smem + C::kRingOff;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const WaitCtx ctx{p.c.status, abort_flag, kKernelDecode, p.c.seq};
  // The join kernel may be put on the SMs' leftovers now; it waits for this grid's end.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < 7; ++i) share[i] = 0;
    if ((smem_u32(smem) & 1023u) != 0) {
      record_failure(ctx, kStatusInternal, 0);
      share[6] = 1;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar_q[i], 32);
      mbar_init(&bar_q_empty[i], E4M3 ? 5 : 1);  // the issuer's commit; e4m3: and the softmax warps, for q's scale
      mbar_init(&bar_s[i], 1);
      mbar_init(&bar_s_empty[i], 4);
      mbar_init(&bar_p[i], 4);
      mbar_init(&bar_p_empty[i], 1);
      mbar_init(&bar_o[i], 1);
      mbar_init(&bar_o_empty[i], 4);
      mbar_init(&bar_stat[i], 4);
    }
    mbar_init(bar_drain, 1);
    for (int i = 0; i < C::kScStages; ++i) {
      mbar_init(&bar_sc[i], 32);
      mbar_init(&bar_sc_empty[i], 4);
    }
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&bar_full[i], 1);
      mbar_init(&bar_empty[i], 1);
    }
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == kDecIssuer) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }

  // ---------------------------------------------------------------- the share
  // Thread i counts the tiles of sequences [i * per, (i + 1) * per); a scan over the
  // threads gives every share's first sequence.
  {
    const int items = p.c.H * p.nblk;
    const int per = (p.c.B + kDecodeThreads - 1) / kDecodeThreads;
    const int b_lo = min(p.c.B, static_cast<int>(threadIdx.x) * per), b_hi = min(p.c.B, b_lo + per);
    auto tiles_of = [&](int b) {
      const int len = cache_len(p.c, b, kKernelDecode);
      const int first = p.window > 0 ? max(0, len - p.window) : 0;
      return ((len + 127) >> 7) - (first >> 7);
    };
    int mine = 0;
    for (int b = b_lo; b < b_hi; ++b) mine += tiles_of(b) * items;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    int *sums = reinterpret_cast<int *>(xmax);  // [12], used before the softmax warps start
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < kDecodeThreads / 32; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    const int nc = min(static_cast<int>(gridDim.x), total);
    if (static_cast<int>(blockIdx.x) < nc) {
      const int t0 = static_cast<int>(static_cast<long long>(total) * blockIdx.x / nc);
      const int t1 = static_cast<int>(static_cast<long long>(total) * (blockIdx.x + 1) / nc);
      const int excl = before + incl - mine;
      if (mine > 0 && t0 >= excl && t0 < excl + mine) {
        int b = b_lo, at = t0 - excl;
        int n = tiles_of(b);
        while (at >= n * items) {
          at -= n * items;
          n = tiles_of(++b);
        }
        share[0] = b;
        share[1] = at / n;
        share[2] = at % n;
        share[3] = t1 - t0;
        share[4] = total;
        share[5] = nc;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t kOCol0 = 2 * C::kQCols;

  DecodeWalk wk;
  wk.start(p, share[0], share[1], share[2], share[6] ? 0 : share[3]);

  if (warp == kDecProducer) {
    // ------------------------------------------------------------- producer
    // Lane i loads page i of a tile (pages of 128 rows or more: lane 0 alone).  The page
    // ids of the next tile are read while this tile's slots are waited for.
    const int rows = min(p.c.page_size, 128);
    const int pages = 128 / rows;
    auto page_of = [&](bool &need) {
      const int pos = (wk.tile0 + wk.off) * 128 + lane * rows;
      need = wk.rem > 0 && lane < pages && pos < wk.len && pos + rows > wk.first;
      int row = 0, page = 0;
      if (need) {
        page = cache_page(p.c, wk.b, pos, row, kKernelDecode);
        if (page < 0) page = p.c.num_pages;  // out of the tensor map's range: TMA fills with zeros
      }
      return make_int2(page, row);
    };
    bool need, ok = true;
    int2 at = page_of(need);
    int g = 0;  // slots filled so far
    while (wk.rem > 0 && ok) {
      const int h = wk.x / p.nblk;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, need)) * rows * C::kRowBytes;
      const bool now = need;
      const int2 here = at;
      wk.advance(p, 1);
      at = page_of(need);
      for (int kv = 0; kv < 2; ++kv, ++g) {
        const int s = g % C::kSlots, r = g / C::kSlots;
        if (r > 0 && !(ok = __all_sync(0xffffffffu, mbar_wait(ctx, &bar_empty[s], (r - 1) & 1, kTagDEmpty)))) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar_full[s], bytes);
        __syncwarp();
        if (now)
          for (int i = 0; i < C::kPanels; ++i)
            tma_load_4d(kv == 0 ? &tmK : &tmV, &bar_full[s],
                        ring + s * C::kTileBytes + i * C::kPanelBytes + lane * rows * C::kPanelRow,
                        i * (C::kPanelRow / C::kElem), here.y, h, here.x);
        __syncwarp();
      }
    }
    // The last loads have landed before the CTA can exit.
    for (int s = 0; s < C::kSlots && s < g; ++s) mbar_drain(&bar_full[s], ((g - 1 - s) / C::kSlots) & 1);
    __syncwarp();
  } else if (warp == kDecIssuer) {
    // --------------------------------------------------------------- issuer
    // S^T of tile i + 1 goes in ahead of V^T P of tile i, across segments too.
    constexpr uint32_t idesc_s = E4M3 ? make_idesc_e4m3(128, C::kQCols, 0, 0) : make_idesc_bf16(128, C::kQCols, 0, 0);
    constexpr uint32_t idesc_o = E4M3 ? make_idesc_e4m3(128, C::kOCols, 1, 0) : make_idesc_bf16(128, C::kOCols, 1, 0);
    constexpr bool kSw64 = C::kPanelRow == 64;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t ring0 = smem_u32(ring);
    // K (rows are keys) and Q (rows are heads) are K-major in the same panels.
    const uint64_t k_desc0 = kSw64 ? make_sdesc64(ring0, 16, 512) : make_sdesc(ring0, 16, 1024);
    const uint64_t q_desc0 = kSw64 ? make_sdesc64(smem_u32(smem + C::kQOff), 16, 512)
                                   : make_sdesc(smem_u32(smem + C::kQOff), 16, 1024);
    // V as the M x K operand V^T is MN-major.  M = 128 features are d = 128's, in panels
    // kPanelBytes apart; for d = 64 the second half repeats the first (offset 0), and its
    // half of O^T is not read.
    constexpr uint32_t v_lbo = D == 128 ? C::kPanelBytes : 0;
    const uint64_t v_desc0 = kSw64 ? make_sdesc64(ring0, v_lbo, 512) : make_sdesc(ring0, v_lbo, 1024);
    const uint64_t p_desc0 = make_sdesc(smem_u32(smem + C::kPOff), 16, 1024);
    bool ok = true;
    auto wait = [&](uint64_t *bar, int parity, int tag) {
      return __all_sync(0xffffffffu, mbar_wait(ctx, bar, static_cast<uint32_t>(parity), tag));
    };
    int n = 0;  // tiles whose S^T was issued
    // What V^T P of the previous tile needs to know.
    bool pend = false, pend_first = false, pend_last = false;
    int pend_seg = 0;
    auto issue_o = [&](int i) {  // tile i's V^T P
      const int buf = i & 1, g = 2 * i + 1, s = g % C::kSlots, ob = pend_seg & 1;
      if (pend_first && pend_seg >= 2 && !wait(&bar_o_empty[ob], ((pend_seg >> 1) - 1) & 1, kTagDOEmpty)) return false;
      if (!wait(&bar_full[s], (g / C::kSlots) & 1, kTagDFull)) return false;
      if (!wait(&bar_p[buf], (i >> 1) & 1, kTagDP)) return false;
      tc_fence_after();
      const uint64_t vd = sdesc_add(v_desc0, s * C::kTileBytes), pd = sdesc_add(p_desc0, buf * C::kPBytes);
      const uint32_t to = tm + kOCol0 + ob * C::kOCols;
      if constexpr (E4M3) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)  // 32 keys each
          mma_ss_f8_w(to, sdesc_add(vd, ks * 32 * C::kPanelRow), sdesc_add(pd, ks * 32), idesc_o,
                      (!pend_first || ks > 0) ? 1u : 0u);
      } else {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks)  // 16 keys each; P's panels hold 64
          mma_ss_w(to, sdesc_add(vd, ks * 16 * 128), sdesc_add(pd, (ks >> 2) * C::kOCols * 128 + (ks & 3) * 32),
                   idesc_o, (!pend_first || ks > 0) ? 1u : 0u);
      }
      mma_commit_w(&bar_empty[s]);
      mma_commit_w(&bar_p_empty[buf]);
      if (pend_last) mma_commit_w(&bar_o[ob]);
      return true;
    };
    for (int seg = 0; wk.rem > 0 && ok; ++seg) {
      const int run = wk.run(), qb = seg & 1;
      if (!(ok = wait(&bar_q[qb], (seg >> 1) & 1, kTagDQ))) break;
      for (int i = 0; i < run && ok; ++i, ++n) {
        const int buf = n & 1, g = 2 * n, s = g % C::kSlots;
        if (n >= 2 && !(ok = wait(&bar_s_empty[buf], ((n >> 1) - 1) & 1, kTagDSEmpty))) break;
        if (!(ok = wait(&bar_full[s], (g / C::kSlots) & 1, kTagDFull))) break;
        tc_fence_after();
        const uint64_t kd = sdesc_add(k_desc0, s * C::kTileBytes), qd = sdesc_add(q_desc0, qb * C::kQBytes);
        const uint32_t ts = tm + buf * C::kQCols;
        if constexpr (E4M3) {
#pragma unroll
          for (int ks = 0; ks < D / 32; ++ks)
            mma_ss_f8_w(ts, sdesc_add(kd, ks * 32), sdesc_add(qd, ks * 32), idesc_s, ks > 0);
        } else {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks)
            mma_ss_w(ts, sdesc_add(kd, (ks >> 2) * C::kPanelBytes + (ks & 3) * 32),
                     sdesc_add(qd, (ks >> 2) * C::kQCols * 128 + (ks & 3) * 32), idesc_s, ks > 0);
        }
        mma_commit_w(&bar_empty[s]);
        mma_commit_w(&bar_s[buf]);
        if (i + 1 == run) mma_commit_w(&bar_q_empty[qb]);
        if (pend && !(ok = issue_o(n - 1))) {
          ++n;
          break;
        }
        pend = true;
        pend_first = i == 0;
        pend_last = i + 1 == run;
        pend_seg = seg;
      }
      if (ok) wk.advance(p, run);
    }
    if (ok && pend) ok = issue_o(n - 1);
    if (!ok) {
      mma_commit_w(bar_drain);
      mbar_drain(bar_drain, 0);
    }
    __syncwarp();
  } else if (warp == kDecQ) {
    // ---------------------------------------------------------------- Q rows
    // Rows of the segment's query heads into swizzled shared memory; the next segment's
    // rows are read while this one's buffer is waited for.  Rows past the last head are 0.
    constexpr int kWords = D / 64;  // 32-bit words (2 elements) of a row per lane
    uint32_t w[GB][kWords];
    auto load = [&]() {
      const int h = wk.x / p.nblk, g0 = (wk.x % p.nblk) * GB;
      const uint32_t *src = reinterpret_cast<const uint32_t *>(
          p.q + (static_cast<long long>(wk.b) * p.Hq + h * p.G + g0) * D);
#pragma unroll
      for (int r = 0; r < GB; ++r)
#pragma unroll
        for (int i = 0; i < kWords; ++i)
          w[r][i] = (wk.rem > 0 && g0 + r < p.G) ? __ldg(src + r * (D / 2) + lane * kWords + i) : 0u;
    };
    bool ok = true;
    load();
    for (int seg = 0; wk.rem > 0 && ok; ++seg) {
      const int qb = seg & 1;
      if (seg >= 2 && !(ok = __all_sync(0xffffffffu, mbar_wait(ctx, &bar_q_empty[qb], ((seg >> 1) - 1) & 1, kTagDQEmpty))))
        break;
      uint8_t *dst = smem + C::kQOff + qb * C::kQBytes;
      if constexpr (!E4M3) {
#pragma unroll
        for (int r = 0; r < C::kQCols; ++r) {
          // Lane's elements start at byte lane * 4 * kWords of the row.
          const int byte = lane * 4 * kWords, panel = byte >> 7, in = byte & 127;
          uint8_t *at = dst + panel * (C::kQCols * 128) + r * 128 + ((((in >> 4) ^ (r & 7)) << 4) | (in & 15));
#pragma unroll
          for (int i = 0; i < kWords; ++i) reinterpret_cast<uint32_t *>(at)[i] = r < GB ? w[r < GB ? r : 0][i] : 0u;
        }
      } else {
        // Scale each row by the power of two that brings its largest element into
        // [128, 256), then split: hi = e4m3(x), lo = e4m3(16 (x - hi)).
        float x[2 * kWords];
#pragma unroll
        for (int r = 0; r < GB; ++r) {
          float m = 0.f;
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            x[2 * i] = bf16_lo(w[r][i]);
            x[2 * i + 1] = bf16_hi(w[r][i]);
            m = fmaxf(m, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          // Exponent field e of m: m in [2^(e-127), 2^(e-126)); x * 2^(134 - e).
          // An infinity (e = 255) makes every score of the head NaN.
          const int e0 = static_cast<int>(__float_as_uint(m) >> 23), e = min(max(e0, 16), 250);
          const float up = __uint_as_float(static_cast<uint32_t>(261 - e) << 23);
          if (lane == 0)
            qscale[qb * GB + r] =
                __uint_as_float(e0 == 255 ? 0x7fc00000u : static_cast<uint32_t>(e - 7) << 23) * p.scale_log2;
          uint32_t hi = 0, lo = 0;
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            const float a = x[2 * i] * up, c = x[2 * i + 1] * up;
            const uint32_t h2 = pack_e4m3x4(a, c, 0.f, 0.f);
            const float2 back = e4m3x2_to_float2(static_cast<uint16_t>(h2));
            const uint32_t l2 = pack_e4m3x4((a - back.x) * 16.f, (c - back.y) * 16.f, 0.f, 0.f);
            hi |= h2 << (16 * i);
            lo |= l2 << (16 * i);
          }
          const int byte = lane * 2 * kWords;
#pragma unroll
          for (int part = 0; part < 2; ++part) {
            const int row = part * GB + r;
            const uint32_t v = part == 0 ? hi : lo;
            const int chunk = C::kPanelRow == 64 ? ((byte >> 4) ^ ((row >> 1) & 3)) : ((byte >> 4) ^ (row & 7));
            uint8_t *at = dst + row * C::kPanelRow + ((chunk << 4) | (byte & 15));
            if constexpr (kWords == 2)
              *reinterpret_cast<uint32_t *>(at) = v;
            else
              *reinterpret_cast<uint16_t *>(at) = static_cast<uint16_t>(v);
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&bar_q[qb]);
      wk.advance(p, wk.run());
      load();
    }
    __syncwarp();
  } else if (warp == kDecScales) {
    // ------------------------------------------------- the keys' factors (e4m3)
    if constexpr (E4M3) {
      // Lane i copies the factors of keys i, i + 32, ... of a tile; the next tile's page
      // ids are read ahead.
      int page[4], row[4];
      auto pages_of = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int pos = (wk.tile0 + wk.off) * 128 + 32 * i + lane;
          page[i] = -1;
          if (wk.rem > 0 && pos >= wk.first && pos < wk.len) page[i] = cache_page(p.c, wk.b, pos, row[i], kKernelDecode);
        }
      };
      bool ok = true;
      pages_of();
      for (int n = 0; wk.rem > 0; ++n) {
        const int st = n % C::kScStages;
        if (n >= C::kScStages &&
            !(ok = __all_sync(0xffffffffu, mbar_wait(ctx, &bar_sc_empty[st], (n / C::kScStages - 1) & 1, kTagDScEmpty))))
          break;
        const int h = wk.x / p.nblk;
        const uint32_t dst = smem_u32(smem + C::kScOff) + st * 1024;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool live = page[i] >= 0;
            const long long off = live ? page[i] * p.c.scale_stride[kv][0] + h * p.c.scale_stride[kv][1] +
                                             row[i] * p.c.scale_stride[kv][2]
                                       : 0;
            cp_async4(dst + kv * 512 + (32 * i + lane) * 4, p.c.scale[kv] + off, live);
          }
        cp_async_arrive(&bar_sc[st]);
        wk.advance(p, 1);
        pages_of();
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
    }
  } else if (warp < 4) {
    // -------------------------------------------------------------- softmax
    // Thread = key (row of S^T, tensor memory lane 32 * warp + lane), GB scores each.
    // All waits are bounded and every thread reaches every bar_any, so a failed wait
    // (`bad`) ends the four warps together.
    const int key = warp * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    float mref[GB], l[GB];
    float vref = 1.f;  // e4m3: power of two that V's factors are taken relative to
    bool bad = false, stop = false;
    int n = 0, nred = 0;
    for (int seg = 0; wk.rem > 0 && !stop; ++seg) {
      const int run = wk.run(), qb = seg & 1;
      float qs[E4M3 ? GB : 1];
      if constexpr (E4M3) {
        bad |= !mbar_wait(ctx, &bar_q[qb], (seg >> 1) & 1, kTagDQ);
#pragma unroll
        for (int g = 0; g < GB; ++g) qs[g] = qscale[qb * GB + g];
      }
#pragma unroll
      for (int g = 0; g < GB; ++g) {
        mref[g] = -INFINITY;
        l[g] = 0.f;
      }
      for (int i = 0; i < run; ++i, ++n) {
        const int buf = n & 1;
        const int pos0 = (wk.tile0 + wk.off + i) * 128, pos = pos0 + key;
        const bool partial = pos0 < wk.first || pos0 + 128 > wk.len;
        const bool valid = pos >= wk.first && pos < wk.len;
        bad |= !mbar_wait(ctx, &bar_s[buf], (n >> 1) & 1, kTagDS);
        if (n >= 2) bad |= !mbar_wait(ctx, &bar_p_empty[buf], ((n >> 1) - 1) & 1, kTagDPEmpty);
        float fk = p.scale_log2, fv = 1.f;
        if constexpr (E4M3) {
          const int st = n % C::kScStages;
          bad |= !mbar_wait(ctx, &bar_sc[st], (n / C::kScStages) & 1, kTagDSc);
          const float *sc = reinterpret_cast<const float *>(smem + C::kScOff + st * 1024);
          fk = sc[key];
          fv = sc[128 + key];
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_sc_empty[st]);
        }
        if (partial) {
          // Masked rows of V: weight 0 times whatever the page holds has to be 0.
          const int gv = 2 * n + 1, sv = gv % C::kSlots;
          bad |= !mbar_wait(ctx, &bar_full[sv], (gv / C::kSlots) & 1, kTagDFull);
          if (!valid) {
            uint8_t *rowp = ring + sv * C::kTileBytes + key * C::kPanelRow;
#pragma unroll
            for (int ch = 0; ch < C::kRowBytes / 16; ++ch) {
              // Lanes start at different chunks, so that their stores fall into different banks.
              const int c = (ch + lane) % (C::kRowBytes / 16);
              *reinterpret_cast<uint4 *>(rowp + (c * 16 / C::kPanelRow) * C::kPanelBytes + (c * 16) % C::kPanelRow) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
          }
        }
        __syncwarp();
        tc_fence_after();
        float s[GB];
        {
          const uint32_t ts = tmem + lane_off + buf * C::kQCols;
          uint32_t raw[C::kQCols < GB ? GB : (E4M3 ? 2 * GB : GB)];
#pragma unroll
          for (int c = 0; c < (E4M3 ? 2 * GB : GB); c += 8) tmem_ld8(ts + c, raw + c);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_s_empty[buf]);
#pragma unroll
          for (int g = 0; g < GB; ++g) {
            float v = __uint_as_float(raw[g]);
            if constexpr (E4M3) v = fmaf(__uint_as_float(raw[GB + g]), 0.0625f, v) * qs[g];
            s[g] = valid ? v * fk : -INFINITY;
          }
        }
        // Does a score outgrow the reference?
        bool grow = i == 0;
        if (i > 0) {
#pragma unroll
          for (int g = 0; g < GB; ++g) grow |= s[g] > mref[g] + C::kGrow;
          if constexpr (E4M3) grow |= valid && fabsf(fv) > vref;
        }
        if (i == 0 || bar_any(1, 128, grow || bad)) {
          float *xm = xmax + (nred & 1) * GB * 4;
          float v[GB];
#pragma unroll
          for (int g = 0; g < GB; ++g) v[g] = s[g];
          reduce_columns<GB>(v, [](float a, float b) { return fmaxf(a, b); });
          if ((lane & (32 / GB - 1)) == 0) xm[(lane / (32 / GB)) * 4 + warp] = v[0];
          if constexpr (E4M3) {
            const uint32_t vm = __reduce_max_sync(0xffffffffu, valid ? __float_as_uint(fabsf(fv)) : 0u);
            if (lane == 0) vmaxw[(nred & 1) * 4 + warp] = __uint_as_float(vm);
          }
          if (bar_any(2, 128, bad)) {
            stop = true;
            break;
          }
          float alpha[GB], vscale = 1.f;
          if constexpr (E4M3) {
            const float4 v4 = *reinterpret_cast<const float4 *>(vmaxw + (nred & 1) * 4);
            const uint32_t top = __float_as_uint(fmaxf(fmaxf(v4.x, v4.y), fmaxf(v4.z, v4.w)));
            // The next power of two, within [2^-120, 2^126].
            const uint32_t up = (min(top, 0x7e800000u) + 0x7fffffu) & 0x7f800000u;
            float now = __uint_as_float(max(up, 7u << 23));
            if (i > 0) {
              now = fmaxf(now, vref);
              vscale = vref / now;
            }
            vref = now;
          }
#pragma unroll
          for (int g = 0; g < GB; ++g) {
            const float4 m4 = *reinterpret_cast<const float4 *>(xm + g * 4);
            const float m = fmaxf(fmaxf(mref[g], m4.x), fmaxf(fmaxf(m4.y, m4.z), m4.w));
            alpha[g] = (i == 0 || m == mref[g]) ? 1.f : ex2(mref[g] - m);
            mref[g] = m;
            l[g] *= alpha[g];
          }
          ++nred;
          if (i > 0) {
            // O holds tiles of this segment on the old reference: bring it to the new one.
            bad |= !mbar_wait(ctx, &bar_p_empty[(n - 1) & 1], ((n - 1) >> 1) & 1, kTagDPEmpty);
            tc_fence_after();
            const uint32_t to = tmem + lane_off + kOCol0 + (seg & 1) * C::kOCols;
#pragma unroll
            for (int part = 0; part < C::kOParts; ++part)
#pragma unroll
              for (int g = 0; g < GB; g += 8) {
                uint32_t o[8];
                tmem_ld8(to + part * GB + g, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * (alpha[g + e] * vscale));
                tmem_st8(to + part * GB + g, o);
              }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        // Weights into P: row (part, head), column key.
        const uint32_t pb = smem_u32(smem + C::kPOff) + buf * C::kPBytes;
        float pw[GB];
#pragma unroll
        for (int g = 0; g < GB; ++g) {
          pw[g] = ex2(s[g] - (mref[g] == -INFINITY ? 0.f : mref[g]));
          l[g] += pw[g];
        }
        if constexpr (!E4M3) {
          const uint32_t a0 = pb + (key >> 6) * (C::kOCols * 128) + ((key & 63) >> 3) * 16 + (key & 7) * 2;
#pragma unroll
          for (int g = 0; g < GB; g += 2) {
            const uint32_t hi = pack_bf16(pw[g], pw[g + 1]);
            const uint32_t lo = pack_bf16(pw[g] - bf16_lo(hi), pw[g + 1] - bf16_hi(hi));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r0 = g + e, r1 = GB + g + e;
              asm volatile("st.shared.u16 [%0], %1;" ::"r"((a0 ^ ((r0 & 7) << 4)) + r0 * 128),
                           "h"(static_cast<uint16_t>(e ? hi >> 16 : hi))
                           : "memory");
              asm volatile("st.shared.u16 [%0], %1;" ::"r"((a0 ^ ((r1 & 7) << 4)) + r1 * 128),
                           "h"(static_cast<uint16_t>(e ? lo >> 16 : lo))
                           : "memory");
            }
          }
        } else {
          const float fw = valid ? fv * (C::kWeight / vref) : 0.f;
          const uint32_t a0 = pb + (key >> 4) * 16 + (key & 15);
#pragma unroll
          for (int g = 0; g < GB; g += 4) {
            float r[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) r[e] = pw[g + e] * fw;
#pragma unroll
            for (int part = 0; part < 3; ++part) {
              const uint32_t code = pack_e4m3x4(r[0], r[1], r[2], r[3]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int row = part * GB + g + e;
                asm volatile("st.shared.u8 [%0], %1;" ::"r"((a0 ^ ((row & 7) << 4)) + row * 128), "r"(code >> (8 * e))
                             : "memory");
              }
              if (part < 2) {
                const float2 lo2 = e4m3x2_to_float2(static_cast<uint16_t>(code));
                const float2 hi2 = e4m3x2_to_float2(static_cast<uint16_t>(code >> 16));
                r[0] = (r[0] - lo2.x) * 16.f;
                r[1] = (r[1] - lo2.y) * 16.f;
                r[2] = (r[2] - hi2.x) * 16.f;
                r[3] = (r[3] - hi2.y) * 16.f;
              }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_p[buf]);
      }
      if (stop) break;
      // The segment's statistics for the epilogue.
      const int ob = seg & 1;
      if (seg >= 2) bad |= !mbar_wait(ctx, &bar_o_empty[ob], ((seg >> 1) - 1) & 1, kTagDOEmpty);
      reduce_columns<GB>(l, [](float a, float b) { return a + b; });
      if ((lane & (32 / GB - 1)) == 0) lpart[(ob * 4 + warp) * GB + lane / (32 / GB)] = l[0];
      if (threadIdx.x == 0) {
#pragma unroll
        for (int g = 0; g < GB; ++g) mstat[ob * GB + g] = mref[g];
        if constexpr (E4M3) vstat[ob] = vref;
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&bar_stat[ob]);
        if constexpr (E4M3) mbar_arrive(&bar_q_empty[qb]);
      }
      wk.advance(p, run);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------- epilogue
    // Thread = feature (tensor memory lane).  Idle sequences first: o = 0, lse = -inf.
    const int f = (warp - 4) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp - 4) * 32) << 16;
    for (int b = blockIdx.x; b < p.c.B; b += gridDim.x) {
      if (cache_len(p.c, b, kKernelDecode) > 0) continue;
      const long long row0 = static_cast<long long>(b) * p.Hq;
      for (int e = f; e < p.Hq * D / 8; e += 128) reinterpret_cast<uint4 *>(p.o + row0 * D)[e] = make_uint4(0u, 0u, 0u, 0u);
      if (p.lse)
        for (int e = f; e < p.Hq; e += 128) p.lse[row0 + e] = -INFINITY;
    }
    // The item that starts in this CTA's last segment and goes on in the next CTA, if any.
    int4 mt = make_int4(0, 0, 0, 0);
    const int total = share[4], nc = share[5];
    bool ok = true;
    for (int seg = 0; wk.rem > 0 && ok; ++seg) {
      const int ob = seg & 1, run = wk.run();
      const int h = wk.x / p.nblk, g0 = (wk.x % p.nblk) * GB, ng = min(GB, p.G - g0);
      const bool starts = wk.off == 0, ends = wk.off + run == wk.n;
      ok = __all_sync(0xffffffffu, mbar_wait(ctx, &bar_stat[ob], (seg >> 1) & 1, kTagDStat) &&
                                       mbar_wait(ctx, &bar_o[ob], (seg >> 1) & 1, kTagDO));
      if (!ok) break;
      tc_fence_after();
      const uint32_t to = tmem + lane_off + kOCol0 + ob * C::kOCols;
      const float unit = E4M3 ? vstat[ob] * (1.f / C::kWeight) : 1.f;
      const long long row0 = static_cast<long long>(wk.b) * p.Hq + h * p.G + g0;
      const int slot = 2 * blockIdx.x + (starts ? 1 : 0);
#pragma unroll
      for (int gc = 0; gc < GB; gc += 8) {
        uint32_t o[C::kOParts][8];
#pragma unroll
        for (int part = 0; part < C::kOParts; ++part) tmem_ld8(to + part * GB + gc, o[part]);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int g = gc + e;
          float v = __uint_as_float(o[0][e]);
          if constexpr (E4M3)
            v = (v + (__uint_as_float(o[1][e]) + __uint_as_float(o[2][e]) * 0.0625f) * 0.0625f) * unit;
          else
            v += __uint_as_float(o[1][e]);
          if (g >= ng) continue;
          const float *lp = lpart + ob * 4 * GB + g;
          const float lt = (lp[0] + lp[GB]) + (lp[2 * GB] + lp[3 * GB]);
          if (starts && ends) {
            if (f < D) p.o[(row0 + g) * D + f] = static_cast<uint16_t>(pack_bf16(v / lt, 0.f));
            if (f == 0 && p.lse) p.lse[row0 + g] = (mstat[ob * GB + g] + log2f(lt)) * 0.69314718055994531f;
          } else {
            if (f < D) p.part_o[(static_cast<long long>(slot) * GB + g) * D + f] = v;
            if (f == 0) p.part_ml[slot * GB + g] = make_float2(mstat[ob * GB + g], lt);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_o_empty[ob]);
      if (starts && !ends) {
        // Tile x lies in CTA ceil((x + 1) nc / T) - 1.
        const int t1 = static_cast<int>(static_cast<long long>(total) * (blockIdx.x + 1) / nc);
        const long long last = static_cast<long long>(t1) + (wk.n - run) - 1;
        const int c1 = static_cast<int>(((last + 1) * nc + total - 1) / total) - 1;
        mt = make_int4(wk.b, wk.x, c1 - static_cast<int>(blockIdx.x) + 1, 0);
      }
      wk.advance(p, run);
    }
    if (threadIdx.x == 128) p.meta[blockIdx.x] = mt;
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kDecIssuer) tmem_dealloc(tmem, C::kTmemCols);
}

// Joins the parts of one item for query head blockIdx.y of its block: CTA c's item starts
// in c (its second slot) and goes on in the first slots of CTAs c + 1 ...  The parts' sums
// are added in order, in kThreads / D interleaved groups that are then added in order too.
constexpr int kJoinThreads = 256;

template <int D, int GB>
__global__ void __launch_bounds__(kJoinThreads) fa_decode_join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kGroups = kJoinThreads / D;
  __shared__ float wgt[kDecodeMaxCtas], red[kJoinThreads / 32], part[kGroups][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 mt = p.meta[blockIdx.x];
  const int g = blockIdx.y;
  const int h = mt.y / p.nblk, g0 = (mt.y % p.nblk) * GB;
  if (mt.z == 0 || g0 + g >= p.G) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto slot = [&](int i) { return i == 0 ? 2 * static_cast<int>(blockIdx.x) + 1 : 2 * (static_cast<int>(blockIdx.x) + i); };
  // Weights 2^(m_i - M) of the parts, and the total of l.
  const float2 ml = tid < mt.z ? p.part_ml[slot(tid) * GB + g] : make_float2(-INFINITY, 0.f);
  float M = ml.x;
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  if (lane == 0) red[warp] = M;
  __syncthreads();
  M = red[0];
  for (int w = 1; w < kJoinThreads / 32; ++w) M = fmaxf(M, red[w]);
  __syncthreads();
  const float w0 = ml.x == -INFINITY ? 0.f : ex2(ml.x - M);
  if (tid < mt.z) wgt[tid] = w0;
  float L = w0 * ml.y;
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  if (lane == 0) red[warp] = L;
  __syncthreads();
  L = red[0];
  for (int w = 1; w < kJoinThreads / 32; ++w) L += red[w];
  const int f = tid % D, grp = tid / D;
  float acc = 0.f;
  for (int i = grp; i < mt.z; i += kGroups) acc += wgt[i] * p.part_o[(static_cast<long long>(slot(i)) * GB + g) * D + f];
  part[grp][f] = acc;
  __syncthreads();
  if (grp != 0) return;
  for (int k = 1; k < kGroups; ++k) acc += part[k][f];
  const long long row = static_cast<long long>(mt.x) * p.Hq + h * p.G + g0 + g;
  p.o[row * D + f] = static_cast<uint16_t>(pack_bf16(acc / L, 0.f));
  if (f == 0 && p.lse) p.lse[row] = (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace fa
