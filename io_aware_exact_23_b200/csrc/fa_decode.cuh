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
// Measured, in a replayed graph, of the 6465 GB/s that a copy reaches here: 1 x 131072 x 16
// heads of d = 128 in bf16 161 us (1074 MB, 6.65 TB/s: reads alone), 64 ragged sequences of up to
// 8192 x 8 heads in e4m3 94 us (551 MB, 5.9 TB/s; SMs differ by 6% in their time per tile).  Where
// a CTA has few tiles the time is latency: one sequence of 777 takes 8.4 us, 3 to the first load
// (lengths, share, page ids), 3 for a tile, 2.4 for the join.
//
// Work split.  A tile is 128 positions of one (sequence, cache head, block of at most GB
// query heads), and an item such a triple's tiles.  All tiles, in that order, are dealt out by their
// cost, an item's start and end included (DecodeCfg, DecodeSplit): CTA c of nc takes those that
// begin in its nc-th part of the total, so SMs finish together whatever the lengths, and a
// sequence is split over the cache's length exactly where a CTA's share ends.  A CTA walks its
// share as segments (runs of one item's tiles); an item held by one CTA is written out
// whole, the others leave (m, l, O) per segment in the workspace and fa_decode_join_kernel
// adds them up in a fixed order.
//
// Precision.  N is at least 16 in an M = 128 instruction, so for G <= 8 half of it is
// idle; the idle columns carry the low part of the operand that has to be rounded:
// * bf16: P = hi + lo, both bf16 (16 significant bits), as 2 GB columns of O^T;
// * e4m3: codes are multiplied as they are (kind::f8f6f4), the factor of K goes into the
//   score, that of V into the weight.  q (8 bits, a power of two taken out of each head) is
//   hi + lo / 32 in e4m3, exact to 2^-22 of the head's largest element.  A weight times V's factor is
//   four e5m2 parts (decode_parts): off by 2^-15 of itself at most, or by 2^-27 of the head's
//   largest such product, so that many keys far below one still count (three e4m3 parts of
//   fp16's 11 bits stopped at 2^-20 of it).
// The columns' sums meet again in fp32.
//
// Softmax warps.  Four warps own the 128 keys of a tile for 8 query heads, GB / 8 such
// groups per CTA.  P is the MN-major operand: a key's weights are adjacent bytes, so a
// thread stores its 8 heads with one vector store a part.  (With P K-major, one 2-byte
// or 1-byte store per head and part, and all GB heads in one thread, a tile took 3000 to
// 4000 cycles in e4m3; its share of the memory's rate allows 1430 at d = 128.)
#pragma once

#include <cstdint>

#include "fa_cache.cuh"
#include "ptx.cuh"

namespace fa {

constexpr int kDecodeMaxCtas = 320;  // workspace slots; the grid never exceeds it

struct DecodeParams {
  CacheView c;
  const uint16_t *q;  // [B, Hq, d]
  uint16_t *o;        // [B, Hq, d]
  float *lse;         // [B, Hq] or null
  int Hq, G;          // query heads, and query heads per cache head
  int nblk;           // blocks of GB query heads per cache head
  int window;         // 0: all positions
  int vec_scales;     // e4m3: four neighbouring tokens' factors are one aligned 16-byte piece
  float scale_log2;   // scale * log2(e)
  // [kDecodeMaxCtas] items in parts, {b, first query head, parts, first CTA}, parts 0: none.  Entry c
  // is for the item that begins in CTA c and goes on in the next, or (by_item, where there are
  // fewer items than CTAs) entry i for item i.
  int4 *meta;
  int by_item;
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
  static constexpr int kHeads = GB < 8 ? GB : 8;                   // query heads per softmax thread
  static constexpr int kGroups = GB / kHeads;                      // softmax warp groups
  static constexpr int kQUsed = E4M3 ? 2 * GB : GB;                // rows of Q that are written
  static constexpr int kQRows = kQUsed < 8 ? 8 : kQUsed;           // rows of Q in shared memory
  static constexpr int kQCols = kQRows < 16 ? 16 : kQRows;         // columns of S^T
  static constexpr int kOParts = E4M3 ? 4 : 2;
  static constexpr int kOCols = (kOParts * GB + 15) / 16 * 16;     // columns of O^T
  static constexpr int kPRow = GB <= 8 ? 32 : 4 * GB;              // bytes of a key's row of P
  static constexpr int kQBytes = kQRows * kRowBytes;
  static constexpr int kPBytes = 128 * kPRow;
  static constexpr int kScStages = 4;  // ring of the keys' factors (e4m3)
  // A score may exceed the running reference by kGrow (log2) before the reference moves.  e4m3: what
  // goes into the product is a code, weight * V's factor * a power of two per 8 heads.  A head's
  // reference is put so that its largest code is 2^kCodeLog2 (decode_references), and moves before a
  // code passes 2^(kCodeLog2 + kGrowV), or a weight 2^(kHeadLog2 + kGrow).
  // (Room of 2^5 instead of 2^7: 64 x 16384 with 32 heads, d = 64, 71.4 us, 68.7 so.)
  static constexpr float kGrow = 8.f;
  static constexpr int kCodeLog2 = 2, kGrowV = 7, kHeadLog2 = 80;

  static constexpr int kSoftmaxWarps = 4 * kGroups;
  static constexpr int kWarps = kSoftmaxWarps + 8;  // softmax, 4 epilogue, producer, issuer, Q, scales
  static constexpr int kThreads = 32 * kWarps;
  // Two CTAs per SM with up to 8 heads: one's tile hides the other's waits.
  static constexpr int kCtas = GB <= 8 ? 2 : 1;
  // The share of a CTA is dealt out by cost: kTileCost a tile, and kItemCost for what an item
  // costs besides (its Q, first maximum, sums and epilogue).  256 short e4m3 sequences x 16
  // heads, d = 64: 57.1 us without an item's cost, 55.2 with 2, 57.4 with 4, 59.7 with 8; long
  // sequences do not tell them apart.  Below kItemTiles tiles a CTA only the tiles count: one
  // tile more is what a CTA then takes longer than the others (one sequence of 777, 8 heads:
  // 9.9 us with an item's cost, which gives some of the 56 CTAs two tiles and others none, 8.4
  // without; at 3 tiles a CTA 15.2 against 16.1 us speak for it).
  static constexpr int kTileCost = 4, kItemCost = 2, kItemTiles = 2;
  static constexpr int kSmemMax = kCtas == 2 ? 115712 : 232448;

  static constexpr int kPOff = 0;
  static constexpr int kQOff = kPOff + 2 * kPBytes;
  static constexpr int kRingOff = (kQOff + 2 * kQBytes + 1023) / 1024 * 1024;
  // Behind the ring: factors, then floats xmax[2][GB][4], lpart[2][4][GB], mstat[2][GB], of e4m3
  // vmax[2][GB][4], refs[4][4][GB], qscale[2][GB], vstat[2][GB] and vspan[2][kGroups][4] pairs, then barriers and words.
  static constexpr int kScBytes = E4M3 ? kScStages * 1024 : 0;
  static constexpr int kMiscFloats = 2 * GB * 4 + 2 * 4 * GB + 2 * GB + (E4M3 ? 28 * GB + 16 * kGroups : 0);
  static constexpr int kFixedBars = 20 + 2 * kScStages;
  static constexpr int kTailBytes = kScBytes + kMiscFloats * 4 + kFixedBars * 8 + 16 * 4;
  static constexpr int kFit = (kSmemMax - kRingOff - kTailBytes) / (kTileBytes + 16);
  static constexpr int kSlots = kFit > 24 ? 24 : kFit;
  // How the softmax warps learn, before they rescale O, that the previous tile's V^T P is
  // complete: its V's slot is free again.  With three slots the slot could be two rounds
  // further by then, and a barrier of its own (bar_pv) says it.
  static constexpr bool kPvBar = kSlots < 5;
  static constexpr int kScOff = kRingOff + kSlots * kTileBytes;
  static constexpr int kMiscOff = kScOff + kScBytes;
  static constexpr int kBarOff = kMiscOff + kMiscFloats * 4;
  static constexpr int kSmemBytes = kScOff + kTailBytes + kSlots * 16;
  static constexpr int kTmemUse = 2 * (kQCols + kOCols);
  static constexpr int kTmemCols = kTmemUse <= 64 ? 64 : kTmemUse <= 128 ? 128 : kTmemUse <= 256 ? 256 : 512;
  static_assert(kPBytes % 1024 == 0 && kQOff % 1024 == 0 && kBarOff % 16 == 0, "alignment");
  static_assert(kSmemBytes <= kSmemMax && kSlots >= 3, "shared memory budget");
  static_assert(kTmemCols * kCtas <= 512, "tensor memory budget");
  // Warp roles behind the softmax warps; the epilogue's sit on the tensor memory lanes of
  // their number mod 4.
  static constexpr int kEpilogue = kSoftmaxWarps, kProducer = kEpilogue + 4, kIssuer = kProducer + 1,
                       kQWarp = kProducer + 2, kScales = kProducer + 3;
};

enum DecodeTag : int {
  kTagDFull = 1, kTagDEmpty = 2, kTagDQ = 3, kTagDQEmpty = 4, kTagDS = 5, kTagDP = 6, kTagDPv = 7,
  kTagDO = 8, kTagDOEmpty = 9, kTagDStat = 10, kTagDSc = 11, kTagDScEmpty = 12
};

// 4-D tiled load (x = feature, y = row of the page, z = head, w = page).
__device__ __forceinline__ void tma_load_4d(const CUtensorMap *m, uint64_t *bar, void *dst, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// make_sdesc for rows of 32, 64 or 128 bytes, swizzled by their own width (modes 6, 4, 2).
__device__ __forceinline__ uint64_t make_sdesc_row(int row_bytes, uint32_t saddr, uint32_t lbo_bytes, uint32_t sbo_bytes) {
  const uint64_t mode = row_bytes == 128 ? 2 : row_bytes == 64 ? 4 : 6;
  return (make_sdesc(saddr, lbo_bytes, sbo_bytes) & ~(7ull << 61)) | (mode << 61);
}

// Where byte `byte` of row `row` sits in such a tile: 16-byte chunks are exchanged by the
// address bits above the row's 128-byte line.
template <int ROW>
__device__ __forceinline__ uint32_t swizzled(int row, int byte) {
  const int f = ROW == 128 ? (row & 7) : ROW == 64 ? ((row >> 1) & 3) : ((row >> 2) & 1);
  return static_cast<uint32_t>(row * ROW + (byte ^ (f << 4)));
}

// mbar_wait for a CTA of many waiting warps: the test may suspend the warp for some
// microseconds (without the hint, the roles' polling took most of the issue slots), and
// what follows a failed one is out of line (instruction fetch is scarce too).
__device__ __forceinline__ bool decode_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}
// Whether the phase is complete, without suspending.
__device__ __forceinline__ bool decode_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __noinline__ bool decode_wait_slow(const WaitCtx &c, uint32_t bar, uint32_t parity, int tag) {
  const uint64_t t0 = globaltimer();
  while (!decode_try_wait(bar, parity)) {
    if (*c.abort || reinterpret_cast<volatile int *>(c.status)[4] == c.seq) {
      *c.abort = 1;
      return false;
    }
    if (globaltimer() - t0 > kWaitLimitNs) {
      record_failure(c, kStatusTimeout, tag);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool decode_wait(const WaitCtx &c, uint64_t *bar, uint32_t parity, int tag) {
  const uint32_t b = smem_u32(bar);
  return decode_try_wait(b, parity) || decode_wait_slow(c, b, parity, tag);
}

// N = 2, 4 or 8 columns of this thread's tensor memory lane.
template <int N>
__device__ __forceinline__ void tmem_ld_n(uint32_t taddr, uint32_t *r) {
  if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  else if constexpr (N == 4)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr));
  else
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
}

template <int N>
__device__ __forceinline__ void tmem_st_n(uint32_t taddr, const uint32_t *r) {
  if constexpr (N == 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  else if constexpr (N == 4)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
  else
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};" ::"r"(taddr), "r"(r[0]), "r"(r[1]) : "memory");
}

__device__ __forceinline__ void st_shared_v2(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}

// Two fp32 -> fp16x2, fp16x2 -> e4m3x2 (both to nearest even) and e4m3x2 -> fp16x2 (exact).
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint16_t f16x2_to_e4m3x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// Two fp32 -> e5m2x2 (to nearest even), the low one first; fp16x2 -> two fp32; a - b on fp16 pairs.
__device__ __forceinline__ uint32_t pack_e5m2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint64_t f16x2_to_f32x2(uint32_t h) {
  float lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
  return f2pack(lo, hi);
}
__device__ __forceinline__ uint32_t f16x2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// A pair of codes c, |c| < 2^10, as four e5m2 parts each: c = p0 + (p1 + p2) / 2^8 + p3 / 2^17.
// e5m2 is fp16's upper byte, so h = fp16(c) is taken apart by integer rounding to that byte (to
// nearest, halves up) and exact fp16 differences.  In h's units in the last place (2^-24 below its
// normal numbers) |h| < 2^11: |h - p0| <= 2^7, 2^8 of it is at most 2^14; p1 leaves at most 2^3, three
// bits, which p2 holds as it is (in units of no less than 2^-16).  p3 is c - h, which fp32 has exactly, to
// nearest and three bits: off by 2^-15 of c, or by 2^-29 where that is more.  A NaN gets through in
// p2 and p3.
// The upper bytes of p0, p1 and p2's halves are their codes; p3 is two codes.
constexpr float kPartUnit1 = 1.f / (1 << 8), kPartUnit3 = 1.f / (1 << 17);
__device__ __forceinline__ void decode_parts(uint64_t c, uint32_t (&p)[4]) {
  float a, b;
  f2unpack(c, a, b);
  const uint32_t h = pack_f16(a, b);
  p[0] = (h + 0x00800080u) & 0xff00ff00u;
  const uint32_t r = f16x2_mul(f16x2_sub(h, p[0]), 0x5c005c00u);  // 2^8
  p[1] = (r + 0x00800080u) & 0xff00ff00u;
  p[2] = f16x2_sub(r, p[1]);
  f2unpack(ffma2(f16x2_to_f32x2(h), f2pack(-131072.f, -131072.f), mul2(c, f2pack(131072.f, 131072.f))), a, b);
  p[3] = pack_e5m2(a, b);
}

// Where a tile's factors are within this of each other, the largest one and a head's largest weight stand for
// its largest product (else that takes a second exchange between the warps).
constexpr float kFactorSpan = 8.f;

// The references of one query head of an e4m3 cache: m, its largest score (log2) so far; e, a power
// of two that its products of weight (relative to m) and V's factor have not passed; and r = m -
// delta, the reference of the scores, with a whole delta in [0, kHeadLog2].
// A code is 2^(score - r) * factor * code, where `code` is one power of two for the 8 heads of a
// softmax warp: 2^kCodeLog2 / the largest of their e, so that theirs is the largest code.  A head whose
// products are smaller has its scores' reference lowered by as much (its weights raised), and so its own
// largest code where the others' is; only below 2^-kHeadLog2 of them does it lose resolution.
// Weights, codes and sums stay in range: a weight is at most 2^kHeadLog2 on r, and r is rounded up (m with
// it) where it cannot hold the difference.  A segment's sums leave it on m again: l * unit, exact.
struct DecodeRefs {
  float m, r, e, unit;  // unit: 2^-delta
};
// Products as powers of two, within [2^-116, 2^126].
__device__ __forceinline__ uint32_t decode_power(float x) {
  return max((min(__float_as_uint(x), 0x7e800000u) + 0x7fffffu) & 0x7f800000u, 11u << 23);
}
template <class C>
__device__ __forceinline__ DecodeRefs decode_references(float m, float product, uint32_t &code) {
  const uint32_t mine = decode_power(product), most = __reduce_max_sync(0xffffffffu, mine);
  code = ((254u + C::kCodeLog2) << 23) - most;  // 2^kCodeLog2 / most
  const uint32_t delta = min((most - mine) >> 23, static_cast<uint32_t>(C::kHeadLog2));
  const float less = static_cast<float>(delta), r = __fadd_ru(m, -less);
  return {r + less, r, __uint_as_float(most - (delta << 23)), __uint_as_float((127u - delta) << 23)};
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
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

// 4- and 16-byte asynchronous copies global -> shared.
__device__ __forceinline__ void cp_async4(uint32_t dst, const float *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const float *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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

// The columns' largest values, in the lanes that reduce_columns leaves them in (NaN aside).  Few columns
// go through the integer reduction, on bits ordered as the numbers are (256 short e4m3 sequences of one
// head, d = 64, 62.5 us with the shuffles, 57.5 so); of 8, the shuffles are as fast.
template <int N>
__device__ __forceinline__ float max_columns(float (&v)[N]) {
  if constexpr (N > 4) {
    reduce_columns<N>(v, [](float a, float b) { return fmaxf(a, b); });
    return v[0];
  } else {
    const int mine = (threadIdx.x & 31) / (32 / N);
    int best = 0;
#pragma unroll
    for (int g = 0; g < N; ++g) {
      const int b = __float_as_int(fmaxf(v[g], -INFINITY));
      const int r = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7fffffff));
      best = mine == g ? r : best;
    }
    return __int_as_float(best ^ ((best >> 31) & 0x7fffffff));
  }
}

// `total` units of cost dealt out to `nc` CTAs, the first of them one more where it does not
// divide.  A unit x of an item that begins at x0 stands for its tile (x - x0 - item's cost) /
// kTileCost (the first one below), so a CTA's tiles are those between the tiles that its
// first unit and the next CTA's stand for.
struct DecodeSplit {
  int q, r;
  __device__ __forceinline__ DecodeSplit(int total, int nc) : q(total / nc), r(total % nc) {}
  __device__ __forceinline__ int begin(int c) const { return q * c + min(c, r); }
  __device__ __forceinline__ int owner(int x) const {
    const int wide = r * (q + 1);
    return x < wide ? x / (q + 1) : r + (x - wide) / q;
  }
};

// The next sequence after b with a tile (-1: none), from the 32 lengths held from `base` on
// and then further ones.  Out of line: it is rare, and instruction fetch is scarce.
struct DecodeNext {
  int b, base, lane_len;
};
__device__ __noinline__ DecodeNext decode_next(const int *seq_lens, int B, int b, int base, int lane_len) {
  for (;;) {
    const uint32_t later = __ballot_sync(0xffffffffu, lane_len > 0 && base + static_cast<int>(lane_id()) > b);
    if (later) return {base + __ffs(later) - 1, base, lane_len};
    base += 32;
    if (base >= B) return {-1, base, 0};
    const int i = base + static_cast<int>(lane_id());
    lane_len = i < B ? __ldg(seq_lens + i) : 0;
  }
}

// A walk over this CTA's tiles, run by a whole warp.  Lane i holds the length of sequence
// base + i as it is in memory, so that moving on to another sequence costs a load once in 32
// (and the first one none: the share brings its length).
struct DecodeWalk {
  int b, h, blk, off, rem;   // sequence, cache head, block of query heads, tile of the item, tiles left to this CTA
  int len, first, tile0, n;  // b's length, first visible position, its tile, and the item's tiles
  int base, lane_len;

  __device__ __forceinline__ static int first_of(const DecodeParams &p, int len) {
    return p.window > 0 ? max(0, len - p.window) : 0;
  }
  __device__ __forceinline__ void sequence(const DecodeParams &p, int raw) {
    len = min(raw, p.c.cap);
    first = first_of(p, len);
    tile0 = first >> 7;
    n = ((len + 127) >> 7) - tile0;
  }
  __device__ __forceinline__ void start(const DecodeParams &p, const int *share) {
    base = b = share[0];
    h = share[1];
    off = share[2];
    rem = share[7] ? 0 : share[11] - share[10];
    blk = share[6];
    const int i = b + static_cast<int>(lane_id());
    lane_len = rem > 0 && i < p.c.B ? __ldg(p.c.seq_lens + i) : 0;
    sequence(p, share[8]);
  }
  // Tiles of the current segment: the item's tiles from `off` on, as far as the share goes.
  __device__ __forceinline__ int run() const { return min(n - off, rem); }
  // Past `k` tiles of the current item, to the next item if they were its last.
  __device__ __forceinline__ void advance(const DecodeParams &p, int k) {
    rem -= k;
    off += k;
    if (rem <= 0 || off < n) return;
    off = 0;
    if (++blk < p.nblk) return;
    blk = 0;
    if (++h < p.c.H) return;
    h = 0;
    const DecodeNext nx = decode_next(p.c.seq_lens, p.c.B, b, base, lane_len);
    if (nx.b < 0) {  // not reached while tiles are left
      rem = 0;
      return;
    }
    b = nx.b;
    base = nx.base;
    lane_len = nx.lane_len;
    sequence(p, __shfl_sync(0xffffffffu, lane_len, b - base));
  }
};

// The page ids of the walk's position, 32 at a time (lane i: page 32 * blk + i of sequence b),
// with the next 32 that will be asked for already on their way.  An id is -1 where the
// sequence needs no page and num_pages where the table is out of range.
struct DecodePages {
  int b = -1, blk = -1, ids = -1;
  int nb = -1, nblk = -1, nids = -1;
  bool moved = false;

  __device__ __forceinline__ static int load(const CacheView &c, int b, int blk, int len, int first) {
    const int i = 32 * blk + static_cast<int>(lane_id());
    return i >= cache_page_index(c, first) && i <= cache_page_index(c, len - 1) ? __ldg(c.block_table + b * c.bt_stride + i) : -1;
  }
  // To the pages of the walk's tile, which begins at position pos0; returns its first page.
  __device__ __forceinline__ int seek(const DecodeParams &p, const DecodeWalk &wk, int pos0) {
    const CacheView &c = p.c;
    const int pi = cache_page_index(c, pos0), at = pi >> 5;
    if (wk.b == b && at == blk) return pi;
    int id = wk.b == nb && at == nblk ? nids : load(c, wk.b, at, wk.len, wk.first);
    b = wk.b;
    blk = at;
    if (id >= c.num_pages || id < -1 || (id == -1 && load_needed(c, wk, at))) {
      record_cache_error(c.status, kKernelDecode, b, c.seq);
      id = c.num_pages;
    }
    ids = id;
    moved = true;
    return pi;
  }
  // After a move: ask for what comes next.
  __device__ __forceinline__ void ahead(const DecodeParams &p, const DecodeWalk &wk) {
    if (!moved) return;
    moved = false;
    const CacheView &c = p.c;
    const int at = blk;
    // The sequence's next block, its first one for the next head, or the
    // next sequence's first (as far as the walk holds its length).
    const int home = cache_page_index(c, wk.tile0 << 7) >> 5;
    nb = -1;
    if (at < (cache_page_index(c, wk.len - 1) >> 5) || (wk.h + 1 < c.H && home != at)) {
      nb = b;
      nblk = at < (cache_page_index(c, wk.len - 1) >> 5) ? at + 1 : home;
      nids = load(c, nb, nblk, wk.len, wk.first);
    } else {
      const uint32_t later =
          __ballot_sync(0xffffffffu, wk.lane_len > 0 && wk.base + static_cast<int>(lane_id()) > b);
      if (later) {
        nb = wk.base + __ffs(later) - 1;
        const int len = min(__shfl_sync(0xffffffffu, wk.lane_len, nb - wk.base), c.cap);
        const int first = DecodeWalk::first_of(p, len);
        nblk = cache_page_index(c, first & ~127) >> 5;
        nids = load(c, nb, nblk, len, first);
      }
    }
  }
  __device__ __forceinline__ static bool load_needed(const CacheView &c, const DecodeWalk &wk, int at) {
    const int i = 32 * at + static_cast<int>(lane_id());
    return i >= cache_page_index(c, wk.first) && i <= cache_page_index(c, wk.len - 1);
  }
};

// The tile's largest products of weight (relative to mx, of head lane / (32 / H)) and factor, over a
// group's four warps: head lane / (32 / H)'s.  Out of line: rare, and instruction fetch is scarce (256 short
// e4m3 sequences of one head, d = 64: 57.0 us, 58.1 in line).
template <int N>
struct DecodeScores {
  uint64_t v2[N];
};
template <int H>
__device__ __noinline__ float decode_products(DecodeScores<H / 2> s, float mx, float fv, float *vr, uint32_t bar) {
  constexpr int kSpan = 32 / H;
  const int lane = threadIdx.x & 31, w4 = (threadIdx.x >> 5) & 3;
  float t[H];
#pragma unroll
  for (int g = 0; g < H / 2; ++g) {
    float a, b;
    f2unpack(s.v2[g], a, b);
    t[2 * g] = fmaxf(ex2(a - __shfl_sync(0xffffffffu, mx, 2 * g * kSpan)), 0x1p-120f) * fabsf(fv);
    t[2 * g + 1] = fmaxf(ex2(b - __shfl_sync(0xffffffffu, mx, (2 * g + 1) * kSpan)), 0x1p-120f) * fabsf(fv);
  }
  const float most = max_columns<H>(t);
  if (lane % kSpan == 0) vr[lane / kSpan * 4 + w4] = most;
  bar_any(bar, 128, false);
  const float4 t4 = *reinterpret_cast<const float4 *>(vr + lane / kSpan * 4);
  return fmaxf(fmaxf(t4.x, t4.y), fmaxf(t4.z, t4.w));
}

// Note an item that begins in this CTA for the join kernel: its parts up to the CTA that holds
// its last unit of cost (0: it is whole).  Out of line: once an item at most.
__device__ __noinline__ void decode_note(const DecodeParams &p, int b, int h, int blk, int row, int last, int total, int nc) {
  const int c = static_cast<int>(blockIdx.x);
  const int parts = last > 0 ? DecodeSplit(total, nc).owner(last) - c + 1 : 0;
  p.meta[p.by_item ? (b * p.c.H + h) * p.nblk + blk : c] = make_int4(b, row, parts, c);
}

template <int D, bool E4M3, int GB>
__global__ void __launch_bounds__(DecodeCfg<D, E4M3, GB>::kThreads, DecodeCfg<D, E4M3, GB>::kCtas)
    fa_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ DecodeParams p) {
  using C = DecodeCfg<D, E4M3, GB>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
  uint64_t *bar_q = bars + 0;         // [2] Q of a segment is in shared memory
  uint64_t *bar_q_empty = bars + 2;   // [2] ... and read for the last time
  uint64_t *bar_s = bars + 4;         // [2] S^T of a tile is in tensor memory
  uint64_t *bar_p = bars + 8;         // [2] P of a tile is in shared memory (V's masked rows are zero, O is rescaled)
  uint64_t *bar_pv = bars + 10;       // [2] the tile's V^T P has completed (kPvBar)
  uint64_t *bar_o = bars + 12;        // [2] a segment's last V^T P has completed
  uint64_t *bar_o_empty = bars + 14;  // [2] the epilogue has read O and the segment's sums
  uint64_t *bar_stat = bars + 16;     // [2] the segment's m and l are in shared memory
  uint64_t *bar_drain = bars + 18;    // abort path: the issuer's MMAs completed
  uint64_t *bar_sc = bars + 20;       // [kScStages] the keys' factors
  uint64_t *bar_sc_empty = bar_sc + C::kScStages;
  int *words = reinterpret_cast<int *>(bars + C::kFixedBars);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(words);
  volatile int *abort_flag = words + 1;
  // The share: first sequence, head and tile, an item's cost; total cost, CTAs with a share, first block of
  // heads, "do nothing"; first sequence's length, cost before the first item, first and end tile.
  int *share = words + 2;
  uint64_t *bar_full = reinterpret_cast<uint64_t *>(words + 16);  // [kSlots]
  uint64_t *bar_empty = bar_full + C::kSlots;                     // [kSlots]
  float *xmax = reinterpret_cast<float *>(smem + C::kMiscOff);    // [2][GB][4]
  float *lpart = xmax + 2 * GB * 4;                               // [2][4][GB]
  float *mstat = lpart + 2 * 4 * GB;                              // [2][GB]
  float *vmaxw = mstat + 2 * GB;                                  // e4m3: [2][GB][4], read as float4 like xmax
  float *refs = vmaxw + 8 * GB;                                   // e4m3: [4][4][GB], a warp's own
  float *qscale = E4M3 ? refs + 16 * GB : vmaxw;                  // e4m3: [2][GB]
  float *vstat = E4M3 ? qscale + 2 * GB : vmaxw;                  // e4m3: [2][GB]
  float2 *vspan = reinterpret_cast<float2 *>(vstat + 2 * GB);       // e4m3: [2][kGroups][4]
  static_assert(C::kMiscOff % 16 == 0 && (18 * GB) % 4 == 0 && C::kMiscFloats % 4 == 0, "xmax and vmaxw on 16 bytes");
  uint8_t *ring = smem + C::kRingOff;

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const WaitCtx ctx{p.c.status, abort_flag, kKernelDecode, p.c.seq};
  if (warp == C::kQWarp) {
    if (lane < 2) {
      mbar_init(&bar_q[lane], 32);
      // The issuer's commit; e4m3: and the softmax warps, for q's scale.
      mbar_init(&bar_q_empty[lane], 1 + (E4M3 ? C::kSoftmaxWarps : 0));
      mbar_init(&bar_s[lane], 1);
      mbar_init(&bar_p[lane], C::kSoftmaxWarps);
      mbar_init(&bar_pv[lane], 1);
      mbar_init(&bar_o[lane], 1);
      mbar_init(&bar_o_empty[lane], 4);
      mbar_init(&bar_stat[lane], C::kSoftmaxWarps);
    }
    if (lane < C::kScStages) {
      mbar_init(&bar_sc[lane], 32);
      mbar_init(&bar_sc_empty[lane], C::kSoftmaxWarps);
    }
    if (lane < C::kSlots) {
      mbar_init(&bar_full[lane], 1);
      mbar_init(&bar_empty[lane], 1);
    }
    if (lane < 12) share[lane] = 0;
    __syncwarp();
    if (lane == 0) {
      mbar_init(bar_drain, 1);
      *abort_flag = 0;
      if ((smem_u32(smem) & 1023u) != 0) {
        record_failure(ctx, kStatusInternal, 0);
        share[7] = 1;
      }
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
    }
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == C::kIssuer) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
    // Only now: a kernel that starts early must not take the tensor memory that this one, which
    // it will wait for, has yet to get.
    pdl_launch();
  }
  pdl_wait();  // nothing before this reads or writes what the stream's earlier kernels may touch

  // ---------------------------------------------------------------- the share
  // Thread i counts tiles and cost of sequences [i * per, (i + 1) * per); a scan over the
  // threads gives every share's first sequence.  Up to 32 sequences are a warp's scan, done by
  // every warp for itself (the shared sums and a barrier later a call takes 0.3 us more).
  {
    const bool small = p.c.B <= 32;
    const int per = small ? 1 : (p.c.B + C::kThreads - 1) / C::kThreads;
    const int b_lo = min(p.c.B, small ? lane : static_cast<int>(threadIdx.x) * per), b_hi = min(p.c.B, b_lo + per);
    const int len_lo = b_lo < b_hi ? __ldg(p.c.seq_lens + b_lo) : 0;
    const int items = p.c.H * p.nblk;
    auto tiles_of = [&](int b) {
      const int raw = b == b_lo ? len_lo : __ldg(p.c.seq_lens + b);
      const int len = min(max(raw, 0), p.c.cap);
      if (raw != len) record_cache_error(p.c.status, kKernelDecode, b, p.c.seq);
      return ((len + 127) >> 7) - (DecodeWalk::first_of(p, len) >> 7);
    };
    int tiles = 0, live = 0;  // of these sequences: tiles, and items that have any
#pragma unroll 1
    for (int b = b_lo; b < b_hi; ++b) {
      const int n = tiles_of(b);
      tiles += n * items;
      live += n > 0 ? items : 0;
    }
    int it = tiles, ic = live;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int ut = __shfl_up_sync(0xffffffffu, it, o), uc = __shfl_up_sync(0xffffffffu, ic, o);
      if (lane >= o) {
        it += ut;
        ic += uc;
      }
    }
    int total_t = __shfl_sync(0xffffffffu, it, 31), total_i = __shfl_sync(0xffffffffu, ic, 31);
    int before_t = it - tiles, before_i = ic - live;
    if (!small) {
      int2 *sums = reinterpret_cast<int2 *>(smem);  // [kWarps], before anything else is there
      if (lane == 31) sums[warp] = make_int2(it, ic);
      __syncthreads();
      const int2 v = lane < C::kWarps ? sums[lane] : make_int2(0, 0);
      total_t = __reduce_add_sync(0xffffffffu, v.x);
      total_i = __reduce_add_sync(0xffffffffu, v.y);
      before_t += __reduce_add_sync(0xffffffffu, lane < warp ? v.x : 0);
      before_i += __reduce_add_sync(0xffffffffu, lane < warp ? v.y : 0);
    } else {
      __syncthreads();  // share[] is zero
    }
    const int nc = min(static_cast<int>(gridDim.x), total_t), c = static_cast<int>(blockIdx.x);
    if (c < nc) {
      const int extra = total_t / C::kItemTiles >= nc ? C::kItemCost : 0;
      const int total_c = C::kTileCost * total_t + extra * total_i;
      const int before_c = C::kTileCost * before_t + extra * before_i, cost = C::kTileCost * tiles + extra * live;
      auto cost_of = [&](int n) { return n > 0 ? (extra + C::kTileCost * n) * items : 0; };
      const DecodeSplit sp(total_c, nc);
      // The share's first unit, and the next share's (of a small batch: by warp 0 and warp 1).
#pragma unroll 1
      for (int e = small ? warp : 0; e < (small ? min(warp + 1, 2) : 2); ++e) {
        const int x = sp.begin(c + e);
        if (e == 1 && x == total_c && lane == 0) share[11] = total_t;
        if (cost == 0 || x < before_c || x >= before_c + cost) continue;
        int b = b_lo, n = tiles_of(b), at = x - before_c, t0 = before_t;
#pragma unroll 1
        while (at >= cost_of(n)) {
          at -= cost_of(n);
          t0 += n * items;
          n = tiles_of(++b);
        }
        const int one = extra + C::kTileCost * n, item = at / one;
        const int off = max(at - item * one - extra, 0) / C::kTileCost;
        share[10 + e] = t0 + item * n + off;
        if (e == 0) {
          share[0] = b;
          share[1] = p.nblk == 1 ? item : item / p.nblk;
          share[2] = off;
          share[6] = p.nblk == 1 ? 0 : item % p.nblk;
          share[8] = min(b == b_lo ? len_lo : __ldg(p.c.seq_lens + b), p.c.cap);
          share[9] = x - at + item * one;
          share[3] = extra;
          share[4] = total_c;
          share[5] = nc;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t kOCol0 = 2 * C::kQCols;

  DecodeWalk wk;
  wk.start(p, share);

  if (warp == C::kProducer) {
    // ------------------------------------------------------------- producer
    // Lane i loads page i of a tile (pages of 128 rows or more: lane 0 alone).
    const int rows = min(p.c.page_size, 128);
    const int pages = 128 / rows;
    DecodePages pg;
    bool ok = true;
    int g = 0, s = 0;        // slots filled so far, and the next one
    uint32_t ph = 1;         // its "empty" phase: the first round passes at once
    while (wk.rem > 0 && ok) {
      const int pos0 = (wk.tile0 + wk.off) << 7;
      const int pi = pg.seek(p, wk, pos0);
      // A page out of the table's range is out of the tensor map's: TMA fills with zeros.
      const int page = __shfl_sync(0xffffffffu, pg.ids, (pi + lane) & 31);
      const bool need = lane < pages && page >= 0;
      const int row = pages == 1 ? pos0 - pi * p.c.page_size : 0;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, need)) * rows * C::kRowBytes;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv, ++g) {
        if (!(ok = __all_sync(0xffffffffu, decode_wait(ctx, &bar_empty[s], ph, kTagDEmpty)))) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar_full[s], bytes);
        __syncwarp();
        if (need)
          for (int i = 0; i < C::kPanels; ++i)
            tma_load_4d(kv == 0 ? &tmK : &tmV, &bar_full[s],
                        ring + s * C::kTileBytes + i * C::kPanelBytes + lane * rows * C::kPanelRow,
                        i * (C::kPanelRow / C::kElem), row, wk.h, page);
        __syncwarp();
        if (++s == C::kSlots) {
          s = 0;
          ph ^= 1;
        }
      }
      pg.ahead(p, wk);
      wk.advance(p, 1);
    }
    // The last loads have landed before the CTA can exit.
#pragma unroll 1
    for (int i = 0; i < C::kSlots && i < g; ++i) mbar_drain(&bar_full[i], ((g - 1 - i) / C::kSlots) & 1);
    __syncwarp();
  } else if (warp == C::kIssuer) {
    // --------------------------------------------------------------- issuer
    // S^T of tile n goes in ahead of V^T P of tile n - 1, across segments too.  That order
    // stands for barriers: P of tile n - 2 tells that the softmax warps have read S^T of it,
    // whose columns tile n takes; and S^T of tile n being complete tells them that V^T P of
    // tile n - 2 is, whose P they overwrite.  The loop is what a CTA's tile takes at least,
    // and a satisfied wait is some 100 cycles of it.  So V and P, usually both there, are
    // looked at by two lanes at once (a wait that may suspend must not be: with lanes on
    // different barriers it sleeps to its limit).
    constexpr uint32_t kBIsE5m2 = 1u << 10;  // B's format: the weights' parts
    constexpr uint32_t idesc_s = E4M3 ? make_idesc_e4m3(128, C::kQCols, 0, 0) : make_idesc_bf16(128, C::kQCols, 0, 0);
    constexpr uint32_t idesc_o = E4M3 ? make_idesc_e4m3(128, C::kOCols, 1, 1) | kBIsE5m2 : make_idesc_bf16(128, C::kOCols, 1, 1);
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint32_t ring0 = smem_u32(ring);
    // K (rows are keys) and Q (rows are heads) are K-major in the same panels.  With 8 bf16
    // rows of Q the 16 columns repeat them (row groups 0 bytes apart).
    const uint64_t k_desc0 = make_sdesc_row(C::kPanelRow, ring0, 16, 8 * C::kPanelRow);
    const uint64_t q_desc0 =
        make_sdesc_row(C::kPanelRow, smem_u32(smem + C::kQOff), 16, C::kQRows < 16 ? 0 : 8 * C::kPanelRow);
    // V as the M x K operand V^T is MN-major.  M = 128 features are d = 128's, in panels
    // kPanelBytes apart; for d = 64 the second half repeats the first (offset 0), and its
    // half of O^T is not read.
    const uint64_t v_desc0 = make_sdesc_row(C::kPanelRow, ring0, D == 128 ? C::kPanelBytes : 0, 8 * C::kPanelRow);
    // P as the K x N operand is MN-major too, one row of kPRow bytes per key.
    const uint64_t p_desc0 = make_sdesc_row(C::kPRow, smem_u32(smem + C::kPOff), 16, 8 * C::kPRow);
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity, int tag) {
      return __all_sync(0xffffffffu, decode_wait(ctx, bar, parity, tag));
    };
    int s = 0;          // ring slot of the next K; its V is in the next one
    uint32_t ph = 0;    // the slot's "full" phase
    auto next_slot = [&]() {
      if (++s == C::kSlots) {
        s = 0;
        ph ^= 1;
      }
    };
    // The previous tile's segment, place in it and V slot (seg -1: no tile yet).
    int seg = 0, pend_seg = -1, pend_s = 0;
    uint32_t pend_ph = 0;
    bool begins = true, pend_first = false, pend_last = false;
    for (int n = 0;; ++n) {
      const int buf = n & 1, qb = seg & 1;
      const bool more = wk.rem > 0, ends = wk.run() == 1;
      if (more) {
        if (begins && !(ok = wait(&bar_q[qb], (seg >> 1) & 1, kTagDQ))) break;
        if (!(ok = wait(&bar_full[s], ph, kTagDFull))) break;
        tc_fence_after();
        const uint64_t kd = sdesc_add(k_desc0, s * C::kTileBytes), qd = sdesc_add(q_desc0, qb * C::kQBytes);
        const uint32_t ts = tm + buf * C::kQCols;
#pragma unroll
        for (int ks = 0; ks < C::kRowBytes / 32; ++ks) {  // 32 bytes of the rows per instruction
          const uint64_t a = sdesc_add(kd, (ks >> 2) * C::kPanelBytes + (ks & 3) * 32);
          const uint64_t b = sdesc_add(qd, (ks >> 2) * C::kQRows * C::kPanelRow + (ks & 3) * 32);
          if constexpr (E4M3)
            mma_ss_f8_w(ts, a, b, idesc_s, ks > 0);
          else
            mma_ss_w(ts, a, b, idesc_s, ks > 0);
        }
        mma_commit_w(&bar_empty[s]);
        mma_commit_w(&bar_s[buf]);
        if (ends) mma_commit_w(&bar_q_empty[qb]);
      }
      if (pend_seg >= 0) {  // V^T P of tile n - 1
        const int pb = buf ^ 1, ob = pend_seg & 1;
        if (pend_first && pend_seg >= 2 && !(ok = wait(&bar_o_empty[ob], ((pend_seg >> 1) - 1) & 1, kTagDOEmpty))) break;
        const uint32_t php = ((n - 1) >> 1) & 1;
        if (!__all_sync(0xffffffffu, decode_test(lane == 0 ? &bar_full[pend_s] : &bar_p[pb], lane == 0 ? pend_ph : php))) {
          if (!(ok = wait(&bar_full[pend_s], pend_ph, kTagDFull))) break;
          if (!(ok = wait(&bar_p[pb], php, kTagDP))) break;
        }
        tc_fence_after();
        const uint64_t vd = sdesc_add(v_desc0, pend_s * C::kTileBytes), pd = sdesc_add(p_desc0, pb * C::kPBytes);
        const uint32_t to = tm + kOCol0 + ob * C::kOCols;
        constexpr int kStep = E4M3 ? 32 : 16;  // keys per instruction
#pragma unroll
        for (int ks = 0; ks < 128 / kStep; ++ks) {
          const uint64_t a = sdesc_add(vd, ks * kStep * C::kPanelRow), b = sdesc_add(pd, ks * kStep * C::kPRow);
          if constexpr (E4M3)
            mma_ss_f8_w(to, a, b, idesc_o, (!pend_first || ks > 0) ? 1u : 0u);
          else
            mma_ss_w(to, a, b, idesc_o, (!pend_first || ks > 0) ? 1u : 0u);
        }
        mma_commit_w(&bar_empty[pend_s]);
        if constexpr (C::kPvBar) mma_commit_w(&bar_pv[pb]);
        if (pend_last) mma_commit_w(&bar_o[ob]);
      }
      if (!more) break;
      pend_seg = seg;
      pend_first = begins;
      pend_last = ends;
      begins = ends;
      seg += ends ? 1 : 0;
      next_slot();
      pend_s = s;
      pend_ph = ph;
      next_slot();
      wk.advance(p, 1);
    }
    if (!ok) {
      mma_commit_w(bar_drain);
      mbar_drain(bar_drain, 0);
    }
    __syncwarp();
  } else if (warp == C::kQWarp) {
    // ---------------------------------------------------------------- Q rows
    // Rows of the segment's query heads into swizzled shared memory, kHeads at a time; the next
    // ones (of this segment or the next) are read meanwhile.  A lane's piece i is 16 bytes, of bf16 the
    // (32 i + lane)th of the rows.  Rows past the last head are 0.
    constexpr int kPerRow = D / 8, kAll = C::kHeads * kPerRow, kPieces = (kAll + 31) / 32;
    // (e4m3: of kLanes lanes to a row, so that its maximum takes few shuffles: 64 ragged sequences up to
    // 4096 with 32 heads 26.5 us, 28.3 with the pieces in order.)
    constexpr int kLanes = 32 / C::kHeads;
    auto row_of = [&](int i) { return E4M3 ? lane / kLanes : (32 * i + lane) / kPerRow; };
    auto piece_of = [&](int i) { return E4M3 ? i * kLanes + lane % kLanes : (32 * i + lane) % kPerRow; };
    auto there = [&](int i) { return E4M3 ? piece_of(i) < kPerRow : 32 * i + lane < kAll; };
    uint4 w[kPieces];
    auto load = [&](int c) {
      const int g0 = wk.blk * GB + C::kHeads * c;
      const uint16_t *src = p.q + (static_cast<long long>(wk.b) * p.Hq + wk.h * p.G + g0) * D;
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (wk.rem > 0 && there(i) && g0 + row_of(i) < p.G)
          w[i] = __ldg(reinterpret_cast<const uint4 *>(src) + row_of(i) * kPerRow + piece_of(i));
      }
    };
    bool ok = true;
    load(0);
    for (int seg = 0; wk.rem > 0 && ok; ++seg) {
      const int qb = seg & 1;
      if (seg >= 2 && !(ok = __all_sync(0xffffffffu, decode_wait(ctx, &bar_q_empty[qb], ((seg >> 1) - 1) & 1, kTagDQEmpty))))
        break;
      const uint32_t dst = smem_u32(smem + C::kQOff) + qb * C::kQBytes;
#pragma unroll 1
      for (int c = 0; c < C::kGroups; ++c) {
        uint4 v[kPieces];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) v[i] = w[i];
        if (c + 1 == C::kGroups) wk.advance(p, wk.run());
        load(c + 1 == C::kGroups ? 0 : c + 1);
        if constexpr (!E4M3) {
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const int row = C::kHeads * c + row_of(i), in = piece_of(i);
            if (!there(i)) break;
            st_shared_v4(dst + (in >> 3) * (C::kQRows * 128) + swizzled<128>(row, (in & 7) * 16), v[i].x, v[i].y, v[i].z,
                         v[i].w);
          }
        } else {
          // Scale each row by the power of two that brings its largest element into
          // [128, 256), then split: hi = e4m3(x), lo = e4m3(32 (x - hi)) (bf16 values are
          // fp16 values in that range, |x - hi| is at most 8).  An element is off by at most 2^-22 of its
          // row's largest.  (One scale for 8 rows would make a head's error another's affair, a NaN included.)
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const uint32_t a = __vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu);
            const uint32_t b = __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu);
            top = __vmaxu2(top, __vmaxu2(a, b));
          }
          top = max(top >> 16, top & 0xffffu);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
          // The row's largest element is in [2^(e-127), 2^(e-126)); x * 2^(134 - e).  An infinity or
          // NaN (e = 255) makes every score of the head NaN.
          const int e0 = static_cast<int>(top >> 7), e = min(max(e0, 16), 250), row = C::kHeads * c + row_of(0);
          const float up = __uint_as_float(static_cast<uint32_t>(261 - e) << 23);
          if (lane % kLanes == 0)
            qscale[qb * GB + row] =
                __uint_as_float(e0 == 255 ? 0x7fc00000u : static_cast<uint32_t>(e - 7) << 23) * p.scale_log2;
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            const uint32_t words[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t part[2][2] = {{0u, 0u}, {0u, 0u}};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t r = pack_f16(bf16_lo(words[k]) * up, bf16_hi(words[k]) * up);
              const uint16_t hi = f16x2_to_e4m3x2(r);
              const uint16_t lo = f16x2_to_e4m3x2(f16x2_mul(f16x2_sub(r, e4m3x2_to_f16x2(hi)), 0x50005000u));  // 32
              part[0][k >> 1] |= static_cast<uint32_t>(hi) << (16 * (k & 1));
              part[1][k >> 1] |= static_cast<uint32_t>(lo) << (16 * (k & 1));
            }
            const int byte = piece_of(i) * 8;
            if (!there(i)) break;
#pragma unroll
            for (int k = 0; k < 2; ++k)
              st_shared_v2(dst + swizzled<C::kPanelRow>(k * GB + row, byte & ~15) + (byte & 8), part[k][0], part[k][1]);
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&bar_q[qb]);
    }
    __syncwarp();
  } else if (warp == C::kScales) {
    // ------------------------------------------------- the keys' factors (e4m3)
    if constexpr (E4M3) {
      // A lane copies the factors of keys 4 lane .. 4 lane + 3 at once where they are one
      // aligned piece (tokens adjacent), else those of keys lane, lane + 32, ...  Keys without
      // a page are left as they are: the softmax warps mask them.
      const int rows = min(p.c.page_size, 128), shift = 31 - __clz(rows);
      DecodePages pg;
      for (int n = 0; wk.rem > 0; ++n) {
        const int st = n % C::kScStages;
        const int pos0 = (wk.tile0 + wk.off) << 7;
        const int pi = pg.seek(p, wk, pos0);
        const int row0 = rows == 128 ? pos0 - pi * p.c.page_size : 0;
        if (n >= C::kScStages &&
            !__all_sync(0xffffffffu, decode_wait(ctx, &bar_sc_empty[st], (n / C::kScStages - 1) & 1, kTagDScEmpty)))
          break;
        const uint32_t dst = smem_u32(smem + C::kScOff) + st * 1024;
#pragma unroll 1
        for (int i = 0; i < (p.vec_scales ? 1 : 4); ++i) {
          const int key = p.vec_scales ? 4 * lane : 32 * i + lane;
          const int page = __shfl_sync(0xffffffffu, pg.ids, (pi + (key >> shift)) & 31);
          if (page >= 0 && page < p.c.num_pages) {
            const int row = row0 + (key & (rows - 1));
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
              const float *src = p.c.scale[kv] + (page * p.c.scale_stride[kv][0] + wk.h * p.c.scale_stride[kv][1] +
                                                  row * p.c.scale_stride[kv][2]);
              if (p.vec_scales)
                cp_async16(dst + kv * 512 + key * 4, src);
              else
                cp_async4(dst + kv * 512 + key * 4, src);
            }
          }
        }
        __syncwarp();
        cp_async_arrive(&bar_sc[st]);
        pg.ahead(p, wk);
        wk.advance(p, 1);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
    }
  } else if (warp < C::kSoftmaxWarps) {
    // -------------------------------------------------------------- softmax
    // Thread = key (row of S^T, tensor memory lane) and group of kHeads heads, kept in pairs.
    // All waits are bounded and every thread of the group reaches every bar_any, so a
    // failed wait (`bad`) ends the group's four warps together.
    const int grp = warp >> 2, w4 = warp & 3, key = w4 * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(w4 * 32) << 16;
    const uint32_t bar_a = 1 + 2 * grp, bar_b = 2 + 2 * grp;
    constexpr int kH = C::kHeads, kPairs = kH / 2, kSpan = 32 / kH;  // kSpan lanes end up with one head's maximum
    float *xm = xmax + kH * grp * 4;
    uint64_t nm2[kPairs], l2[kPairs];           // minus the reference, and this key's sum of weights
    float code = 1.f;  // e4m3: of the group's heads (decode_references)
    float *ref = refs + 4 * w4 * GB + kH * grp + lane / kSpan;  // of head lane / kSpan: m, r, e and unit, GB apart
    bool bad = false, stop = false;
    int n = 0, nred = 0, sv = 1;      // tiles, reductions, ring slot of the tile's V
    uint32_t vph = 0;
    for (int seg = 0; wk.rem > 0 && !stop; ++seg) {
      const int run = wk.run(), qb = seg & 1;
      const float *qs = qscale + qb * GB + kH * grp;  // e4m3: scale and what was taken out of q, per head
      if constexpr (E4M3) bad |= !decode_wait(ctx, &bar_q[qb], (seg >> 1) & 1, kTagDQ);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) nm2[i] = l2[i] = 0ull;
#pragma unroll 1
      for (int i = 0; i < run; ++i, ++n) {
        const int buf = n & 1;
        const int pos0 = (wk.tile0 + wk.off + i) * 128;
        float fk = 1.f, fv = 1.f;
        if constexpr (E4M3) {  // the factors are there first, as a rule
          const int st = n % C::kScStages;
          bad |= !decode_wait(ctx, &bar_sc[st], (n / C::kScStages) & 1, kTagDSc);
          const float *sc = reinterpret_cast<const float *>(smem + C::kScOff + st * 1024);
          // x + 0 x: an infinite factor counts as NaN.  Of an appended row its codes are 0 and NaN, and
          // elsewhere it would give a score or a weight of one sign only where its codes have both.
          fk = __fmaf_rn(sc[key], 0.f, sc[key]);
          fv = __fmaf_rn(sc[128 + key], 0.f, sc[128 + key]);
        }
        // How far a weight (log2) may go before the references move.  e4m3: the code's limit, or the weight's.
        float room = E4M3 ? fminf(C::kCodeLog2 + C::kGrowV - lg2(fabsf(fv * code)), C::kHeadLog2 + C::kGrow) : C::kGrow;
        bad |= !decode_wait(ctx, &bar_s[buf], (n >> 1) & 1, kTagDS);
        __syncwarp();
        tc_fence_after();
        uint64_t v2[kPairs];  // scores (before their factor at first)
        {
          const uint32_t ts = tmem + lane_off + buf * C::kQCols + kH * grp;
          uint32_t hi[kH], lo[kH];
          tmem_ld_n<kH>(ts, hi);
          if constexpr (E4M3) tmem_ld_n<kH>(ts + GB, lo);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (E4M3 && lane == 0) mbar_arrive(&bar_sc_empty[n % C::kScStages]);
#pragma unroll
          for (int g = 0; g < kPairs; ++g) {
            v2[g] = f2pack(__uint_as_float(hi[2 * g]), __uint_as_float(hi[2 * g + 1]));
            if constexpr (E4M3)
              v2[g] = ffma2(f2pack(__uint_as_float(lo[2 * g]), __uint_as_float(lo[2 * g + 1])), f2pack(0.03125f, 0.03125f),
                            v2[g]);
          }
        }
        // Scores in the log2 domain, rounded here: a fused multiply-subtract below would be
        // off from the maximum by the rounding of a product, however large that is.
#pragma unroll
        for (int g = 0; g < kPairs; ++g) {
          uint64_t f = f2pack(p.scale_log2, p.scale_log2);
          if constexpr (E4M3) f = mul2(f2pack(fk, fk), reinterpret_cast<const uint64_t *>(qs)[g]);
          v2[g] = mul2(v2[g], f);
        }
        if (pos0 < wk.first || pos0 + 128 > wk.len) {
          const int pos = pos0 + key;
          const bool valid = pos >= wk.first && pos < wk.len;
          if (!valid) {
            fv = 0.f;
            room = INFINITY;  // what the row has for a factor must not move anything
#pragma unroll
            for (int g = 0; g < kPairs; ++g) v2[g] = f2pack(-INFINITY, -INFINITY);
          }
          // Masked rows of V: weight 0 times whatever the page holds has to be 0.
          if (grp == 0) {
            bad |= !decode_wait(ctx, &bar_full[sv], vph, kTagDFull);
            if (!valid) {
              uint8_t *rowp = ring + sv * C::kTileBytes + key * C::kPanelRow;
#pragma unroll 1
              for (int ch = 0; ch < C::kRowBytes / 16; ++ch) {
                // Lanes start at different chunks, so that their stores fall into different banks.
                const int c = (ch + lane) % (C::kRowBytes / 16);
                *reinterpret_cast<uint4 *>(rowp + (c * 16 / C::kPanelRow) * C::kPanelBytes + (c * 16) % C::kPanelRow) =
                    make_uint4(0u, 0u, 0u, 0u);
              }
            }
          }
          __syncwarp();
        }
        float x[kH];  // log2 of the weights
        bool grow = true;
        if (i > 0) {
#pragma unroll
          for (int g = 0; g < kPairs; ++g) f2unpack(fadd2(v2[g], nm2[g]), x[2 * g], x[2 * g + 1]);
          float top = x[0];
#pragma unroll
          for (int g = 1; g < kH; ++g) top = fmaxf(top, x[g]);
          grow = top >= room;  // (room is -inf where factor * code overflows, and top where all weights are 0)
          grow = bar_any(bar_a, 128, grow || bad);
        }
        if (grow) {
          // The reference moves (or a segment begins) to the maximum over the keys so far.
          float *xr = xm + (nred & 1) * GB * 4;
          float v[kH];
#pragma unroll
          for (int g = 0; g < kPairs; ++g) f2unpack(v2[g], v[2 * g], v[2 * g + 1]);
          if constexpr (E4M3)
            v[0] = max_columns<kH>(v);
          else
            reduce_columns<kH>(v, [](float a, float b) { return fmaxf(a, b); });
          if (lane % kSpan == 0) xr[lane / kSpan * 4 + w4] = v[0];
          float2 *span = vspan + ((nred & 1) * C::kGroups + grp) * 4;
          if constexpr (E4M3) {
            const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(fv)));
            const bool seen = pos0 + key >= wk.first && pos0 + key < wk.len;
            const uint32_t least = __reduce_min_sync(0xffffffffu, seen ? __float_as_uint(fabsf(fv)) : 0x7f800000u);
            if (lane == 0) span[w4] = make_float2(__uint_as_float(most), __uint_as_float(least));
          }
          if (bar_any(bar_b, 128, bad)) {
            stop = true;
            break;
          }
          // Head lane / kSpan's maximum; the lowest number stands in for -inf, so that differences stay defined.
          const float4 m4 = *reinterpret_cast<const float4 *>(xr + lane / kSpan * 4);
          const float mc = fmaxf(fmaxf(fmaxf(m4.x, m4.y), fmaxf(m4.z, m4.w)), -3.402823466e38f);
          float alpha[kH];  // what O is multiplied by
          if constexpr (!E4M3) {
#pragma unroll
            for (int g = 0; g < kPairs; ++g) {
              float a, b;
              f2unpack(nm2[g], a, b);
              float m0 = __shfl_sync(0xffffffffu, mc, 2 * g * kSpan), m1 = __shfl_sync(0xffffffffu, mc, (2 * g + 1) * kSpan);
              if (i > 0) {
                m0 = fmaxf(m0, -a);
                m1 = fmaxf(m1, -b);
              }
              alpha[2 * g] = ex2(-a - m0);
              alpha[2 * g + 1] = ex2(-b - m1);
              nm2[g] = f2pack(-m0, -m1);
              if (i > 0) l2[g] = mul2(l2[g], f2pack(alpha[2 * g], alpha[2 * g + 1]));
            }
          } else {
            // Rows of Q without a head (next to ones that have) have no say and no weight.
            const int live = p.G - wk.blk * GB - kH * grp;
            const bool none = live > 0 && lane / kSpan >= live;
            const float4 s0 = reinterpret_cast<const float4 *>(span)[0], s1 = reinterpret_cast<const float4 *>(span)[1];
            const float most = fmaxf(fmaxf(s0.x, s0.z), fmaxf(s1.x, s1.z)), least = fminf(fminf(s0.y, s0.w), fminf(s1.y, s1.w));
            DecodeRefs now;
            uint32_t next;
            float of_l = 1.f, of_o = 1.f;  // what l and O are multiplied by
            const bool alike = most <= kFactorSpan * least;
            if (i == 0 && alike) {
              // Every head has a weight of 1 in the tile: the largest factor will do for all their products.
              const uint32_t e = decode_power(most);
              next = ((254u + C::kCodeLog2) << 23) - e;
              now = {mc, mc, __uint_as_float(e), 1.f};
            } else {
              DecodeRefs old = {mc, 0.f, 0.f, 0.f};
              if (i > 0) old = {ref[0], ref[GB], ref[2 * GB], 0.f};
              const float mx = fmaxf(mc, old.m);
              // The tile's largest product relative to the new maximum.  (No factor, seen or not, above 2^120
              // times it: factor * code stays finite.)
              float product;
              if (alike) {
                product = fmaxf(ex2(mc - mx), 0x1p-120f) * most;  // its own largest weight times any factor
              } else {
                // A value row counts with the weight it has: one much larger than the others that is hardly
                // seen leaves their resolution alone.
                DecodeScores<kPairs> scores;
#pragma unroll
                for (int g = 0; g < kPairs; ++g) scores.v2[g] = v2[g];
                product = decode_products<kH>(scores, mx, fv, vmaxw + (kH * grp + (nred & 1) * GB) * 4, bar_b);
              }
              now = decode_references<C>(mx, none ? 0.f : fmaxf(product, old.e * ex2(old.m - mx)), next);
              // O goes by the codes, l by the weights.
              const float up = static_cast<float>(static_cast<int>(next >> 23) - static_cast<int>(__float_as_uint(code) >> 23));
              of_l = ex2(old.r - now.r);
              of_o = ex2((old.r - now.r) + up);
            }
            if (none) now.r = INFINITY;
            code = __uint_as_float(next);
            __syncwarp();
            if (lane % kSpan == 0) {
              ref[0] = now.m;
              ref[GB] = now.r;
              ref[2 * GB] = now.e;
              ref[3 * GB] = now.unit;
            }
            __syncwarp();
            auto head = [&](float v, int g) { return __shfl_sync(0xffffffffu, v, g * kSpan); };
#pragma unroll
            for (int g = 0; g < kPairs; ++g) {
              nm2[g] = f2pack(-head(now.r, 2 * g), -head(now.r, 2 * g + 1));
              if (i > 0) {
                alpha[2 * g] = head(of_o, 2 * g);
                alpha[2 * g + 1] = head(of_o, 2 * g + 1);
                l2[g] = mul2(l2[g], f2pack(head(of_l, 2 * g), head(of_l, 2 * g + 1)));
              }
            }
          }
          ++nred;
          if (i > 0) {
            // O holds tiles of this segment on the old reference: bring it to the new one.
            if constexpr (C::kPvBar) {
              bad |= !decode_wait(ctx, &bar_pv[(n - 1) & 1], ((n - 1) >> 1) & 1, kTagDPv);
            } else {
              const int back = sv - 2 + (sv < 2 ? C::kSlots : 0);
              bad |= !decode_wait(ctx, &bar_empty[back], vph ^ (sv < 2 ? 1u : 0u), kTagDPv);
            }
            __syncwarp();
            tc_fence_after();
            const uint32_t to = tmem + lane_off + kOCol0 + (seg & 1) * C::kOCols + kH * grp;
#pragma unroll 1
            for (int part = 0; part < C::kOParts; ++part) {
              uint32_t o[kH];
              tmem_ld_n<kH>(to + part * GB, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < kH; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha[e]);
              tmem_st_n<kH>(to + part * GB, o);
            }
            tmem_wait_st();
            tc_fence_before();
          }
#pragma unroll
          for (int g = 0; g < kPairs; ++g) f2unpack(fadd2(v2[g], nm2[g]), x[2 * g], x[2 * g + 1]);
        }
        // Weights into P: row = key, this group's heads of each part.
        const uint32_t pb = smem_u32(smem + C::kPOff) + buf * C::kPBytes;
        uint32_t part[C::kOParts][kPairs];
#pragma unroll
        for (int g = 0; g < kPairs; ++g) {
          const float a = ex2(x[2 * g]), b = ex2(x[2 * g + 1]);
          l2[g] = fadd2(l2[g], f2pack(a, b));
          if constexpr (!E4M3) {
            part[0][g] = pack_bf16(a, b);
            part[1][g] = pack_bf16(a - bf16_lo(part[0][g]), b - bf16_hi(part[0][g]));
          } else {
            const float fc = fv * code;
            uint32_t four[4];
            decode_parts(mul2(f2pack(a, b), f2pack(fc, fc)), four);
#pragma unroll
            for (int k = 0; k < 4; ++k) part[k][g] = four[k];
          }
        }
        if constexpr (E4M3 && kPairs > 1) {  // the codes of two pairs a word
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int g = 0; g < kPairs / 2; ++g)
              part[k][g] = __byte_perm(part[k][2 * g], part[k][2 * g + 1], k < 3 ? 0x7531 : 0x5410);
        }
        constexpr int kPartBytes = kH * C::kElem;  // of this thread, per part
        if constexpr (kPartBytes == 16) {
#pragma unroll
          for (int k = 0; k < C::kOParts; ++k)
            st_shared_v4(pb + swizzled<C::kPRow>(key, 2 * (k * GB + kH * grp)), part[k][0], part[k][1], part[k][2],
                         part[k][3]);
        } else if constexpr (kPartBytes == 8 && E4M3) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int byte = k * GB + kH * grp;
            st_shared_v2(pb + swizzled<C::kPRow>(key, byte & ~15) + (byte & 8), part[k][0], part[k][1]);
          }
        } else if constexpr (!E4M3) {  // 2 or 4 heads: the parts are neighbours
          const uint32_t at = pb + swizzled<C::kPRow>(key, 0);
          if constexpr (kH == 4)
            st_shared_v4(at, part[0][0], part[0][1], part[1][0], part[1][1]);
          else
            st_shared_v2(at, part[0][0], part[1][0]);
        } else {
          const uint32_t at = pb + swizzled<C::kPRow>(key, 0);
          if constexpr (kH == 4)
            st_shared_v4(at, part[0][0], part[1][0], part[2][0], part[3][0]);
          else  // two heads: two codes of each part
            st_shared_v2(at, __byte_perm(part[0][0], part[1][0], 0x7531), __byte_perm(part[2][0], part[3][0], 0x5431));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_p[buf]);
        if ((sv += 2) >= C::kSlots) {
          sv -= C::kSlots;
          vph ^= 1;
        }
      }
      if (stop) break;
      // The segment's statistics for the epilogue.
      const int ob = seg & 1;
      if (seg >= 2) bad |= !decode_wait(ctx, &bar_o_empty[ob], ((seg >> 1) - 1) & 1, kTagDOEmpty);
      __syncwarp();
      float l[kH], m[kH];
#pragma unroll
      for (int g = 0; g < kPairs; ++g) {
        f2unpack(l2[g], l[2 * g], l[2 * g + 1]);
        f2unpack(nm2[g], m[2 * g], m[2 * g + 1]);
      }
      reduce_columns<kH>(l, [](float a, float b) { return a + b; });
      if constexpr (E4M3) {
        // On the maximum, and what a code stands for.  (Parts of a sequence have references of their
        // own, and the join's exponentials no room for their deltas.)
        l[0] *= ref[3 * GB];
        if (w4 == 0 && lane % kSpan == 0) {
          mstat[ob * GB + kH * grp + lane / kSpan] = ref[0];
          vstat[ob * GB + kH * grp + lane / kSpan] = ref[2 * GB] * (1.f / (1 << C::kCodeLog2));
        }
      } else if (w4 == 0 && lane == 0) {
#pragma unroll
        for (int g = 0; g < kH; ++g) mstat[ob * GB + kH * grp + g] = -m[g];
      }
      if (lane % kSpan == 0) lpart[(ob * 4 + w4) * GB + kH * grp + lane / kSpan] = l[0];
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
    const int f = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
#pragma unroll 1
    for (int at = 0; at < p.c.B; at += 128 * gridDim.x) {
      const int mine = at + f * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
      uint32_t idle = __ballot_sync(0xffffffffu, mine < p.c.B && __ldg(p.c.seq_lens + mine) <= 0);
      for (; idle; idle &= idle - 1) {
        const int b = __shfl_sync(0xffffffffu, mine, __ffs(idle) - 1);
        const long long row0 = static_cast<long long>(b) * p.Hq;
        if (p.by_item)
#pragma unroll 1
          for (int e = lane; e < p.c.H * p.nblk; e += 32) p.meta[b * p.c.H * p.nblk + e] = make_int4(0, 0, 0, 0);
#pragma unroll 1
        for (int e = lane; e < p.Hq * D / 8; e += 32)
          reinterpret_cast<uint4 *>(p.o + row0 * D)[e] = make_uint4(0u, 0u, 0u, 0u);
        if (p.lse)
#pragma unroll 1
          for (int e = lane; e < p.Hq; e += 32) p.lse[row0 + e] = -INFINITY;
      }
    }
    if (!p.by_item && f == 0) p.meta[blockIdx.x] = make_int4(0, 0, 0, 0);
    const int extra = share[3], total = share[4], nc = share[5], c = static_cast<int>(blockIdx.x);
    int x0 = share[9];  // cost before the walk's item
    bool ok = true;
    for (int seg = 0; wk.rem > 0 && ok; ++seg) {
      const int ob = seg & 1, run = wk.run();
      const int g0 = wk.blk * GB, ng = min(GB, p.G - g0);
      const bool starts = wk.off == 0, ends = wk.off + run == wk.n;
      ok = __all_sync(0xffffffffu, decode_wait(ctx, &bar_stat[ob], (seg >> 1) & 1, kTagDStat) &&
                                       decode_wait(ctx, &bar_o[ob], (seg >> 1) & 1, kTagDO));
      if (!ok) break;
      tc_fence_after();
      const uint32_t to = tmem + lane_off + kOCol0 + ob * C::kOCols;
      const long long row0 = static_cast<long long>(wk.b) * p.Hq + wk.h * p.G + g0;
      const int slot = 2 * c + (starts ? 1 : 0);
      const bool whole = starts && ends;
      constexpr int kH = C::kHeads;
#pragma unroll 1
      for (int gc = 0; gc < (f < D || D == 128 ? ng : 0); gc += kH) {  // d = 64: lanes from 64 on hold nothing new
        uint32_t o[C::kOParts][kH];
#pragma unroll
        for (int part = 0; part < C::kOParts; ++part) tmem_ld_n<kH>(to + part * GB + gc, o[part]);
        // Lane g < kH has head gc + g's sums.
        const float *lp = lpart + ob * 4 * GB + gc + (lane & (kH - 1));
        const float lt = (lp[0] + lp[GB]) + (lp[2 * GB] + lp[3 * GB]);
        const float mh = mstat[ob * GB + gc + (lane & (kH - 1))];
        const float mul = whole ? __fdividef(1.f, lt) : 1.f;
        float unit[kH];  // e4m3: what a code stands for
#pragma unroll
        for (int e = 0; e < kH; ++e) unit[e] = E4M3 ? vstat[ob * GB + gc + e] : 1.f;
        if ((warp & 3) == 0 && lane < kH && gc + lane < ng) {
          if (!whole)
            p.part_ml[slot * GB + gc + lane] = make_float2(mh, lt);
          else if (p.lse)
            p.lse[row0 + gc + lane] = (mh + log2f(lt)) * 0.69314718055994531f;
        }
        tmem_wait_ld();
        uint16_t *po = p.o + (row0 + gc) * D + f;
        float *pp = p.part_o + (static_cast<long long>(slot) * GB + gc) * D + f;
#pragma unroll
        for (int e = 0; e < kH; ++e) {
          float v = __uint_as_float(o[0][e]);
          if constexpr (E4M3)
            v += (__uint_as_float(o[1][e]) + __uint_as_float(o[2][e])) * kPartUnit1 + __uint_as_float(o[3][e]) * kPartUnit3;
          else if (fabsf(v) != INFINITY)  // an infinite value: the low part's product with it may be NaN
            v += __uint_as_float(o[1][e]);
          v *= __shfl_sync(0xffffffffu, mul, e);
          if constexpr (E4M3) v *= unit[e];  // apart: their product may lie below fp32's range
          if (gc + e < ng) {
            if (whole)
              po[e * D] = static_cast<uint16_t>(pack_bf16(v, 0.f));
            else
              pp[e * D] = v;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_o_empty[ob]);
      const int cost = extra + C::kTileCost * wk.n;
      if (starts && f == 0 && (p.by_item || !ends))
        decode_note(p, wk.b, wk.h, wk.blk, wk.h * p.G + g0, ends ? 0 : x0 + cost - 1, total, nc);
      if (ends) x0 += cost;
      wk.advance(p, run);
    }
    // A share without a tile may still lie inside an item: an empty part.
    if (warp == C::kEpilogue && c < nc && share[10] == share[11] && lane < GB) p.part_ml[2 * c * GB + lane] = make_float2(-INFINITY, 0.f);
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == C::kIssuer) tmem_dealloc(tmem, C::kTmemCols);
}

// Whether an entry of meta is one that fa_decode_kernel can have written for this call, with parts
// to join.  A CTA that gives up (a wait that ran out, an unusable launch) leaves entries as the
// workspace held them, and what is read and written by way of one that passes lies inside the
// parts' slots and o and lse: CTAs [c, c + parts), rows of sequence b from `row` up to the end
// of its block of at most G - row % G heads.  (What such an entry's parts hold is another matter:
// the launch has failed, and its status says so.  To look at the status word here as well took
// 2.5 us where 1500 blocks do: every warp's load went to one place of the L2.)
__host__ __device__ inline bool decode_entry_ok(int b, int row, int parts, int c, int B, int Hq) {
  return parts > 0 && parts <= kDecodeMaxCtas && c >= 0 && c <= kDecodeMaxCtas - parts && b >= 0 && b < B && row >= 0 &&
         row < Hq;
}

// Joins the parts of the item of entry blockIdx.x for query head blockIdx.y of its block: it
// starts in CTA c (its second slot) and goes on in the first slots of CTAs c + 1 ...  An empty part
// (m = -inf, O as the workspace held it) is not read into the sum; a part of weight 0 is, so that
// a NaN in it stays one.  The order of every sum is fixed by the number of parts.  Two dependent
// loads deep (which item, then its parts) and one barrier: the kernel's time is its latency.
constexpr int kJoinThreads = 256;

template <int D, int GB>
__global__ void __launch_bounds__(kJoinThreads) fa_decode_join_kernel(const __grid_constant__ DecodeParams p) {
  constexpr int kCols = D / 4, kGroups = kJoinThreads / kCols;  // four features a thread, a part a group
  __shared__ float4 part[kGroups][kCols];
  pdl_launch();
  pdl_wait();
  const int4 mt = p.meta[blockIdx.x];
  const int c = mt.w, g = static_cast<int>(blockIdx.y);
  if (!decode_entry_ok(mt.x, mt.y, mt.z, c, p.c.B, p.Hq) || mt.y % p.G + g >= p.G) return;
  const int tid = threadIdx.x, lane = tid & 31, col = tid % kCols, grp = tid / kCols;
  auto row = [&](int i) { return static_cast<long long>(i == 0 ? 2 * c + 1 : 2 * (c + i)) * GB + g; };
  auto ml_of = [&](int i) { return i < mt.z ? p.part_ml[row(i)] : make_float2(-INFINITY, 0.f); };
  auto o_of = [&](int i) {
    return i < mt.z ? *reinterpret_cast<const float4 *>(p.part_o + row(i) * D + 4 * col) : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  const float2 ml0 = ml_of(lane);
  float2 mine = ml_of(grp);
  float4 o = o_of(grp);
  // Every warp takes the parts' maximum and sum for itself.
  float M = ml0.x;
  for (int i = lane + 32; i < mt.z; i += 32) M = fmaxf(M, ml_of(i).x);
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
  float L = ml0.y * ex2(ml0.x - M);
  for (int i = lane + 32; i < mt.z; i += 32) {
    const float2 ml = ml_of(i);
    L += ml.y * ex2(ml.x - M);
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = grp; i < mt.z; i += kGroups) {
    const float w = ex2(mine.x - M);
    if (mine.x != -INFINITY) {
      acc.x += w * o.x;
      acc.y += w * o.y;
      acc.z += w * o.z;
      acc.w += w * o.w;
    }
    mine = ml_of(i + kGroups);
    o = o_of(i + kGroups);
  }
  part[grp][col] = acc;
  __syncthreads();
  if (grp != 0) return;
#pragma unroll
  for (int k = 1; k < kGroups; ++k) {
    const float4 a = part[k][col];
    acc.x += a.x;
    acc.y += a.y;
    acc.z += a.z;
    acc.w += a.w;
  }
  const long long out = static_cast<long long>(mt.x) * p.Hq + mt.y + g;
  const float inv = __fdividef(1.f, L);
  *reinterpret_cast<uint2 *>(p.o + out * D + 4 * col) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (col == 0 && p.lse) p.lse[out] = (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace fa
