// fa_cache.cuh -- the paged key/value cache: its device view, the kernel that
// writes new tokens into it and the kernel that reads sequences back.
//
// Both kernels move rows of d elements, in 16-byte chunks of 8 bf16 values
// a thread, and do next to no arithmetic: their floor is the bytes they move at the
// memory's rate.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "ptx.cuh"

namespace fa {

enum : int { kKernelAppend = 6, kKernelGather = 7, kKernelDecode = 8 };

// Programmatic dependent launch.  The cache's kernels are launched so that they may start while
// the stream's previous kernel ends: a kernel lets the next one come at once (pdl_launch) and
// touches no memory that is not its own before the previous one is complete (pdl_wait).
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// The cache as the kernels see it (include/fa_cache.h describes the fields).
struct CacheView {
  uint8_t *kv[2];        // K, V base addresses
  float *scale[2];       // K, V factors (e4m3)
  long long stride[2][3];        // page, head, token, in elements
  long long scale_stride[2][3];  // page, head, token, in floats
  const int *block_table;
  const int *seq_lens;
  long long bt_stride;
  int num_pages, H, page_size, B, max_pages;
  int cap;         // max_pages * page_size: the longest sequence
  int page_shift;  // log2(page_size), or -1: then page_size is a multiple of 128
  unsigned long long page_magic;  // ceil(2^64 / (page_size / 128)), where page_shift is -1
  int *status;
  int seq;
};

// Record a page id or a length out of range (the first one sticks): words 5 to 7 of the status
// block, launch number, sequence, and block and kernel.  Words 0 to 4 are those of failures that
// spoil more than a sequence (ptx.cuh), which must not be hidden by this one; word 4 also makes
// a pipeline of that launch give up, and these kernels carry on with their other sequences.
__device__ __noinline__ void record_cache_error(int *status, int kernel, int b, int seq) {
  if (atomicCAS(status + 5, 0, seq) == 0) {
    status[6] = b;
    status[7] = static_cast<int>(blockIdx.x) << 4 | kernel;
  }
}

// Sequence b's length, clamped to what its row of the block table can hold.
__device__ __forceinline__ int cache_len(const CacheView &c, int b, int kernel) {
  const int n = __ldg(c.seq_lens + b);
  if (n < 0 || n > c.cap) {
    record_cache_error(c.status, kernel, b, c.seq);
    return n < 0 ? 0 : c.cap;
  }
  return n;
}

// The index of position `pos`'s page in its sequence: pos / page_size.  floor(t / k) is the
// high word of t * ceil(2^64 / k) for every t < 2^32.
__device__ __forceinline__ int cache_page_index(const CacheView &c, int pos) {
  if (c.page_shift >= 0) return pos >> c.page_shift;
  return static_cast<int>(__umul64hi(static_cast<unsigned long long>(pos >> 7), c.page_magic));
}

// Page and row of position `pos` of sequence b; -1 (and a record) for a bad page id.
__device__ __forceinline__ int cache_page(const CacheView &c, int b, int pos, int &row, int kernel) {
  const int pi = cache_page_index(c, pos);
  row = pos - pi * c.page_size;
  const int page = __ldg(c.block_table + b * c.bt_stride + pi);
  if (static_cast<unsigned>(page) >= static_cast<unsigned>(c.num_pages)) {
    record_cache_error(c.status, kernel, b, c.seq);
    return -1;
  }
  return page;
}

// max that keeps a NaN, so that a row with a NaN gets a NaN factor.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two e4m3 codes -> two fp32 values (exact).
__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3);
  return __half22float2(__half2(h));
}

// Both kernels below give a warp `rows` (at most 32) rows of d elements.  Lane i first finds
// where row i lies (sequence, page, strides: some hundred cycles of dependent loads and 64-bit
// arithmetic, once per row), then the warp walks over the rows, kLanes lanes to a row with 16
// bytes of bf16 (append: twice 16) each, taking the addresses from the lanes that know them.  (With every lane
// finding its own piece's address, 145 to 245 instructions went into a piece, and the two
// cases given below took 25 and 90 us.)
constexpr int kCacheThreads = 256;
constexpr int kCacheWarps = kCacheThreads / 32;

template <class T>
__device__ __forceinline__ T *shfl_ptr(T *p, int lane) {
  return reinterpret_cast<T *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), lane));
}

// ------------------------------------------------------------------- append
struct AppendParams {
  CacheView c;
  const uint16_t *x[2];      // k_new, v_new
  long long x_stride[2][2];  // token, head
  const int *cu_new;
  int T;
  int rows;  // per warp
};

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// q = x / f for a pair, correctly rounded.  Markstein's division (IBM J. Res. Dev. 34(1),
// 1990): with r = 1 / f correctly rounded and y = x r, the remainder x - y f is exact in a
// fused multiply-add, and y + (x - y f) r rounds to the quotient.  Only quotients that e4m3
// can tell from 0 matter (2^-11 and up), whose remainders stay representable for f in
// [2^-80, 2^100] (and of zeros always); other rows take the division itself.
__device__ __forceinline__ uint64_t divide2(uint64_t x, uint64_t f, uint64_t r) {
  const uint64_t y = mul2(x, r);
  return ffma2(ffma2(y ^ 0x8000000080000000ull, f, x), r, y);
}

// Rows are (token, K or V, head), head fastest.  Bound by its instructions: 8275 tokens x 8
// heads x 128 as e4m3 take 13.0 us, 51 MB at 3.9 TB/s, and 60000 tokens 67.9 us, 5.5 TB/s (with
// one piece a lane, twice the lanes to a row and so twice the shuffles: 15.0 and 78.6 us; five
// resident blocks, with fewer registers: 15.2 us; the next pass's loads ahead of this one's
// division: 14.8 us, for want of registers).
template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads, 4) fa_cache_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int kLanes = D / 16;        // lanes per row, two 16-byte pieces each
  constexpr int kAtOnce = 32 / kLanes;  // rows per pass
  constexpr int kBatch = 2;             // passes in flight
  pdl_launch();
  pdl_wait();
  const CacheView &c = p.c;
  const int lane = threadIdx.x & 31;
  const long long total = 2ll * p.T * c.H;
  const long long r0 = (static_cast<long long>(blockIdx.x) * kCacheWarps + (threadIdx.x >> 5)) * p.rows;
  if (r0 >= total) return;
  const int rows = static_cast<int>(total - r0 < p.rows ? total - r0 : p.rows);
  const uint16_t *src = nullptr;
  uint8_t *dst = nullptr;
  float *fdst = nullptr;
  if (lane < rows) {
    const unsigned r = static_cast<unsigned>(r0) + lane, vec = r / static_cast<unsigned>(c.H);
    const int h = static_cast<int>(r - vec * c.H), t = static_cast<int>(vec >> 1), which = static_cast<int>(vec & 1);
    int b = t, pos = -1;
    if (p.cu_new == nullptr) {
      pos = cache_len(c, b, kKernelAppend) - 1;
    } else if (t < __ldg(p.cu_new + c.B)) {
      int lo = 0, hi = c.B;  // cu_new[lo] <= t < cu_new[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu_new + mid) <= t)
          lo = mid;
        else
          hi = mid;
      }
      b = lo;
      pos = cache_len(c, b, kKernelAppend) - (__ldg(p.cu_new + b + 1) - t);
    }
    int row = 0;
    const int page = pos >= 0 ? cache_page(c, b, pos, row, kKernelAppend) : -1;
    if (page >= 0) {
      src = p.x[which] + t * p.x_stride[which][0] + h * p.x_stride[which][1];
      const long long off = page * c.stride[which][0] + h * c.stride[which][1] + row * c.stride[which][2];
      dst = c.kv[which] + off * (E4M3 ? 1 : 2);
      if constexpr (E4M3)
        fdst = c.scale[which] + (page * c.scale_stride[which][0] + h * c.scale_stride[which][1] +
                                 row * c.scale_stride[which][2]);
    }
  }
  const int chunk = lane % kLanes, sub = lane / kLanes;  // and chunk + kLanes
  float mine = 0.f;  // lane i: row i's factor
  for (int q0 = 0; q0 < rows; q0 += kBatch * kAtOnce) {
    uint4 w[kBatch][2];
    uint8_t *to[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int q = q0 + k * kAtOnce + sub;
      const uint16_t *from = shfl_ptr(src, q & 31);
      to[k] = shfl_ptr(dst, q & 31);
      if (q >= rows) to[k] = nullptr;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        w[k][i] = make_uint4(0u, 0u, 0u, 0u);
        if (to[k]) w[k][i] = __ldg(reinterpret_cast<const uint4 *>(from) + chunk + i * kLanes);
      }
    }
    if constexpr (!E4M3) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (to[k])
#pragma unroll
          for (int i = 0; i < 2; ++i) reinterpret_cast<uint4 *>(to[k])[chunk + i * kLanes] = w[k][i];
    } else {
      // The rows' largest magnitudes, as bf16 bits (a NaN is above all), brought to the rows'
      // lanes: lane q - q0 makes the factor of row q and its reciprocal, once for the row.
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        uint32_t m2 = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(w[k][i].x & 0x7fff7fffu, w[k][i].y & 0x7fff7fffu),
                                     __vmaxu2(w[k][i].z & 0x7fff7fffu, w[k][i].w & 0x7fff7fffu)));
        m2 = max(m2 >> 16, m2 & 0xffffu);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) m2 = max(m2, __shfl_xor_sync(0xffffffffu, m2, o));
        const uint32_t its = __shfl_sync(0xffffffffu, m2, (lane % kAtOnce) * kLanes);
        if (lane / kAtOnce == k) top = its;
      }
      const float f = __fdiv_rn(max_nan(__uint_as_float(top << 16), 1e-30f), 448.f);
      const float r = (f >= 0x1p-80f && f <= 0x1p100f) || top == 0 ? __frcp_rn(f) : 0.f;  // 0: divide
      const float back = __shfl_sync(0xffffffffu, f, (lane - q0) & 31);
      if (lane >= q0 && lane < q0 + kBatch * kAtOnce) mine = back;
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, k * kAtOnce + sub), rk = __shfl_sync(0xffffffffu, r, k * kAtOnce + sub);
        const uint64_t f2 = f2pack(fk, fk), r2 = f2pack(rk, rk);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t words[4] = {w[k][i].x, w[k][i].y, w[k][i].z, w[k][i].w};
          float a[8];
          if (rk != 0.f) {
#pragma unroll
            for (int e = 0; e < 4; ++e) f2unpack(divide2(f2pack(bf16_lo(words[e]), bf16_hi(words[e])), f2, r2), a[2 * e], a[2 * e + 1]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              a[2 * e] = __fdiv_rn(bf16_lo(words[e]), fk);
              a[2 * e + 1] = __fdiv_rn(bf16_hi(words[e]), fk);
            }
          }
          if (to[k])
            reinterpret_cast<uint2 *>(to[k])[chunk + i * kLanes] =
                make_uint2(pack_e4m3x4(a[0], a[1], a[2], a[3]), pack_e4m3x4(a[4], a[5], a[6], a[7]));
        }
      }
    }
  }
  if (E4M3 && fdst) *fdst = mine;
}

// ------------------------------------------------------------------- gather
struct GatherParams {
  CacheView c;
  uint16_t *out[2];  // k_out, v_out [B, H * rep, N, d], or null
  int rep, N;
  int rows, parts;  // rows per warp, and warps per sequence and head
};

// A warp writes the rows [part * rows, ...) of one (sequence, cache head, K or V); heads are
// the warps' fastest index: the heads of a token may be neighbours in the cache.  A row is
// read once and stored rep times.  Bound by the stores: 4 x 4096 positions x 8 heads x 128 of
// bf16, each stored four times, take 57.3 us (336 MB at 5.9 TB/s), 32 ragged e4m3 sequences x
// 16 heads x 64 56.2 us (332 MB; with six resident blocks 58.8 us, for bf16 with seven 58.5 us).
template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads, E4M3 ? 7 : 6) fa_cache_gather_kernel(const __grid_constant__ GatherParams p) {
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kBatch = 4;
  pdl_launch();
  pdl_wait();
  const CacheView &c = p.c;
  const int which = blockIdx.y, lane = threadIdx.x & 31;
  uint16_t *out = p.out[which];
  const unsigned unit = blockIdx.x * kCacheWarps + (threadIdx.x >> 5);
  if (out == nullptr || unit >= static_cast<unsigned>(c.B) * c.H * p.parts) return;
  const unsigned run = unit / static_cast<unsigned>(c.H);
  const int h = static_cast<int>(unit - run * c.H), b = static_cast<int>(run / static_cast<unsigned>(p.parts));
  const int n0 = static_cast<int>(run - static_cast<unsigned>(b) * p.parts) * p.rows;
  const int rows = min(p.rows, p.N - n0);
  // Lane i's row; its page id is read beside the length it depends on (the table has it in any case).
  const uint8_t *src = nullptr;
  float f = 0.f;
  {
    const int n = n0 + lane, pi = cache_page_index(c, n);
    const int page = lane < rows && n < c.cap ? __ldg(c.block_table + b * c.bt_stride + pi) : -1;
    if (lane < rows && n < cache_len(c, b, kKernelGather)) {
      if (static_cast<unsigned>(page) >= static_cast<unsigned>(c.num_pages)) {
        record_cache_error(c.status, kKernelGather, b, c.seq);
      } else {
        const int row = n - pi * c.page_size;
        src = c.kv[which] + (page * c.stride[which][0] + h * c.stride[which][1] + row * c.stride[which][2]) * (E4M3 ? 1 : 2);
        if constexpr (E4M3)
          f = __ldg(c.scale[which] + (page * c.scale_stride[which][0] + h * c.scale_stride[which][1] +
                                      row * c.scale_stride[which][2]));
      }
    }
  }
  const int chunk = lane % kLanes, sub = lane / kLanes;
  out += ((static_cast<long long>(b) * c.H + h) * p.rep * p.N + n0) * D;
  const long long next = static_cast<long long>(p.N) * D;  // to the same row of the next repeat
  for (int q0 = 0; q0 < rows; q0 += kBatch * kAtOnce) {
    uint4 w[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const uint8_t *from = shfl_ptr(src, (q0 + k * kAtOnce + sub) & 31);
      w[k] = make_uint4(0u, 0u, 0u, 0u);
      if (from && q0 + k * kAtOnce + sub < rows) {
        if constexpr (!E4M3) {
          w[k] = __ldg(reinterpret_cast<const uint4 *>(from) + chunk);
        } else {
          const uint2 codes = __ldg(reinterpret_cast<const uint2 *>(from) + chunk);
          w[k].x = codes.x;
          w[k].y = codes.y;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int q = q0 + k * kAtOnce + sub;
      if constexpr (E4M3) {
        // Rows behind a sequence's end are code 0 times factor 0; of any other row every code counts,
        // zeros too: the factor may be an infinity or NaN, and a zero has a sign.
        const float s = __shfl_sync(0xffffffffu, f, q & 31);
        const uint64_t s2 = f2pack(s, s);
        const uint32_t codes[2] = {w[k].x, w[k].y};
        uint32_t r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = e4m3x2_to_float2(static_cast<uint16_t>(codes[e >> 1] >> (16 * (e & 1))));
          float x, y;
          f2unpack(mul2(f2pack(a.x, a.y), s2), x, y);
          r[e] = pack_bf16(x, y);
        }
        w[k] = make_uint4(r[0], r[1], r[2], r[3]);
      }
      if (q < rows) {
        uint16_t *at = out + q * D + chunk * 8;
        for (int r = 0; r < p.rep; ++r, at += next) *reinterpret_cast<uint4 *>(at) = w[k];
      }
    }
  }
}

}  // namespace fa
