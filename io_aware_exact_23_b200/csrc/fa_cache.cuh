// fa_cache.cuh -- the paged key/value cache: its device view, the kernel that
// writes new tokens into it and the kernel that reads sequences back.
//
// Both kernels move rows of d elements, one 16-byte chunk of 8 bf16 values per
// thread, and do next to no arithmetic: their floor is the bytes they move at the
// memory's rate.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "ptx.cuh"

namespace fa {

enum : int { kStatusCache = 9 };
enum : int { kKernelAppend = 6, kKernelGather = 7, kKernelDecode = 8 };

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

// Record a page id or a length out of range (the first one sticks).  Word 4 of the
// status block stays as it is: it makes a pipeline of that launch give up, and
// these kernels carry on with their other sequences.
__device__ __noinline__ void record_cache_error(int *status, int kernel, int b, int seq) {
  if (atomicCAS(status, 0, kStatusCache) == 0) {
    status[1] = kernel;
    status[2] = b;
    status[3] = static_cast<int>(blockIdx.x);
    status[5] = seq;
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

// ------------------------------------------------------------------- append
struct AppendParams {
  CacheView c;
  const uint16_t *x[2];     // k_new, v_new
  long long x_stride[2][2];  // token, head
  const int *cu_new;
  int T;
};

constexpr int kCacheThreads = 256;

// One thread per 16-byte chunk of an input row; rows (token, K or V, head), head
// fastest, so that neighbouring threads read neighbouring memory.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) fa_cache_append_kernel(const AppendParams p) {
  constexpr int kLanes = D / 8;  // threads per row
  const CacheView &c = p.c;
  const long long i = static_cast<long long>(blockIdx.x) * kCacheThreads + threadIdx.x;
  const long long vec = i / kLanes;
  const int chunk = static_cast<int>(i % kLanes);
  const long long row2 = vec / c.H;
  const int h = static_cast<int>(vec % c.H);
  const int t = static_cast<int>(row2 >> 1), which = static_cast<int>(row2 & 1);
  int b = t, pos = -1;
  bool live = t < p.T;
  if (live) {
    if (p.cu_new == nullptr) {
      pos = cache_len(c, b, kKernelAppend) - 1;
    } else {
      // The sequence whose tokens hold t: the last b with cu_new[b] <= t.
      int lo = 0, hi = c.B;  // cu_new[lo] <= t < cu_new[hi], if t is a token at all
      live = t < __ldg(p.cu_new + c.B);
      if (live) {
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
    }
    live = live && pos >= 0;
  }
  int row = 0, page = -1;
  if (live) page = cache_page(c, b, pos, row, kKernelAppend);
  live = page >= 0;
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if (live)
    w = *reinterpret_cast<const uint4 *>(p.x[which] + t * p.x_stride[which][0] + h * p.x_stride[which][1] + chunk * 8);
  const long long off = page * c.stride[which][0] + h * c.stride[which][1] + row * c.stride[which][2] + chunk * 8;
  if constexpr (!E4M3) {
    if (live) *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(c.kv[which]) + off) = w;
  } else {
    const float x[8] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y),
                        bf16_lo(w.z), bf16_hi(w.z), bf16_lo(w.w), bf16_hi(w.w)};
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(x[e]));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float f = __fdiv_rn(max_nan(m, 1e-30f), 448.f);
    if (live) {
      const uint32_t lo = pack_e4m3x4(__fdiv_rn(x[0], f), __fdiv_rn(x[1], f), __fdiv_rn(x[2], f), __fdiv_rn(x[3], f));
      const uint32_t hi = pack_e4m3x4(__fdiv_rn(x[4], f), __fdiv_rn(x[5], f), __fdiv_rn(x[6], f), __fdiv_rn(x[7], f));
      *reinterpret_cast<uint2 *>(c.kv[which] + off) = make_uint2(lo, hi);
      if (chunk == 0)
        c.scale[which][page * c.scale_stride[which][0] + h * c.scale_stride[which][1] +
                       row * c.scale_stride[which][2]] = f;
    }
  }
}

// ------------------------------------------------------------------- gather
struct GatherParams {
  CacheView c;
  uint16_t *out[2];  // k_out, v_out [B, H * rep, N, d], or null
  int rep, N;
};

// One thread per 16-byte chunk of an output row of the cache's heads; the value is
// read once and stored rep times.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheThreads) fa_cache_gather_kernel(const GatherParams p) {
  constexpr int kLanes = D / 8;
  const CacheView &c = p.c;
  const int which = blockIdx.y;
  if (p.out[which] == nullptr) return;
  const long long i = static_cast<long long>(blockIdx.x) * kCacheThreads + threadIdx.x;
  const int chunk = static_cast<int>(i % kLanes);
  const long long r = i / kLanes;
  const int n = static_cast<int>(r % p.N);
  const long long bh = r / p.N;
  if (bh >= static_cast<long long>(c.B) * c.H) return;
  const int b = static_cast<int>(bh / c.H), h = static_cast<int>(bh % c.H);
  uint4 w = make_uint4(0u, 0u, 0u, 0u);
  if (n < cache_len(c, b, kKernelGather)) {
    int row = 0;
    const int page = cache_page(c, b, n, row, kKernelGather);
    if (page >= 0) {
      const long long off = page * c.stride[which][0] + h * c.stride[which][1] + row * c.stride[which][2] + chunk * 8;
      if constexpr (!E4M3) {
        w = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(c.kv[which]) + off);
      } else {
        const float f = c.scale[which][page * c.scale_stride[which][0] + h * c.scale_stride[which][1] +
                                       row * c.scale_stride[which][2]];
        const uint2 q = *reinterpret_cast<const uint2 *>(c.kv[which] + off);
        const float2 a0 = e4m3x2_to_float2(static_cast<uint16_t>(q.x)), a1 = e4m3x2_to_float2(static_cast<uint16_t>(q.x >> 16));
        const float2 a2 = e4m3x2_to_float2(static_cast<uint16_t>(q.y)), a3 = e4m3x2_to_float2(static_cast<uint16_t>(q.y >> 16));
        w = make_uint4(pack_bf16(a0.x * f, a0.y * f), pack_bf16(a1.x * f, a1.y * f), pack_bf16(a2.x * f, a2.y * f),
                       pack_bf16(a3.x * f, a3.y * f));
      }
    }
  }
  uint16_t *out = p.out[which] + (bh * p.rep * p.N + n) * D + chunk * 8;
  for (int k = 0; k < p.rep; ++k, out += static_cast<long long>(p.N) * D) *reinterpret_cast<uint4 *>(out) = w;
}

}  // namespace fa
