// fa_decode.cuh -- attention of one new token per sequence over the paged cache.
#pragma once

#include <cstdint>

#include "fa_cache.cuh"
#include "ptx.cuh"

namespace fa {

struct DecodeParams {
  CacheView c;
  const uint16_t *q;  // [B, Hq, d]
  uint16_t *o;        // [B, Hq, d]
  float *lse;         // [B, Hq] or null
  int Hq, G;          // query heads, and query heads per cache head
  int window;         // 0: all positions
  float scale_log2;   // scale * log2(e)
};

constexpr int kDecodeThreads = 256;

// One block per (query head, sequence); warp w takes keys w, w + 8, ... with the
// running maximum and sum of its keys, and the warps' parts are joined at the end.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kDecodeThreads) fa_decode_kernel(const DecodeParams p) {
  constexpr int kPer = D / 32;
  constexpr int kWarps = kDecodeThreads / 32;
  const CacheView &c = p.c;
  const int hq = blockIdx.x, b = blockIdx.y, h = hq / p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  const int len = cache_len(c, b, kKernelDecode);
  const int first = p.window > 0 ? max(0, len - p.window) : 0;
  float q[kPer], o[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    q[e] = bf16_lo(p.q[(static_cast<long long>(b) * p.Hq + hq) * D + lane * kPer + e]) * p.scale_log2;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = first + warp; j < len; j += kWarps) {
    int row = 0;
    const int page = cache_page(c, b, j, row, kKernelDecode);
    if (page < 0) continue;
    float kv[2][kPer];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const long long off = page * c.stride[w][0] + h * c.stride[w][1] + row * c.stride[w][2] + lane * kPer;
      float f = 1.f;
      if (E4M3)
        f = c.scale[w][page * c.scale_stride[w][0] + h * c.scale_stride[w][1] + row * c.scale_stride[w][2]];
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        kv[w][e] = E4M3 ? e4m3x2_to_float2(c.kv[w][off + e]).x * f
                        : bf16_lo(reinterpret_cast<const uint16_t *>(c.kv[w])[off + e]);
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kPer; ++e) s += q[e] * kv[0][e];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s);
    const float a = m == -INFINITY ? 0.f : ex2(m - mn), e1 = ex2(s - mn);
    l = l * a + e1;
#pragma unroll
    for (int e = 0; e < kPer; ++e) o[e] = o[e] * a + e1 * kv[1][e];
    m = mn;
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) so[warp][lane * kPer + e] = o[e];
  __syncthreads();
  float M = -INFINITY;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm[w]);
  float L = 0.f, O = 0.f;
  for (int w = 0; w < kWarps; ++w) {
    const float a = sm[w] == -INFINITY ? 0.f : ex2(sm[w] - M);
    L += sl[w] * a;
    if (threadIdx.x < D) O += so[w][threadIdx.x] * a;
  }
  if (threadIdx.x < D) {
    const float v = len == 0 ? 0.f : O / L;
    p.o[(static_cast<long long>(b) * p.Hq + hq) * D + threadIdx.x] = static_cast<uint16_t>(pack_bf16(v, 0.f));
  }
  if (threadIdx.x == 0 && p.lse) p.lse[static_cast<long long>(b) * p.Hq + hq] = (M + log2f(L)) * 0.69314718055994531f;
}

}  // namespace fa
