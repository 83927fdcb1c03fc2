// fa_cache_api.cuh -- the C ABI of the paged key/value cache (declared in
// include/fa_cache.h): argument validation and the launches of the append, gather
// and decode kernels.  Part of fa_api.cu, whose device state and checks it uses.
#pragma once

#include "fa_cache.cuh"
#include "fa_cache.h"
#include "fa_decode.cuh"

namespace {

bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// One of K and V: a stride matters only along an axis of more than one element,
// where it holds at least a row and keeps every row 16-byte aligned.
int check_strides(const long long *stride, const int *extent, int d, int elem_bytes) {
  for (int a = 0; a < 3; ++a) {
    if (extent[a] == 1) continue;
    if (stride[a] < d || stride[a] >= (1ll << 39)) return FA_ERR_UNSUPPORTED;
    if (stride[a] * elem_bytes % 16 != 0) return FA_ERR_MISALIGNED;
  }
  return FA_OK;
}

// Checks of the cache that all entry points share (no CUDA calls).
int check_cache(const fa_paged_cache *c) {
  if (!c || !c->k || !c->v || !c->block_table || !c->seq_lens) return FA_ERR_INVALID_ARG;
  if (c->type != FA_CACHE_BF16 && c->type != FA_CACHE_E4M3) return FA_ERR_INVALID_ARG;
  if (c->type == FA_CACHE_E4M3 && (!c->k_scale || !c->v_scale)) return FA_ERR_INVALID_ARG;
  if (c->B < 1 || c->H < 1 || c->num_pages < 1 || c->max_pages < 1 || c->page_size < 1) return FA_ERR_INVALID_ARG;
  if (c->block_table_stride < c->max_pages && c->B > 1) return FA_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED;
  const int ps = c->page_size;
  if (ps != 16 && ps != 32 && ps != 64 && ps % 128 != 0) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->max_pages) * ps >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->block_table) || !aligned4(c->seq_lens))
    return FA_ERR_MISALIGNED;
  const int extent[3] = {c->num_pages, c->H, ps};
  const int eb = c->type == FA_CACHE_BF16 ? 2 : 1;
  int st = check_strides(c->k_stride, extent, c->d, eb);
  if (st == FA_OK) st = check_strides(c->v_stride, extent, c->d, eb);
  if (st != FA_OK) return st;
  if (c->type == FA_CACHE_E4M3) {
    if (!aligned4(c->k_scale) || !aligned4(c->v_scale)) return FA_ERR_MISALIGNED;
    for (int a = 0; a < 3; ++a)
      if (extent[a] > 1 && (c->k_scale_stride[a] < 1 || c->v_scale_stride[a] < 1 ||
                            c->k_scale_stride[a] >= (1ll << 39) || c->v_scale_stride[a] >= (1ll << 39)))
        return FA_ERR_UNSUPPORTED;
  }
  return FA_OK;
}

int make_view(const fa_paged_cache *c, fa::CacheView *v, DeviceState **ds) {
  const int st = device_state(ds, nullptr);
  if (st != FA_OK) return st;
  v->kv[0] = static_cast<uint8_t *>(c->k);
  v->kv[1] = static_cast<uint8_t *>(c->v);
  v->scale[0] = c->k_scale;
  v->scale[1] = c->v_scale;
  for (int a = 0; a < 3; ++a) {
    v->stride[0][a] = c->k_stride[a];
    v->stride[1][a] = c->v_stride[a];
    v->scale_stride[0][a] = c->k_scale_stride[a];
    v->scale_stride[1][a] = c->v_scale_stride[a];
  }
  v->block_table = c->block_table;
  v->seq_lens = c->seq_lens;
  v->bt_stride = c->block_table_stride;
  v->num_pages = c->num_pages;
  v->H = c->H;
  v->page_size = c->page_size;
  v->B = c->B;
  v->max_pages = c->max_pages;
  v->cap = c->max_pages * c->page_size;
  v->page_shift = -1;
  for (int s = 4; s < 31; ++s)
    if (c->page_size == (1 << s)) v->page_shift = s;
  v->page_magic = v->page_shift >= 0 ? 0 : ~0ull / static_cast<unsigned>(c->page_size / 128) + 1;
  v->status = (*ds)->status;
  v->seq = next_seq();
  return FA_OK;
}

// A launch that may begin while the stream's previous kernel ends (pdl_wait in the kernel).
template <class... Formal, class... Actual>
cudaError_t launch_early(void (*kernel)(Formal...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                         const Actual &...args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Rows of a warp of the append and gather kernels: `many`, so that most lanes find a row's
// address, but one round of loads (1024 / d) where `many` would leave fewer than 16 warps per SM.
// `many` is two rounds (300 positions x 8 heads x 128 read back four times, two rounds / one:
// 3.9 / 3.6 us), and a whole warp's rows for appending e4m3, whose rows need most instructions:
// 6000, 8275, 12000, 24000 and 60000 tokens x 8 heads x 128 with 16 / 32 rows take 10.9 / 11.8,
// 14.1 / 13.0, 17.7 / 18.1, 31.8 / 30.4 and 72.6 / 67.9 us (bf16: 33.1 / 34.2 us at 24000).
int rows_per_warp(long long rows, int d, int many, int num_sms) {
  return rows >= 16ll * many * num_sms ? many : 1024 / d;
}

unsigned blocks_for(long long rows, int per_warp) {
  const long long warps = (rows + per_warp - 1) / per_warp;
  return static_cast<unsigned>((warps + fa::kCacheWarps - 1) / fa::kCacheWarps);
}

// K or V as the 4-D tensor (feature, row of the page, head, page) that the decode kernel
// loads 128-byte (e4m3, d = 64: 64-byte) wide boxes of; pages past the last read as zeros.
int encode_cache(CUtensorMap *m, const void *ptr, const fa_paged_cache *c, const long long *stride) {
  EncodeTiledFn enc = get_encode_fn();
  if (!enc) return FA_ERR_CUDA;
  const int eb = c->type == FA_CACHE_BF16 ? 2 : 1;
  const int row_bytes = c->d * eb, box_bytes = row_bytes < 128 ? row_bytes : 128;
  // A stride along an axis of one element is never used, but has to be a valid one.
  auto bytes = [&](int a, int extent) {
    return static_cast<cuuint64_t>(extent > 1 ? stride[a] * eb : static_cast<long long>(row_bytes));
  };
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c->d), static_cast<cuuint64_t>(c->page_size),
                              static_cast<cuuint64_t>(c->H), static_cast<cuuint64_t>(c->num_pages)};
  const cuuint64_t strides[3] = {bytes(2, c->page_size), bytes(1, c->H), bytes(0, c->num_pages)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(box_bytes / eb),
                             static_cast<cuuint32_t>(c->page_size < 128 ? c->page_size : 128), 1u, 1u};
  const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  const CUresult r = enc(m, eb == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
                         const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// Query heads per block of the decode kernel: the smallest of its instances that holds G.
int decode_block(int G) { return G <= 2 ? 2 : G <= 4 ? 4 : G <= 8 ? 8 : G <= 16 ? 16 : 32; }

// Workspace: meta, then (m, l) and O of two parts per CTA.
size_t decode_ml_offset() { return fa::kDecodeMaxCtas * sizeof(int4); }
size_t decode_o_offset(int gb) { return decode_ml_offset() + 2ull * fa::kDecodeMaxCtas * gb * sizeof(float2); }
size_t decode_bytes(int gb, int d) { return decode_o_offset(gb) + 2ull * fa::kDecodeMaxCtas * gb * d * sizeof(float); }

template <int D, bool E4M3, int GB>
cudaError_t launch_decode(const CUtensorMap &tk, const CUtensorMap &tv, fa::DecodeParams p, int num_sms, long long most,
                          cudaStream_t stream) {
  using C = fa::DecodeCfg<D, E4M3, GB>;
  // As many CTAs as are resident at a time, or one per tile if there can be no more.
  long long ctas = static_cast<long long>(num_sms) * C::kCtas;
  if (ctas > fa::kDecodeMaxCtas) ctas = fa::kDecodeMaxCtas;
  const unsigned grid = static_cast<unsigned>(ctas < most ? ctas : most);
  static std::atomic<unsigned long long> ready{0};  // devices whose kernel has its attribute
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!((ready.load() >> dev) & 1ull)) {
    e = cudaFuncSetAttribute(fa::fa_decode_kernel<D, E4M3, GB>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(1ull << dev);
  }
  const long long items = static_cast<long long>(p.c.B) * p.c.H * p.nblk;
  p.by_item = items < grid;
  e = launch_early(fa::fa_decode_kernel<D, E4M3, GB>, dim3(grid), C::kThreads, C::kSmemBytes, stream, tk, tv, p);
  if (e != cudaSuccess || grid == 1) return e;  // one CTA leaves no parts
  return launch_early(fa::fa_decode_join_kernel<D, GB>, dim3(p.by_item ? static_cast<unsigned>(items) : grid, static_cast<unsigned>(p.G < GB ? p.G : GB)),
                      fa::kJoinThreads, 0, stream, p);
}

template <int D, bool E4M3>
cudaError_t launch_decode_block(int gb, const CUtensorMap &tk, const CUtensorMap &tv, const fa::DecodeParams &p,
                                int num_sms, long long most, cudaStream_t s) {
  return gb == 2    ? launch_decode<D, E4M3, 2>(tk, tv, p, num_sms, most, s)
         : gb == 4  ? launch_decode<D, E4M3, 4>(tk, tv, p, num_sms, most, s)
         : gb == 8  ? launch_decode<D, E4M3, 8>(tk, tv, p, num_sms, most, s)
         : gb == 16 ? launch_decode<D, E4M3, 16>(tk, tv, p, num_sms, most, s)
                    : launch_decode<D, E4M3, 32>(tk, tv, p, num_sms, most, s);
}

}  // namespace

extern "C" {

int fa_cache_append(const fa_paged_cache *cache, const void *k_new, const void *v_new, const long long *k_new_stride,
                    const long long *v_new_stride, int T, const int *cu_new, void *stream) {
  int st = check_cache(cache);
  if (st != FA_OK) return st;
  if (!k_new_stride || !v_new_stride || T < 0) return FA_ERR_INVALID_ARG;
  if (!cu_new && T != cache->B) return FA_ERR_INVALID_ARG;
  if (T == 0) return FA_OK;
  if (!k_new || !v_new) return FA_ERR_INVALID_ARG;
  if (!aligned16(k_new) || !aligned16(v_new) || !aligned4(cu_new)) return FA_ERR_MISALIGNED;
  const long long total = 2ll * T * cache->H;
  if (total >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  const long long *strides[2] = {k_new_stride, v_new_stride};
  const int extent[2] = {T, cache->H};
  fa::AppendParams p;
  for (int w = 0; w < 2; ++w)
    for (int a = 0; a < 2; ++a) {
      const long long s = strides[w][a];
      if (extent[a] > 1 && (s < 0 || s >= (1ll << 39))) return FA_ERR_UNSUPPORTED;
      if (extent[a] > 1 && s % 8 != 0) return FA_ERR_MISALIGNED;
      p.x_stride[w][a] = s;
    }
  DeviceState *ds = nullptr;
  st = make_view(cache, &p.c, &ds);
  if (st != FA_OK) return st;
  p.x[0] = static_cast<const uint16_t *>(k_new);
  p.x[1] = static_cast<const uint16_t *>(v_new);
  p.cu_new = cu_new;
  p.T = T;
  const bool e4m3 = cache->type == FA_CACHE_E4M3;
  p.rows = rows_per_warp(total, cache->d, e4m3 ? 32 : 2048 / cache->d, ds->num_sms);
  const unsigned grid = blocks_for(total, p.rows);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const auto kernel = cache->d == 64 ? (e4m3 ? fa::fa_cache_append_kernel<64, true> : fa::fa_cache_append_kernel<64, false>)
                                     : (e4m3 ? fa::fa_cache_append_kernel<128, true> : fa::fa_cache_append_kernel<128, false>);
  const cudaError_t e = launch_early(kernel, dim3(grid), fa::kCacheThreads, 0, s, p);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

int fa_cache_gather(const fa_paged_cache *cache, void *k_out, void *v_out, int rep, int N, void *stream) {
  int st = check_cache(cache);
  if (st != FA_OK) return st;
  if ((!k_out && !v_out) || rep < 1 || N < 1) return FA_ERR_INVALID_ARG;
  const long double elems = static_cast<long double>(cache->B) * cache->H * rep * N * cache->d;
  if (elems >= 2147483648.0L) return FA_ERR_UNSUPPORTED;
  if (!aligned16(k_out) || !aligned16(v_out)) return FA_ERR_MISALIGNED;
  fa::GatherParams p;
  DeviceState *ds = nullptr;
  st = make_view(cache, &p.c, &ds);
  if (st != FA_OK) return st;
  p.out[0] = static_cast<uint16_t *>(k_out);
  p.out[1] = static_cast<uint16_t *>(v_out);
  p.rep = rep;
  p.N = N;
  const long long heads = static_cast<long long>(cache->B) * cache->H;
  p.rows = rows_per_warp(heads * N, cache->d, 2048 / cache->d, ds->num_sms);
  p.parts = (N - 1) / p.rows + 1;
  const dim3 grid(blocks_for(heads * p.parts, 1), 2);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache->type == FA_CACHE_E4M3;
  const auto kernel = cache->d == 64 ? (e4m3 ? fa::fa_cache_gather_kernel<64, true> : fa::fa_cache_gather_kernel<64, false>)
                                     : (e4m3 ? fa::fa_cache_gather_kernel<128, true> : fa::fa_cache_gather_kernel<128, false>);
  const cudaError_t e = launch_early(kernel, grid, fa::kCacheThreads, 0, s, p);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_decode_workspace_bytes(int B, int Hq, int H, int d) {
  if (B < 1 || H < 1 || Hq < H || Hq % H != 0 || (d != 64 && d != 128)) return 0;
  return decode_bytes(decode_block(Hq / H), d);
}

int fa_decode(const fa_paged_cache *cache, const void *q, void *o, float *lse, int Hq, float scale, int window,
              void *workspace, size_t workspace_bytes, void *stream) {
  int st = check_cache(cache);
  if (st != FA_OK) return st;
  if (!q || !o || Hq < 1 || Hq % cache->H != 0 || window < 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(cache->B) * Hq * cache->d >= (1ll << 31)) return FA_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(o) || !aligned4(lse)) return FA_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < fa_decode_workspace_bytes(cache->B, Hq, cache->H, cache->d))
    return FA_ERR_WORKSPACE;
  if (!aligned16(workspace)) return FA_ERR_MISALIGNED;
  // The kernel counts the cost of tiles of 128 positions, over all sequences and heads, in 31 bits.
  const int G = Hq / cache->H, gb = decode_block(G), nblk = (G + gb - 1) / gb;
  const long long item_tiles = (static_cast<long long>(cache->max_pages) * cache->page_size + 127) / 128;
  const long double most = static_cast<long double>(cache->B) * cache->H * nblk * item_tiles;
  if (most * 6 >= 2147483648.0L) return FA_ERR_UNSUPPORTED;  // kItemCost + kTileCost = 6
  fa::DecodeParams p;
  DeviceState *ds = nullptr;
  st = make_view(cache, &p.c, &ds);
  if (st != FA_OK) return st;
  p.q = static_cast<const uint16_t *>(q);
  p.o = static_cast<uint16_t *>(o);
  p.lse = lse;
  p.Hq = Hq;
  p.G = G;
  p.nblk = nblk;
  p.window = window;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.vec_scales = 0;
  if (cache->type == FA_CACHE_E4M3) {
    const long long *ks = cache->k_scale_stride, *vs = cache->v_scale_stride;
    const int extent[2] = {cache->num_pages, cache->H};
    bool vec = ks[2] == 1 && vs[2] == 1 && aligned16(cache->k_scale) && aligned16(cache->v_scale);
    for (int a = 0; a < 2; ++a) vec = vec && (extent[a] == 1 || (ks[a] % 4 == 0 && vs[a] % 4 == 0));
    p.vec_scales = vec;
  }
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.meta = reinterpret_cast<int4 *>(ws);
  p.part_ml = reinterpret_cast<float2 *>(ws + decode_ml_offset());
  p.part_o = reinterpret_cast<float *>(ws + decode_o_offset(gb));
  CUtensorMap tk, tv;
  if (encode_cache(&tk, cache->k, cache, cache->k_stride) || encode_cache(&tv, cache->v, cache, cache->v_stride))
    return FA_ERR_CUDA;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool e4m3 = cache->type == FA_CACHE_E4M3;
  cudaError_t e;
  const int n = ds->num_sms;
  const long long tiles = static_cast<long long>(most);
  if (cache->d == 64)
    e = e4m3 ? launch_decode_block<64, true>(gb, tk, tv, p, n, tiles, s)
             : launch_decode_block<64, false>(gb, tk, tv, p, n, tiles, s);
  else
    e = e4m3 ? launch_decode_block<128, true>(gb, tk, tv, p, n, tiles, s)
             : launch_decode_block<128, false>(gb, tk, tv, p, n, tiles, s);
  if (e != cudaSuccess) cudaGetLastError();
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
