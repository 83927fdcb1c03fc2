/*
 * fa_cache.h -- C ABI of libfa.so's key/value cache: paged storage written as
 * tokens arrive, read back whole, and attended by one new token per sequence.
 * The companion of fa.h for a model that answers token by token: fa_fwd serves
 * the prompt, fa_cache_append stores its keys and values, and each further token
 * is one fa_cache_append and one fa_decode.
 *
 * The cache.  Keys and values live in pages of page_size tokens.  Position n of
 * sequence b is row n % page_size of page block_table[b][n / page_size], so a
 * sequence's pages may lie anywhere and in any order, and two sequences may read
 * the same pages (a shared prefix).  Row (page, head, token) starts at
 *   k + page * k_stride[0] + head * k_stride[1] + token * k_stride[2]   (elements)
 * and its d elements are adjacent, so [pages, H, page_size, d] and
 * [pages, page_size, H, d] storage, and K and V as slices of one tensor, are all
 * described by their strides.  Two element types:
 *   FA_CACHE_BF16  bf16 words;
 *   FA_CACHE_E4M3  e4m3 codes (as in fa.h), one byte each, with one fp32 factor
 *                  per (page, head, token) in k_scale / v_scale: the row's values
 *                  are code * factor.  Factors have strides of their own
 *                  (k_scale_stride, v_scale_stride: page, head, token).
 * Rows that no sequence's length covers are never read into a result, whatever
 * they hold (NaN included).
 *
 * Limits: d in {64, 128}; page_size 16, 32, 64 or a multiple of 128; k and v
 * 16-byte aligned with strides that are multiples of 16 bytes and at least one
 * row apart; B, H, num_pages, max_pages >= 1; max_pages * page_size < 2^31.
 * The cache itself may be of any size (offsets are 64-bit).  A call's work is counted in
 * 31 bits: fa_cache_append takes 2 * T * H < 2^31, fa_cache_gather the elements that its
 * outputs may have, and fa_decode 6 * B * H * blocks * tiles < 2^31, with blocks = 1 for
 * up to 32 query heads per cache head (one more for every 32 beyond) and tiles = max_pages *
 * page_size / 128, rounded up: the table's capacity counts, whatever the lengths are.
 * Beyond these: FA_ERR_UNSUPPORTED.
 *
 * block_table is [B][max_pages] int32 with rows block_table_stride ints apart;
 * only the entries that a sequence's length reaches are read.  seq_lens is [B]
 * int32, tokens held per sequence, 0 allowed (an idle slot of a padded batch).
 * Both are read on the device.  A page id outside [0, num_pages) or a length
 * outside [0, max_pages * page_size] that a call meets is never followed: the
 * call records FA_ERR_DEVICE_CACHE (read it with fa_device_status; the info words
 * are kernel id (6 append, 7 gather, 8 decode), sequence, block, launch number),
 * and that sequence's outputs are undefined while the others' hold.  A timeout
 * or another failure of any kernel goes before it: it is what the status says then.
 *
 * Calls follow fa.h: asynchronous on `stream`, argument errors returned before
 * anything is launched, no allocation beyond the library's status block, nothing
 * kept between calls.  Every call may be captured into a graph after the device's
 * first call.
 */
#ifndef FA_CACHE_H_
#define FA_CACHE_H_

#include <stddef.h>

#include "fa.h"

#ifdef __cplusplus
extern "C" {
#endif

#define FA_CACHE_BF16 0
#define FA_CACHE_E4M3 1

/* fa_device_status(): a kernel met a page id or a length out of range. */
#define FA_ERR_DEVICE_CACHE 9

typedef struct {
    void *k, *v;                     /* device; 16-byte aligned */
    float *k_scale, *v_scale;        /* device; FA_CACHE_E4M3 only, else ignored */
    long long k_stride[3], v_stride[3];             /* page, head, token, in elements */
    long long k_scale_stride[3], v_scale_stride[3]; /* page, head, token, in floats */
    const int *block_table;          /* device [B][max_pages] */
    const int *seq_lens;             /* device [B] */
    long long block_table_stride;    /* ints between rows, >= max_pages */
    int type;                        /* FA_CACHE_BF16 or FA_CACHE_E4M3 */
    int num_pages, H, page_size, d;
    int B, max_pages;
} fa_paged_cache;

/*
 * Write T new tokens' keys and values.  k_new, v_new: bf16, token t of head h at
 * t * k_new_stride[0] + h * k_new_stride[1] (elements; multiples of 8; d adjacent
 * elements; 16-byte aligned), e.g. slices of a fused projection's output.
 *
 * seq_lens holds the lengths AFTER the write, so that the same tensor serves the
 * fa_decode that follows.  cu_new NULL: one token per sequence (T = B), written
 * at position seq_lens[b] - 1; a sequence of length 0 is skipped.  Otherwise
 * cu_new is [B + 1] int32, ascending from 0: tokens cu_new[b] .. cu_new[b+1] - 1
 * become the last positions of sequence b, in order; tokens that would fall before
 * position 0 are skipped, and tokens from cu_new[B] on (padding) are not read.
 *
 * FA_CACHE_BF16 copies.  FA_CACHE_E4M3 quantises each (token, head) row x:
 *   factor = max(max|x|, 1e-30) / 448,  code = e4m3(x / factor),
 * in fp32 with IEEE division, rounded to nearest even, so that the row's largest
 * element becomes 448, the largest e4m3 value.  The factor of a row that holds an
 * infinity or NaN is one too, and the row is NaN throughout: its codes are 0 or NaN.
 * The pages written by one call must not be shared: two sequences that own the
 * same row leave either's values, or a mix, in it.
 */
int fa_cache_append(const fa_paged_cache *cache, const void *k_new, const void *v_new,
                    const long long *k_new_stride, const long long *v_new_stride,
                    int T, const int *cu_new, void *stream);

/*
 * Read sequences back as the contiguous bf16 [B, H * rep, N, d] tensors that fa_fwd
 * takes: head h of the cache becomes heads h * rep .. h * rep + rep - 1 (rep query
 * heads that share it).  Row n >= seq_lens[b] is zero; positions from N on are left
 * out.  e4m3 rows are code * factor in fp32, rounded to bf16 (0 * infinity is NaN).  k_out or v_out NULL
 * leaves that one out.  B * H * rep * N * d < 2^31, as for fa_fwd.
 */
int fa_cache_gather(const fa_paged_cache *cache, void *k_out, void *v_out, int rep, int N,
                    void *stream);

/*
 * Bytes of scratch fa_decode needs (contents ignored on entry); 0 for invalid
 * arguments.  Concurrent calls, and captured graphs that may run at the same
 * time, each need their own.
 */
size_t fa_decode_workspace_bytes(int B, int Hq, int H, int d);

/*
 * Attention of one new token per sequence over its cache:
 *   o[b, h] = softmax_j(scale * q[b, h] . k_j) v_j,  lse[b, h] = ln sum_j exp(scale * q . k_j)
 * over positions j in [max(0, len - window), len) of cache head h / (Hq / H), with
 * len = seq_lens[b] (the new token's own key and value already appended); window = 0
 * means all of them.  q, o: [B, Hq, d] bf16, contiguous; lse: [B, Hq] fp32 (natural
 * log) or NULL.  Hq is a multiple of H.  o may be q itself (a row of q is last read
 * before its row of o is written), and overlaps nothing else.  A sequence of length 0
 * gets o = 0 and lse = -inf.  Scores, statistics and sums are fp32; o is rounded once, to bf16.
 * What the products round before that: weights below 2^-126 of the largest are 0, other bf16
 * weights have 16 bits; with FA_CACHE_E4M3 an element of q is held to within 2^-22 of the largest of
 * its row, and a weight times V's factor to within 2^-15 of itself or 2^-27 of the head's largest such
 * product (of 2^-80 of the largest among the heads that share the cache head, or 2^-120 of V's
 * largest visible factor, where that is more).  A visible row of such a cache whose factor is not
 * finite makes its heads' o NaN.  The products' sums are the tensor core's, which drop what lies
 * below fp32's last place: a part of 2^-23 at most for every 16 (bf16) or 32 (e4m3) positions
 * that one block takes of a sequence.
 * The result does not depend on where the pages lie, and repeated calls on the
 * same GPU return the same bits.
 */
int fa_decode(const fa_paged_cache *cache, const void *q, void *o, float *lse, int Hq, float scale,
              int window, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FA_CACHE_H_ */
