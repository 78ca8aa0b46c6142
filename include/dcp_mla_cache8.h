/*
 * The 8-bit latent cache of MLA decode, and what works on it: rotary
 * positions, the quantising append, the read-back, and single-token attention
 * over the cache (with an optional sliding window and a few first tokens that
 * stay visible). They chain as a serving step does: rotate the queries, append
 * the new tokens, attend. (dcp_mla_pages.h has the same cache in pages that rows
 * share.)
 *
 * The cache. A row (sequence) holds at most T tokens a shard. A token is Dk
 * e4m3 values, 512 latent dims (key and value) and, with Dk = 576, 64 rotary
 * key dims; Dk = 512 has no rotary part. Every `block` consecutive tokens of a
 * row of a shard share one fp32 scale: the cached value is code * scale.
 *   kv     [B, T, Dk] e4m3 codes (4 exponent, 3 mantissa bits, no infinity),
 *          contiguous, 16-byte aligned
 *   scales [B, ceil(T / block)] fp32, contiguous; positive (the append writes
 *          powers of two; the decode takes any from 2^-60 to 2^32, in any order
 *          along a row, and 0, which counts as 2^-60)
 * block is a power of two, at most DCP_MLA_CACHE8_BLOCK_MAX; 1 gives each token
 * its own scale.
 *
 * Context shards. With cp > 1 position p of a row is held by shard
 * (p / interleave) mod cp, as its token (p / (interleave * cp)) * interleave +
 * p mod interleave: the KV is interleaved over the ranks ("[DCP] Optimize
 * shared Output, Query, and Indexer/Top-K via peer memory", sglang #32851,
 * commit notes). Calls take cp pointers, and a NULL entry is a shard that this
 * device does not hold: the append skips its tokens, the read-back leaves them
 * as they were, and the decode attends to the others (its partial output and
 * LSE then go through dcp_lse_reduce).
 *
 * Asynchrony, ownership, errors: as for dcp_lse_reduce (everything is enqueued
 * on `stream` of the current device, nothing is allocated, calls can be
 * captured into graphs; negative codes are host argument errors with nothing
 * launched, positive codes are cudaError_t).
 */
#ifndef DCP_MLA_CACHE8_H
#define DCP_MLA_CACHE8_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DCP_MLA_CACHE8_BLOCK_MAX 128
#define DCP_MLA_CACHE8_CP_MAX 16
/* besides DCP_DTYPE_BF16 and DCP_DTYPE_F16 (dcp_lse_reduce.h) */
#define DCP_DTYPE_F32 2

enum {
    DCP_MLA_CACHE8_ERR_NULL_POINTER = -201, /* a required pointer is NULL (or every shard's) */
    DCP_MLA_CACHE8_ERR_BAD_SHAPE = -202,    /* a size out of range (see each call) */
    DCP_MLA_CACHE8_ERR_BAD_BLOCK = -203,    /* block not a power of two in [1, DCP_MLA_CACHE8_BLOCK_MAX] */
    DCP_MLA_CACHE8_ERR_BAD_CP = -204,       /* cp outside [1, DCP_MLA_CACHE8_CP_MAX], interleave outside
                                               [1, 2^24], or an append whose shards share a cache or scales */
    DCP_MLA_CACHE8_ERR_MISALIGNED = -205,   /* a pointer or a stride is not aligned as the call asks */
    DCP_MLA_CACHE8_ERR_BAD_DTYPE = -206,    /* a dtype that the call does not take */
    DCP_MLA_CACHE8_ERR_BAD_FLAGS = -207,    /* unknown flag bits */
    DCP_MLA_CACHE8_ERR_WORKSPACE = -208,    /* workspace NULL, not 256-byte aligned, or too small */
    DCP_MLA_CACHE8_ERR_BAD_WINDOW = -209,   /* window or sinks negative, or sinks without a window */
    DCP_MLA_CACHE8_ERR_TENSOR_MAP = -210    /* a TMA tensor map of a cache could not be encoded */
};

/* A message for any status of these calls (and of the library's others). */
const char* dcp_mla_cache8_strerror(int status);

/*
 * Rotary positions on part of each head. x is [N, H, D] (row stride x_row, head
 * stride x_head in elements, unit stride along D). Pairs of the `rot` dims from
 * `start` are turned by the angle positions[n] * inv_freq[i], i < rot / 2, and
 * multiplied by mscale:
 *     out[a] = (x[a] cos - x[b] sin) * mscale
 *     out[b] = (x[b] cos + x[a] sin) * mscale
 * with (a, b) = (start + 2i, start + 2i + 1) when `interleaved`, else
 * (start + i, start + i + rot / 2). The other dims are copied, or left alone
 * where out is x itself (rotating in place). out must either be x with the same
 * strides or not overlap it, and no two rows or heads of out may overlap each
 * other, in place neither (x that is only read may repeat rows or heads).
 *   inv_freq   [rot / 2] doubles on the device, radians per position. The angle
 *              is reduced to a fraction of a turn in 64-bit fixed point, so far
 *              positions keep what the double holds (2^-53 of the angle) and
 *              the rest is fp32. An infinite or NaN one makes its pair NaN.
 *   positions  [N] int32, or int64 with pos64; any sign, below 2^31 in size
 *   dtype      DCP_DTYPE_BF16, DCP_DTYPE_F16 or DCP_DTYPE_F32; the arithmetic
 *              is fp32, rounded once
 *   shapes     N >= 0, 1 <= H <= 65535, rot even and 2 <= rot <= 256,
 *              0 <= start, start + rot <= D <= 65536; any strides (where
 *              everything is a multiple of 16 bytes the call is faster)
 */
int dcp_mla_rope(const void* x, int64_t x_row, int64_t x_head, const void* positions, int pos64,
                 const double* inv_freq, int64_t N, int H, int D, int start, int rot, int interleaved, float mscale,
                 int dtype, void* out, int64_t out_row, int64_t out_head, void* stream);

/*
 * Append new tokens to the cache, quantising them on the way. Row b's new
 * tokens are cu_new[b] .. cu_new[b + 1] of the packed inputs (cu_new: [B + 1]
 * int32, cu_new[0] = 0, ascending, cu_new[B] <= N; or NULL: N / B tokens a row,
 * N a multiple of B), at positions seq_lens[b], seq_lens[b] + 1, ... (seq_lens:
 * [B] int32, the lengths before the call; the caller advances them). A packed
 * token at or past cu_new[B], and a position whose shard holds fewer than T
 * tokens for it, is not written.
 *   latent   [N, 512] bf16 or fp16, row stride latent_row (a multiple of 8
 *            elements), 16-byte aligned
 *   k_rope   [N, 64] of the same type, row stride rope_row (a multiple of 8),
 *            16-byte aligned; NULL with Dk = 512
 *   inv_freq NULL: k_rope is taken as it is; or [32] doubles as for
 *            dcp_mla_rope: k_rope is rotated (fp32, not rounded in between)
 * Scales. A block's scale is the smallest power of two s with |x| <= 448 s over
 * the finite values of its new tokens, at least 2^-60 (and up to 2^120: values
 * beyond 448 * 2^32 are cached and read back, but lie outside what the decode
 * takes). A block that already
 * holds tokens of the row keeps the larger of that and its present scale; where
 * it grows, the tokens that it holds are requantised (exact but for values that
 * become subnormal, which round to nearest even). Codes round to nearest even;
 * NaN and infinities are stored as NaN, and so is the pair of a frequency that is
 * not finite.
 * Each block is written by one CTA in a fixed way: the result does not depend on
 * timing. One launch.
 *   shapes   0 <= N < 2^31, 0 <= B <= 65535, 0 <= T < 2^31, Dk 512 or 576
 */
int dcp_mla_cache8_append(const void* latent, int64_t latent_row, const void* k_rope, int64_t rope_row, int dtype,
                          int64_t N, int64_t B, int Dk, const int32_t* cu_new, const int32_t* seq_lens,
                          void* const* kv_ptrs, float* const* scale_ptrs, int cp, int64_t T, int block,
                          int interleave, const double* inv_freq, int interleaved, float mscale, void* stream);

/*
 * Read cached tokens back: packed token cu[b] + i of out is position
 * starts[b] + i of row b (cu as cu_new above; starts NULL: 0), as code * scale
 * rounded to dtype (bf16, fp16 or fp32; round to nearest even). Packed tokens at
 * or past cu[B], positions of shards that are not held and positions past a
 * shard's T tokens are left as they were in out.
 *   out      [N, Dk], row stride out_row (bytes a multiple of 16), 16-byte
 *            aligned
 */
int dcp_mla_cache8_read(const void* const* kv_ptrs, const float* const* scale_ptrs, int cp, int64_t B, int64_t T,
                        int Dk, int block, int interleave, const int32_t* starts, const int32_t* cu, int64_t N,
                        void* out, int64_t out_row, int dtype, void* stream);

/*
 * Single-token attention over the cache. For row b with L = seq_lens[b]
 * positions (negative: 0), every head attends to
 *     all positions p < L                                   (window = 0)
 *     p < L with p >= L - window or p < sinks               (window > 0)
 * that a held shard has (a position past a shard's T tokens, which the append
 * drops, counts in L but is not seen):
 *     s_p       = scale * <q[b, h, :Dk], kv[p, :Dk]>
 *     out[b, h] = sum_p softmax(s)_p * kv[p, :512]
 *     lse[b, h] = log_base sum_p exp(s_p)
 * A row that sees nothing gives out = 0 and lse = -inf.
 *   q        [B, H, Dk] bf16, row stride q_row, head stride q_head (even
 *            elements), 4-byte aligned
 *   out      [B, H, 512] bf16, contiguous, 16-byte aligned
 *   lse      [B, H] fp32, contiguous, base e or 2; may be NULL
 *   workspace at least dcp_mla_cache8_decode_workspace_bytes(...) bytes,
 *            256-byte aligned, owned by the caller (NULL where that is 0); its
 *            contents on entry do not matter. Calls that share one must be
 *            ordered.
 *   status   as for dcp_mla_decode_partial: NULL, or a device int32 that the
 *            kernel ORs 1 into if a wait for its own copies or MMAs ever
 *            exceeds two seconds; the outputs are then not valid
 *   flags    0 or a combination of DCP_FLAG_PDL (1) and, for tests,
 *            DCP_MLA_FLAG_TEST_STALL (32; see dcp_mla_decode.h: the first tile
 *            of each CTA never counts as landed, waits give up after 20 ms)
 *   shapes   0 <= B <= 65535, 1 <= H <= 1024, Dk 512 or 576, Dv 512,
 *            0 <= T < 2^31, B * cp * (T / 128 + 2) <= 2^30, window and sinks >= 0
 * Numerics. The codes go to the tensor cores as they are. q is split into two
 * e4m3 parts at a power-of-two scale per head, which holds every value above
 * 2^-9 of the head's largest exactly (and the others to 2^-16 of it).
 * Probabilities are split the same way at a power-of-two scale for each head and
 * 32 tokens, to 2^-8 relative like bf16. Products accumulate in fp32, and log2 of
 * a token's scale is added to its score in fp32 (so that scales near 2^-60 leave a
 * score some 2^-18); output rounded once to bf16. A NaN code or scale that is visible, or a NaN or infinity
 * in q, makes the (row, head) NaN; tokens that are not visible may hold anything.
 * In units of ln 2, scores above 2^21 make it NaN too, and one below -2^21 has
 * weight 0 or makes it NaN.
 */
int dcp_mla_cache8_decode(const void* q, int64_t q_row, int64_t q_head, const void* const* kv_ptrs,
                          const float* const* scale_ptrs, const int32_t* seq_lens, int cp, int64_t B, int H, int Dk,
                          int Dv, int64_t T, int block, int interleave, int64_t window, int64_t sinks, float scale,
                          int lse_base_e, void* workspace, int64_t workspace_bytes, void* out, float* lse,
                          int32_t* status, unsigned flags, void* stream);

/*
 * Bytes of workspace dcp_mla_cache8_decode needs for these sizes on a device
 * with num_sms multiprocessors (cudaDevAttrMultiProcessorCount); 0 where no row
 * can be long enough to be split; -1 for sizes out of range. Host only.
 */
int64_t dcp_mla_cache8_decode_workspace_bytes(int cp, int64_t B, int H, int64_t T, int64_t window, int64_t sinks,
                                              int num_sms);

#ifdef __cplusplus
}
#endif

#endif /* DCP_MLA_CACHE8_H */
