/*
 * The 8-bit latent cache in pages (dcp_mla_cache8.h has the format of a token,
 * of scales and of context shards): rows share pages, take over each other's,
 * and give them back; append, read-back and attention go through a table.
 *
 * The pool. A page is `page` tokens of one row of one shard, a power of two in
 * [DCP_MLA_PAGE_MIN, DCP_MLA_PAGE_MAX], and a multiple of `block`.
 *   kv     [P, page, Dk] e4m3 codes, contiguous, 16-byte aligned
 *   scales [P, page / block] fp32, contiguous
 * The tables, per shard, the same for all layers.
 *   tables [B, M] int32, contiguous: entry (b, i) is the page of tokens
 *          i * page .. of row b on this shard. An entry outside [0, P) is no
 *          page. A row's pages are its entries before the first such one; the
 *          append, the read-back and the attention look at each entry by itself.
 *   refs   [P] int32: how many rows hold a page; 0 is a free page. A program
 *          that wants to keep a page without a row adds 1 of its own.
 *
 * Asynchrony, ownership, errors: as for dcp_mla_cache8_decode. All counts stay
 * on the device, so that a step (update, copy, append, attend) can be captured.
 */
#ifndef DCP_MLA_PAGES_H
#define DCP_MLA_PAGES_H

#include <stdint.h>

#include "dcp_mla_cache8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DCP_MLA_PAGE_MIN 32
#define DCP_MLA_PAGE_MAX 4096
#define DCP_MLA_PAGES_POOLS_MAX 128

enum {
    DCP_MLA_CACHE8_ERR_BAD_PAGE = -211,  /* page not a power of two in range, or not a multiple of block */
    DCP_MLA_CACHE8_ERR_ALIAS = -212,     /* outputs that overlap inputs in a way that the call does not take */
    DCP_MLA_CACHE8_ERR_CLUSTER = -213    /* the device or context cannot hold a cluster of 16 blocks */
};

/*
 * One step of the tables: rows take over other rows' pages, are cut back, end,
 * begin and grow, all at once. For row b, with the tables as they are on entry:
 *   it takes the pages of the first keeps[b] positions from row parents[b] (b
 *   itself to go on; outside [0, B): from none, and keeps[b] counts as 0), and
 *   gets fresh pages for what it lacks below max(keeps[b], wants[b]) positions.
 * What it held besides is released: refs goes down by 1 for each page that a row
 * held and up by 1 for each that it holds. So {parents -1, wants 0} ends a row,
 * {b, n, n + k} makes room for k tokens behind n, {a, n, n + 1} forks row a.
 *   Positions are those of a sequence over all cp shards; this shard's share is
 *   what counts here (cp 1: all of them). They are at most M pages of the shard.
 * Copy on write. Where wants[b] > keeps[b] and the kept tokens end inside a page
 * that another row (or a program's own count) holds too, row b gets a fresh page
 * in its place, and copies[b] = (that page, the fresh one); otherwise copies[b] =
 * (-1, -1). If all who hold it are such rows, the last of them keeps it.
 * Fresh pages are those with refs 0 after all releases, the lowest first, dealt to
 * rows in order, in a row the copy's first and then by slot. Where they run out the
 * entry is -1, and *missing counts these; else it is 0. Where that was to be a copy's
 * page there is no copy, and the row has let go of the old one and of its tokens there:
 * a program that wants to go back to the state before writes to other buffers.
 *   tables_out, refs_out  either tables and refs themselves (in place), or buffers
 *            that overlap neither
 *   copies   [B, 2] int32, 8-byte aligned; missing: one int32
 *   parents, keeps, wants  [B] int32 (negative positions: 0)
 *   Nothing else that is written (copies, missing, the workspace) overlaps anything
 *   that the call takes, and tables_out and refs_out do not overlap these three.
 *   workspace at least dcp_mla_pages_update_workspace_bytes(...) bytes, 256-byte
 *            aligned (NULL where that is 0: out of place, with up to 16,384 rows and
 *            262,144 pages); its contents do not matter. Calls that share one are
 *            ordered.
 *   Beyond 32 rows, 8,192 entries or 8,192 pages the call is one cluster of 16 blocks,
 *   each a multiprocessor of its own: a whole GB300 has room for it, a smaller part (a
 *   context with few multiprocessors) may not, and returns DCP_MLA_CACHE8_ERR_CLUSTER.
 *   shapes   0 <= B <= 65535, 1 <= M, M * page < 2^31 (here and in the calls without a
 *            page: M < 2^26), B * (M + 1) < 2^31, 1 <= P < 2^31, 0 <= shard < cp
 */
int dcp_mla_pages_update(const int32_t* tables, const int32_t* refs, const int32_t* parents, const int32_t* keeps,
                         const int32_t* wants, int64_t B, int64_t M, int64_t P, int page, int cp, int shard,
                         int interleave, int32_t* tables_out, int32_t* refs_out, int32_t* copies, int32_t* missing,
                         void* workspace, int64_t workspace_bytes, void* stream);

/* Bytes of workspace for dcp_mla_pages_update, 0 for none; -1 for sizes out of range. Host only. */
int64_t dcp_mla_pages_update_workspace_bytes(int64_t B, int64_t M, int64_t P, int in_place);

/*
 * Move the pages in use to the front of the pool. With n pages of refs > 0, those
 * at n and beyond go, in ascending order, to the free ones below n in ascending
 * order: copies[i] = (page, its new place) for the i-th of them and (-1, -1) behind
 * the last. Entries of tables and refs are changed to match; an entry that is no
 * page, or a page that does not move, stays as it is. Nothing is copied here.
 *   copies   [P / 2, 2] int32, 8-byte aligned (more than P / 2 pages never move)
 *   tables_out, refs_out, workspace, overlaps, shapes as above (B = 0 is allowed)
 */
int dcp_mla_pages_compact(const int32_t* tables, const int32_t* refs, int64_t B, int64_t M, int64_t P,
                          int32_t* tables_out, int32_t* refs_out, int32_t* copies, void* workspace,
                          int64_t workspace_bytes, void* stream);

/* Bytes of workspace for dcp_mla_pages_compact; -1 for sizes out of range. Host only. */
int64_t dcp_mla_pages_compact_workspace_bytes(int64_t P);

/*
 * Copy pages, codes and scales, inside each of several pools (layers) of one
 * geometry: for each pair copies[i] = (src, dst), i < n, page src to page dst. A
 * pair with an entry outside [0, P) is passed over. No page may be the dst of two
 * pairs, or both dst and src.
 *   kv_ptrs, scale_ptrs  [pools] host arrays, pools <= DCP_MLA_PAGES_POOLS_MAX; no
 *            two pools overlap
 *   shapes   n >= 0, n times the parts of 36 KiB of a page below 2^31, 1 <= P < 2^31,
 *            Dk 512 or 576
 */
int dcp_mla_pages_copy(void* const* kv_ptrs, float* const* scale_ptrs, int pools, int64_t P, int page, int Dk,
                       int block, const int32_t* copies, int64_t n, void* stream);

/*
 * dcp_mla_cache8_append and dcp_mla_cache8_read over pages: the same calls, with a
 * token of row b that is number t of shard j at token t mod page of page
 * tables[j][b, t / page] of shard j's pool. A token whose entry is no page, or that
 * lies past M pages, has no place: it is not written, and not read. Two rows must
 * not append to one page in one call (dcp_mla_pages_update sees to it); nor may two
 * shards share a pool. table_ptrs: a pointer per shard, as kv_ptrs.
 *   shapes   0 <= B <= 65535, 0 <= P < 2^31, 1 <= M, B * M < 2^31, M * page < 2^31
 */
int dcp_mla_cache8_append_paged(const void* latent, int64_t latent_row, const void* k_rope, int64_t rope_row, int dtype,
                                int64_t N, int64_t B, int Dk, const int32_t* cu_new, const int32_t* seq_lens,
                                void* const* kv_ptrs, float* const* scale_ptrs, const int32_t* const* table_ptrs,
                                int cp, int64_t P, int page, int64_t M, int block, int interleave,
                                const double* inv_freq, int interleaved, float mscale, void* stream);
int dcp_mla_cache8_read_paged(const void* const* kv_ptrs, const float* const* scale_ptrs,
                              const int32_t* const* table_ptrs, int cp, int64_t B, int64_t P, int page, int64_t M,
                              int Dk, int block, int interleave, const int32_t* starts, const int32_t* cu, int64_t N,
                              void* out, int64_t out_row, int dtype, void* stream);

/*
 * dcp_mla_cache8_decode over pages: the same call and numerics, with the tokens'
 * places as above. A visible position without a page is not attended to (it counts in
 * the length); a row that sees no token gives out = 0 and lse = -inf.
 *
 * Rows that share a prefix. groups (or NULL) and shared say that consecutive rows
 * have their first positions in the same pages: row b belongs to the groups[b][1]
 * rows from row groups[b][0] on, and positions p < shared[b] of all of them are the
 * same; they are looked up in the table of the first of these rows that is at least
 * shared[b] long. Every row of a group has the same entries in groups and shared. A row
 * whose length is below shared (one that has ended, say, with a length of 0) takes no
 * part and is looked up in its own table. The result is that of the call without
 * groups (but for the order of sums); what is saved is work: tiles of the prefix are
 * multiplied with several rows' heads at a time where a row's heads do not fill the
 * kernel's blocks of 64. With H a multiple of 64, more than 2048 rows, or tables with
 * room for fewer than 1024 tiles of 128 tokens in all (B * cp * M * page / 128) or for
 * more than 2^29 (B * cp * (M * page / 128 + 2)), groups make no difference. Elsewhere
 * they are for prefixes that are long beside the rows' own tokens: they pay from about
 * 2000 tiles of rows times prefix on, where the prefix is about as long as what rows
 * have behind it, or longer; short of that they cost time, up to half of the call
 * without them (64 rows of 16 heads, 128 shared tokens and up to 16K of their own: 94
 * us, 66 without), and a caller leaves them out. Groups do not go together with a window.
 *   groups   [B, 2] int32, 8-byte aligned; shared [B] int32 (below 1: nothing is
 *            shared). Entries that break these rules give undefined results in the
 *            rows concerned.
 *   workspace at least dcp_mla_cache8_decode_paged_workspace_bytes(...) bytes
 *   shapes   as for both, T being M * page
 */
int dcp_mla_cache8_decode_paged(const void* q, int64_t q_row, int64_t q_head, const void* const* kv_ptrs,
                                const float* const* scale_ptrs, const int32_t* const* table_ptrs,
                                const int32_t* seq_lens, const int32_t* groups, const int32_t* shared, int cp,
                                int64_t B, int H, int Dk, int Dv, int64_t P, int page, int64_t M, int block,
                                int interleave, int64_t window, int64_t sinks, float scale, int lse_base_e,
                                void* workspace, int64_t workspace_bytes, void* out, float* lse, int32_t* status,
                                unsigned flags, void* stream);

/* Bytes of workspace for it, `grouped` with groups; 0 for none, -1 for sizes out of range. Host only. */
int64_t dcp_mla_cache8_decode_paged_workspace_bytes(int cp, int64_t B, int H, int page, int64_t M, int64_t window,
                                                    int64_t sinks, int grouped, int num_sms);

#ifdef __cplusplus
}
#endif

#endif /* DCP_MLA_PAGES_H */
