// Pages of the 8-bit latent cache, sm_103a: the step of the tables (fork, cut, end,
// grow), the compaction of a pool and the copying of pages. What they do is stated
// in include/dcp_mla_pages.h.
//
// Tables and counts are a few KB to a few MB, and what a call costs is dependent
// round trips, barriers and instructions. Sums over rows and over the pool give
// every row and every free page its rank, so nothing depends on the order in which
// CTAs or atomics come (atomics here are sums and maxima of integers), and no count
// leaves the device.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "dcp_lse_reduce.h"
#include "dcp_mla_pages.h"

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kClusterMax = 16;  // (beyond 8 by the kernel's leave)
constexpr int kSms = 152;  // GB300's multiprocessors, for the launch rules: with another count they cost time only

__device__ __forceinline__ int lane_sums(int x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// A shard's share of the first L positions.
__device__ __forceinline__ int share_of(int L, uint32_t cp, uint32_t shard, uint32_t interleave) {
    if (L <= 0 || cp == 1) return max(L, 0);
    const uint32_t round = cp * interleave, q = (uint32_t)L / round, r = (uint32_t)L - q * round, lo = shard * interleave;
    const uint32_t part = r > lo ? r - lo : 0;
    return (int)(q * interleave + (part < interleave ? part : interleave));
}

// The place of the k-th set bit of a word that has more than k.
__device__ __forceinline__ int bit_of_rank(uint32_t bits, int k) {
    int at = 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const int n = __popc(bits & ((1u << o) - 1));
        if (k >= n) {
            k -= n;
            at += o;
            bits >>= o;
        }
    }
    return at;
}

// Exclusive sum of x over the CTA's threads; *all the CTA's sum.
__device__ __forceinline__ int block_sums(int x, int* all) {
    __shared__ int warp_s[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int incl = lane_sums(x, lane);
    __syncthreads();
    if (lane == 31) warp_s[warp] = incl;
    __syncthreads();
    const int w = warp_s[lane];  // (kWarps = 32)
    *all = __reduce_add_sync(0xffffffffu, w);
    return incl - x + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
}

// The last of n ascending numbers that is at most k (the first is).
__device__ __forceinline__ int last_at_most(const int* v, int n, int k) {
    int lo = 0;
    while (n > 1) {
        const int half = n >> 1;
        if (v[lo + half] <= k) {
            lo += half;
            n -= half;
        } else {
            n = half;
        }
    }
    return lo;
}

// ---- the step of the tables ------------------------------------------------------

// One cluster does a call, in four phases between cluster barriers; each CTA has a contiguous share of the rows, a warp
// a row, and of the pool. The pool's counts live in the CTAs' shared memory, or in the workspace where the pool is too
// large for that: through generic addresses the code is the same. Bound by its chain of round trips and barriers: 4 beams
// 6.5 us, 256 rows x 128 entries and 16,384 pages 9.3 (13.6 and 16.1 with all of it in global memory, lists and six
// barriers), 512 rows x 512 and 120,000 pages 16.0.
struct alignas(16) RowPlan {
    int taken;  // pages that it takes over
    int pages;  // pages that it has afterwards
    int last;   // the page that it is about to write behind kept tokens, or -1; -2 - it if that is copied
    int first;  // rank of its first fresh page among its CTA's
};

// Of a page: how many hold it; how many rows are about to write it behind kept tokens, and the last of them, plus one.
// Of 32 pages: which are free, and how many of the warp's part before them are.
struct Pool {
    int* held;
    int2* writers;
    uint32_t* free;
    int* before;
};

struct UpdateParams {
    const int *tables, *refs, *parents, *keeps, *wants;
    int *tables_out, *refs_out, *copies, *missing;
    RowPlan* plan;    // [B], for rows that a CTA's shared memory has no room for
    Pool pool;        // for pools that it has none for
    int* staged;      // [B, M] pages taken over from another row (in place)
    int M, B, P, page_log2, in_place;
    int part_log2;    // pages of a warp's part
    int cp, shard, interleave;
};

constexpr int kRowsShared = 1024;
constexpr int kPagesShared = 16384;  // of a CTA: 12.25 bytes each

template <bool kShared>
__global__ void __launch_bounds__(kThreads) update_kernel(const __grid_constant__ UpdateParams p) {
    extern __shared__ __align__(16) uint8_t pool_s[];
    __shared__ RowPlan plan_s[kRowsShared];
    __shared__ int free_s[kClusterMax * kWarps + 1];  // free pages before each warp's part
    __shared__ int need_s[kClusterMax];               // fresh pages that each CTA's rows need
    const cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ctas = (int)gridDim.x, cta = (int)blockIdx.x, parts = ctas * kWarps;
    const int rows = (p.B + ctas - 1) / ctas, row0 = cta * rows, row1 = min(row0 + rows, p.B);
    RowPlan* const plan = rows <= kRowsShared ? plan_s : p.plan + row0;  // (of this CTA's rows alone)

    const int own_log2 = p.part_log2 + 5, own = 1 << own_log2;  // pages of a CTA
    Pool mine = p.pool;
    if constexpr (kShared) {
        mine.held = reinterpret_cast<int*>(pool_s);
        mine.writers = reinterpret_cast<int2*>(mine.held + own);
        mine.free = reinterpret_cast<uint32_t*>(mine.writers + own);
        mine.before = reinterpret_cast<int*>(mine.free + own / 32);
    }
    // entry i of an array of Pool, one entry for 2^per_log2 pages, wherever it is
    const auto at = [&](auto* base, int i, int per_log2) {
        if constexpr (kShared)
            return cluster.map_shared_rank(base, (unsigned)i >> (own_log2 - per_log2)) +
                   (i & ((1 << (own_log2 - per_log2)) - 1));
        else return base + i;
    };
    const int64_t page0 = (int64_t)cta << own_log2;
    const int here = page0 >= p.P ? 0 : (int)min((int64_t)own, p.P - page0);  // pages of this CTA
    const int64_t base = kShared ? 0 : page0;                                 // where its first one is in Pool

    // ---- the counts to begin with
    for (int i0 = tid; i0 < here; i0 += 4 * kThreads) {
        int n[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i0 + u * kThreads < here) n[u] = p.refs[page0 + i0 + u * kThreads];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kThreads;
            if (i >= here) break;
            mine.held[base + i] = n[u];
            mine.writers[base + i] = make_int2(0, 0);
        }
    }
    cluster.sync();
    // ---- what each row takes over, and the counts of pages that change hands
    const int room = p.M << p.page_log2;
    const int page_up = (1 << p.page_log2) - 1;
    for (int b = row0 + warp; b < row1; b += kWarps) {
        const int from = p.parents[b], keeps = p.keeps[b], wants = p.wants[b];
        const bool some = from >= 0 && from < p.B, self = from == b;
        const int keep = some ? min(room, share_of(keeps, p.cp, p.shard, p.interleave)) : 0;
        const int want = min(room, share_of(wants, p.cp, p.shard, p.interleave));
        const int n_keep = (keep >> p.page_log2) + ((keep & page_up) != 0);
        const int n_want = (want >> p.page_log2) + ((want & page_up) != 0);
        const int edge = want > keep && (keep & page_up) ? keep >> p.page_log2 : -1;
        const int* const my_row = p.tables + b * p.M;
        const int* const their_row = p.tables + (some ? from : b) * p.M;
        int taken = 0, last = -1;
        bool more_mine = true, more_theirs = !self && n_keep > 0;
        for (int i0 = 0; i0 < p.M && (more_mine || more_theirs); i0 += 128) {
            int e[4], f[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u + lane;
                e[u] = more_mine && i < p.M ? my_row[i] : -1;
                f[u] = more_theirs && i < n_keep ? their_row[i] : -1;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + 32 * u + lane;
                if (i0 + 32 * u >= p.M) break;
                uint32_t bad = __ballot_sync(0xffffffffu, (unsigned)e[u] >= (unsigned)p.P);
                if (!more_mine || lane >= (bad ? __ffs(bad) - 1 : 32)) e[u] = -1;
                more_mine = more_mine && !bad;
                if (self) {
                    f[u] = i < n_keep ? e[u] : -1;
                } else {
                    bad = __ballot_sync(0xffffffffu, (unsigned)f[u] >= (unsigned)p.P);
                    if (!more_theirs || lane >= (bad ? __ffs(bad) - 1 : 32)) f[u] = -1;
                    more_theirs = more_theirs && !bad;
                }
                taken += __popc(__ballot_sync(0xffffffffu, f[u] >= 0));
                if (i == edge) last = f[u];
                if (e[u] != f[u]) {
                    if (e[u] >= 0) atomicSub(at(mine.held, e[u], 0), 1);
                    if (f[u] >= 0) atomicAdd(at(mine.held, f[u], 0), 1);
                }
                if (!p.in_place) {
                    if (i < p.M) p.tables_out[b * p.M + i] = f[u];
                } else if (!self && f[u] >= 0) {
                    p.staged[b * p.M + i] = f[u];
                }
            }
            if (!p.in_place && !more_mine && !more_theirs)  // the rest of the row has no pages
                for (int i = i0 + 128 + lane; i < p.M; i += 32) p.tables_out[b * p.M + i] = -1;
        }
        if (last >= 0) {  // (one lane)
            int2* const who = at(mine.writers, last, 0);
            atomicAdd(&who->x, 1);
            atomicMax(&who->y, b + 1);
        }
        last = __reduce_max_sync(0xffffffffu, last);
        if (lane == 0) plan[b - row0] = {taken, max(n_keep, n_want), last, 0};
    }
    cluster.sync();
    // ---- how many fresh pages each row needs, and which pages are free
    int need_all = 0;
    for (int b0 = row0; b0 < row1; b0 += kThreads) {
        const int b = b0 + tid;
        int need = 0;
        RowPlan w = {0, 0, -1, 0};
        if (b < row1) {
            w = plan[b - row0];
            need = w.pages - w.taken;
            if (w.last >= 0) {
                const int2 who = *at(mine.writers, w.last, 0);
                if (who.x < *at(mine.held, w.last, 0) || who.y != b + 1) {
                    w.last = -2 - w.last;
                    ++need;
                }
            }
        }
        int all;
        w.first = need_all + block_sums(need, &all);
        if (b < row1) plan[b - row0] = w;
        need_all += all;
    }
    const int words = 1 << (p.part_log2 - 5), word0 = warp * words;  // of this warp's part
    int n_free = 0;
    for (int w0 = word0; w0 < word0 + words && w0 * 32 < here; w0 += 4) {
        int n[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = (w0 + u) * 32 + lane;
            n[u] = w0 + u < word0 + words && i < here ? mine.held[base + i] : 1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int w = w0 + u;
            if (w >= word0 + words || w * 32 >= here) break;
            const uint32_t m = __ballot_sync(0xffffffffu, n[u] == 0);
            if (lane == 0) {
                mine.free[(base >> 5) + w] = m;
                mine.before[(base >> 5) + w] = n_free;
            }
            n_free += __popc(m);
        }
    }
    if (lane < ctas) {
        *cluster.map_shared_rank(&free_s[cta * kWarps + warp], lane) = n_free;
        if (warp == 0) *cluster.map_shared_rank(&need_s[cta], lane) = need_all;
    }
    cluster.sync();
    // ---- the rows' new entries
    int need_total = 0, need_before = 0;
    for (int c = 0; c < ctas; ++c) {
        need_before += c < cta ? need_s[c] : 0;
        need_total += need_s[c];
    }
    int free_total;
    {
        const int n = tid < parts ? free_s[tid] : 0;
        const int before = block_sums(n, &free_total);
        if (tid < parts) free_s[tid] = before;
        __syncthreads();
    }
    if (cta == 0 && tid == 0) *p.missing = max(need_total - free_total, 0);
    const auto deal = [&](int rank) {
        if (rank >= free_total) return -1;
        const int part = last_at_most(free_s, parts, rank);
        rank -= free_s[part];
        const int first = part << (p.part_log2 - 5);  // the part's words, of which the pool's last one may have fewer
        const int* const before = at(mine.before, first, 5);
        const int w = last_at_most(before, min(words, (p.P - 1) / 32 + 1 - first), rank);
        const uint32_t bits = *at(mine.free, first + w, 5);
        return (part << p.part_log2) + 32 * w + bit_of_rank(bits, rank - before[w]);
    };
    for (int b = row0 + warp; b < row1; b += kWarps) {
        const RowPlan w = plan[b - row0];
        int* const row = p.tables_out + b * p.M;
        int rank = need_before + w.first;
        if (p.in_place) {
            if (p.parents[b] != b)
                for (int i = lane; i < w.taken; i += 32) row[i] = p.staged[b * p.M + i];
            for (int i = w.pages + lane; i < p.M; i += 32) row[i] = -1;  // (whatever stood behind the row's pages)
            __syncwarp();
        }
        const bool copied = w.last < -1;
        if (lane == 0) {
            int2 pair = make_int2(-1, -1);
            if (copied) {
                const int got = deal(rank);
                row[share_of(p.keeps[b], p.cp, p.shard, p.interleave) >> p.page_log2] = got;
                if (got >= 0) pair = make_int2(-2 - w.last, got);
            }
            reinterpret_cast<int2*>(p.copies)[b] = pair;
        }
        rank += copied;
        for (int i = w.taken + lane; i < w.pages; i += 32) row[i] = deal(rank + (i - w.taken));
    }
    // ---- the counts: a free page that is dealt has one holder; all rows that copy a page (each of its writers, but the
    // last if nobody else holds it) let go of it
#pragma unroll 4
    for (int i = tid; i < here; i += kThreads) {
        const int n = mine.held[base + i], w = mine.writers[base + i].x;
        int to = n - (w < n ? w : max(w - 1, 0));
        if (n == 0) {
            const uint32_t bits = mine.free[(base + i) >> 5];
            const int rank = free_s[cta * kWarps + (i >> p.part_log2)] + mine.before[(base + i) >> 5] +
                             __popc(bits & ((1u << (i & 31)) - 1));
            if (rank < need_total) to = 1;
        }
        p.refs_out[page0 + i] = to;
    }
    cluster.sync();  // (until all have read this CTA's shared memory)
}

// ---- compaction --------------------------------------------------------------------

// With n pages in use, the page at n or beyond that is the k-th such one goes to the k-th free page below n. Two
// launches: the first notes which pages are in use, with sums, the second asks them for every page that moves and every
// entry that names one, all at once: 5.8 us for 16,384 pages and entries, 4.3 for 384. (As one cluster, in five phases,
// 13.2 us.) Bound by the two launches and their round trips.
struct CompactParams {
    const int *tables, *refs;
    int *tables_out, *refs_out, *copies;
    uint32_t* bits;         // [words] pages in use
    int* before;            // [words] how many of the chunk before the word
    int* chunks;            // how many of a chunk
    int64_t entries;        // B x M
    int P, in_place, words, chunk_log2, chunk_count;  // a chunk: 2^chunk_log2 words
};
constexpr int kChunksMax = 1024;
constexpr int kWordsShared = 4096;  // of all words' sums and bits in shared memory: pools of 131,072 pages

__global__ void __launch_bounds__(kThreads) census_kernel(const __grid_constant__ CompactParams p) {
    __shared__ int count_s[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    int before = 0;
    for (int w0 = 0; w0 < 1 << p.chunk_log2; w0 += kWarps) {
        const int64_t w = ((int64_t)blockIdx.x << p.chunk_log2) + w0 + warp, i = w * 32 + lane;
        const uint32_t m = __ballot_sync(0xffffffffu, i < p.P && p.refs[i] > 0);
        if (lane == 0) count_s[warp] = __popc(m);
        __syncthreads();
        const int n = count_s[lane];
        if (lane == 0 && w < p.words) p.bits[w] = m;
        const int mine = before + __reduce_add_sync(0xffffffffu, lane < warp ? n : 0);
        if (lane == 0 && w < p.words) p.before[w] = mine;
        before += __reduce_add_sync(0xffffffffu, n);
        __syncthreads();
    }
    if (threadIdx.x == 0) p.chunks[blockIdx.x] = before;
}

constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) move_kernel(const __grid_constant__ CompactParams p) {
    __shared__ int used_s[kChunksMax + 1], warp_s[kMoveThreads / 32];
    extern __shared__ uint32_t words_s[];
    const int tid = threadIdx.x, lane = tid & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t* bits = p.bits;
    const int* before = p.before;
    if (p.words <= kWordsShared) {
        for (int i = tid; i < p.words; i += kMoveThreads) {
            words_s[i] = p.bits[i];
            words_s[p.words + i] = (uint32_t)p.before[i];
        }
        bits = words_s;
        before = reinterpret_cast<const int*>(words_s + p.words);
    }
    // used pages before each chunk: a thread has kChunksMax / kMoveThreads of them
    constexpr int kPer = kChunksMax / kMoveThreads;
    int n[kPer], sum = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        n[k] = tid * kPer + k < p.chunk_count ? p.chunks[tid * kPer + k] : 0;
        sum += n[k];
    }
    const int incl = lane_sums(sum, lane);
    if (lane == 31) warp_s[tid >> 5] = incl;
    __syncthreads();
    int at = incl - sum + __reduce_add_sync(0xffffffffu, lane < (tid >> 5) ? warp_s[lane & 7] : 0);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        used_s[tid * kPer + k] = at;
        at += n[k];
    }
    if (tid == kMoveThreads - 1) used_s[kChunksMax] = at;
    __syncthreads();
    const int live = used_s[kChunksMax], chunk_pages = 32 << p.chunk_log2;
    // used pages before page i < P
    const auto rank_of = [&](int i) {
        return used_s[i >> (p.chunk_log2 + 5)] + before[i >> 5] + __popc(bits[i >> 5] & ((1u << (i & 31)) - 1));
    };
    const int below = live < p.P ? rank_of(live) : live, moves = live - below;
    // the k-th free page, k < moves
    const auto hole = [&](int k) {
        int lo = 0, hi = p.chunk_count;  // free pages before chunk lo <= k
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (mid * chunk_pages - used_s[mid] <= k) lo = mid; else hi = mid;
        }
        k -= lo * chunk_pages - used_s[lo];
        const int w0 = lo << p.chunk_log2;
        int w = w0, w1 = min(w0 + (1 << p.chunk_log2), p.words);
        while (w1 - w > 1) {
            const int mid = (w + w1) >> 1;
            if ((mid - w0) * 32 - before[mid] <= k) w = mid; else w1 = mid;
        }
        return w * 32 + bit_of_rank(~bits[w], k - ((w - w0) * 32 - before[w]));
    };
    const auto used = [&](int i) { return (bits[i >> 5] >> (i & 31)) & 1u; };
    const int64_t threads = (int64_t)gridDim.x * kMoveThreads, me = (int64_t)blockIdx.x * kMoveThreads + tid;
    for (int64_t i = moves + me; i < p.P / 2; i += threads) reinterpret_cast<int2*>(p.copies)[i] = make_int2(-1, -1);
    for (int64_t i = me; i < p.P; i += threads) {
        if (i >= live && used((int)i)) {
            const int k = rank_of((int)i) - below, to = hole(k);
            reinterpret_cast<int2*>(p.copies)[k] = make_int2((int)i, to);
            p.refs_out[to] = p.refs[i];
            p.refs_out[i] = 0;
        } else if (!p.in_place && (i >= live || used((int)i))) {  // (a free page below `live` gets a count above)
            p.refs_out[i] = p.refs[i];
        }
    }
    for (int64_t i = me; i < p.entries; i += threads) {
        const int e = p.tables[i];
        const int to = e >= live && e < p.P && used(e) ? hole(rank_of(e) - below) : e;
        if (!p.in_place || to != e) p.tables_out[i] = to;
    }
}

// ---- copying pages --------------------------------------------------------------------

struct CopyParams {
    uint8_t* kv[DCP_MLA_PAGES_POOLS_MAX];
    float* scales[DCP_MLA_PAGES_POOLS_MAX];
    const int2* copies;
    int64_t page_bytes;
    int P, scale_words, parts;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 9;  // 16-byte pieces of a thread: a part is 36 KiB, a page of 64 tokens

// A CTA copies a part of a page of one pool, every load in flight before the first store; one with an empty pair has
// nothing to do. Bound by DRAM: 3,605 of 8,192 pairs, pages of 64 tokens, 266 MB read and written, 41.6 us, 6.4 TB/s
// (43.7 with stores that stay in L2; 45.4 with as many CTAs as are resident, each going over the list: a CTA's loads
// then wait for its stores); a few pages 2.6 us. Empty pairs cost their CTAs: ten pages of 8,192 pairs 7.4 us in one
// pool, 263 in 60 (3,605 pages in 20 and in 60 pools: 782 and 2,339).
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
    const int part = (int)(blockIdx.x % (unsigned)p.parts);
    const int2 c = p.copies[blockIdx.x / (unsigned)p.parts];
    if (c.x < 0 || c.x >= p.P || c.y < 0 || c.y >= p.P) return;
    const int64_t at = (int64_t)part * (kCopyThreads * kCopyVecs * 16), bytes = p.page_bytes - at;
    uint8_t* const pool = p.kv[blockIdx.y];
    const uint4* const src = reinterpret_cast<const uint4*>(pool + c.x * p.page_bytes + at);
    uint4* const dst = reinterpret_cast<uint4*>(pool + c.y * p.page_bytes + at);
    uint4 v[kCopyVecs];
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k) {
        const int j = k * kCopyThreads + (int)threadIdx.x;
        if (j * 16 < bytes) v[k] = __ldcs(src + j);
    }
#pragma unroll
    for (int k = 0; k < kCopyVecs; ++k) {
        const int j = k * kCopyThreads + (int)threadIdx.x;
        if (j * 16 < bytes) __stcs(dst + j, v[k]);
    }
    if (part == 0) {
        const float* const from = p.scales[blockIdx.y] + (int64_t)c.x * p.scale_words;
        float* const to = p.scales[blockIdx.y] + (int64_t)c.y * p.scale_words;
        for (int j = threadIdx.x; j < p.scale_words; j += kCopyThreads) to[j] = from[j];
    }
}

// ---- host side -------------------------------------------------------------------------

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
int64_t round_up(int64_t x) { return (x + 255) / 256 * 256; }
// (a row's room, in tokens of the smallest page, is below 2^31: loops over its entries count in 32 bits)
bool sizes_ok(int64_t B, int64_t M, int64_t P) {
    return B >= 0 && B <= 65535 && M >= 1 && M <= 0x7fffffff / DCP_MLA_PAGE_MIN && B * (M + 1) <= 0x7fffffff && P >= 1 &&
           P <= 0x7fffffff;
}
int page_log2_of(int page) {
    for (int k = 0; (1 << k) <= DCP_MLA_PAGE_MAX; ++k)
        if (page == 1 << k) return (1 << k) >= DCP_MLA_PAGE_MIN ? k : -1;
    return -1;
}
bool overlap(const void* a, int64_t an, const void* b, int64_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return an > 0 && bn > 0 && x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

int log2_up(int64_t x) {
    int k = 0;
    while ((int64_t)1 << k < x) ++k;
    return k;
}
// Pages of a warp's part of the pool, as a power of two, at least 32.
int part_log2_of(int64_t P, int ctas) {
    const int k = log2_up((P + ctas * kWarps - 1) / (ctas * kWarps));
    return k < 5 ? 5 : k;
}
struct UpdateSpace {
    int64_t plan, held, writers, free, before, staged, bytes;
};
UpdateSpace update_space(int64_t B, int64_t M, int64_t P, bool in_place) {
    const int64_t pool = P > kClusterMax * kPagesShared ? P : 0, words = (pool + 31) / 32;
    UpdateSpace w;
    w.plan = 0;
    w.held = w.plan + (B > kClusterMax * kRowsShared ? round_up(B * 16) : 0);
    w.writers = w.held + round_up(pool * 4);
    w.free = w.writers + round_up(pool * 8);
    w.before = w.free + round_up(words * 4);
    w.staged = w.before + round_up(words * 4);
    w.bytes = w.staged + (in_place ? round_up(B * M * 4) : 0);
    return w;
}
struct CompactSpace {
    int64_t bits, before, chunks, bytes;
};
CompactSpace compact_space(int64_t P) {
    const int64_t words = (P + 31) / 32;
    CompactSpace w;
    w.bits = 0;
    w.before = w.bits + round_up(words * 4);
    w.chunks = w.before + round_up(words * 4);
    w.bytes = w.chunks + round_up(kChunksMax * 4);
    return w;
}

// CTAs of a step of the tables: one where a row a warp and few entries and pages a thread are, else a cluster of 16. (4
// beams, 256 pages: 6.5 us with one, 7.5 with 8; 256 rows, 16,384 pages: 9.8 with 8, 9.3 with 16; 512 rows x 512, 120,000
// pages: 21.4 with 8, 16.0 with 16.) A cluster of 16 takes 16 whole multiprocessors of one group of them; where a device or
// a context has none that large, the call says so (a cluster of 8 would need a larger workspace than callers bring).
int cluster_of(int64_t rows, int64_t entries, int64_t P) {
    return rows <= kWarps && entries <= 8 * kThreads && P <= 8 * kThreads ? 1 : kClusterMax;
}

template <bool kShared>
int launch_update(const UpdateParams& p, int ctas, int shared_bytes, cudaStream_t st) {
    static int configured[64] = {}, holds[64] = {};  // (holds: a cluster of kClusterMax can be resident)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev < 0 || dev >= 64 || !__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE))) {
        e = cudaFuncSetAttribute(update_kernel<kShared>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kShared ? kPagesShared / 32 * (12 * 32 + 8) : 0);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(update_kernel<kShared>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess && dev >= 0 && dev < 64) __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
    }
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)ctas);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = (size_t)shared_bytes;
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)ctas;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (ctas > 1 && (dev < 0 || dev >= 64 || !__atomic_load_n(&holds[dev], __ATOMIC_ACQUIRE))) {
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, update_kernel<kShared>, &cfg);
            if (e == cudaErrorInvalidClusterSize || (e == cudaSuccess && n < 1)) {
                (void)cudaGetLastError();
                return DCP_MLA_CACHE8_ERR_CLUSTER;
            }
            if (e == cudaSuccess && dev >= 0 && dev < 64) __atomic_store_n(&holds[dev], 1, __ATOMIC_RELEASE);
        }
        if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, update_kernel<kShared>, p);
    }
    if (e != cudaSuccess) (void)cudaGetLastError();
    return (int)e;
}

// in place, or outputs that share nothing with the inputs
int check_alias(const int32_t* tables, const int32_t* refs, const int32_t* tables_out, const int32_t* refs_out,
                int64_t entries, int64_t P) {
    if (tables == tables_out && refs == refs_out) return overlap(tables, entries * 4, refs, P * 4);
    return overlap(tables, entries * 4, tables_out, entries * 4) || overlap(refs, P * 4, refs_out, P * 4) ||
           overlap(tables, entries * 4, refs_out, P * 4) || overlap(refs, P * 4, tables_out, entries * 4) ||
           overlap(tables_out, entries * 4, refs_out, P * 4);
}

struct Span {
    const void* at;
    int64_t bytes;
};
// Whether one of `written` overlaps another one, or one of `others`.
bool meet(std::initializer_list<Span> written, std::initializer_list<Span> others) {
    for (const Span* w = written.begin(); w != written.end(); ++w) {
        for (const Span* v = written.begin(); v != w; ++v)
            if (overlap(w->at, w->bytes, v->at, v->bytes)) return true;
        for (const Span& o : others)
            if (overlap(w->at, w->bytes, o.at, o.bytes)) return true;
    }
    return false;
}

}  // namespace

extern "C" int64_t dcp_mla_pages_update_workspace_bytes(int64_t B, int64_t M, int64_t P, int in_place) {
    return sizes_ok(B, M, P) ? update_space(B, M, P, in_place != 0).bytes : -1;
}

extern "C" int64_t dcp_mla_pages_compact_workspace_bytes(int64_t P) {
    return sizes_ok(0, 1, P) ? compact_space(P).bytes : -1;
}

extern "C" int dcp_mla_pages_update(const int32_t* tables, const int32_t* refs, const int32_t* parents,
                                    const int32_t* keeps, const int32_t* wants, int64_t B, int64_t M, int64_t P,
                                    int page, int cp, int shard, int interleave, int32_t* tables_out,
                                    int32_t* refs_out, int32_t* copies, int32_t* missing, void* workspace,
                                    int64_t workspace_bytes, void* stream) {
    if (!sizes_ok(B, M, P)) return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    const int lg = page_log2_of(page);
    if (lg < 0) return DCP_MLA_CACHE8_ERR_BAD_PAGE;
    if (M * page > 0x7fffffff) return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    if (cp < 1 || cp > DCP_MLA_CACHE8_CP_MAX || shard < 0 || shard >= cp || interleave < 1 || interleave > 1 << 24)
        return DCP_MLA_CACHE8_ERR_BAD_CP;
    if (refs == nullptr || refs_out == nullptr || missing == nullptr ||
        (B > 0 && (tables == nullptr || tables_out == nullptr || parents == nullptr || keeps == nullptr ||
                   wants == nullptr || copies == nullptr)))
        return DCP_MLA_CACHE8_ERR_NULL_POINTER;
    if (!aligned(tables, 4) || !aligned(refs, 4) || !aligned(parents, 4) || !aligned(keeps, 4) || !aligned(wants, 4) ||
        !aligned(tables_out, 4) || !aligned(refs_out, 4) || !aligned(copies, 8) || !aligned(missing, 4))
        return DCP_MLA_CACHE8_ERR_MISALIGNED;
    if (check_alias(tables, refs, tables_out, refs_out, B * M, P)) return DCP_MLA_CACHE8_ERR_ALIAS;
    const bool in_place = refs == refs_out;
    const UpdateSpace ws = update_space(B, M, P, in_place);
    if (ws.bytes > 0 && (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < ws.bytes))
        return DCP_MLA_CACHE8_ERR_WORKSPACE;
    // (parents and positions are read to the end of the call, and address what is written)
    const Span t = {tables, B * M * 4}, r = {refs, P * 4}, to = {tables_out, B * M * 4}, ro = {refs_out, P * 4},
               parent = {parents, B * 4}, keep = {keeps, B * 4}, want = {wants, B * 4};
    if (meet({{copies, B * 8}, {missing, 4}, {workspace, ws.bytes}}, {t, r, to, ro, parent, keep, want}) ||
        meet({to, ro}, {parent, keep, want}))
        return DCP_MLA_CACHE8_ERR_ALIAS;
    uint8_t* const w = static_cast<uint8_t*>(workspace);
    UpdateParams p;
    p.tables = tables;
    p.refs = refs;
    p.parents = parents;
    p.keeps = keeps;
    p.wants = wants;
    p.tables_out = tables_out;
    p.refs_out = refs_out;
    p.copies = copies;
    p.missing = missing;
    p.plan = reinterpret_cast<RowPlan*>(w + ws.plan);
    p.pool = {reinterpret_cast<int*>(w + ws.held), reinterpret_cast<int2*>(w + ws.writers),
              reinterpret_cast<uint32_t*>(w + ws.free), reinterpret_cast<int*>(w + ws.before)};
    p.staged = reinterpret_cast<int*>(w + ws.staged);
    p.M = (int)M;
    p.B = (int)B;
    p.P = (int)P;
    p.page_log2 = lg;
    p.in_place = in_place;
    p.cp = cp;
    p.shard = shard;
    p.interleave = interleave;
    const int ctas = cluster_of(B, B * M, P);
    p.part_log2 = part_log2_of(P, ctas);
    const int64_t own = (int64_t)kWarps << p.part_log2;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return own <= kPagesShared ? launch_update<true>(p, ctas, (int)(own / 32 * (12 * 32 + 8)), st)
                               : launch_update<false>(p, ctas, 0, st);
}

extern "C" int dcp_mla_pages_compact(const int32_t* tables, const int32_t* refs, int64_t B, int64_t M, int64_t P,
                                     int32_t* tables_out, int32_t* refs_out, int32_t* copies, void* workspace,
                                     int64_t workspace_bytes, void* stream) {
    if (!sizes_ok(B, M, P)) return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    if (refs == nullptr || refs_out == nullptr || (B > 0 && (tables == nullptr || tables_out == nullptr)) ||
        (P > 1 && copies == nullptr))
        return DCP_MLA_CACHE8_ERR_NULL_POINTER;
    if (!aligned(tables, 4) || !aligned(refs, 4) || !aligned(tables_out, 4) || !aligned(refs_out, 4) ||
        !aligned(copies, 8))
        return DCP_MLA_CACHE8_ERR_MISALIGNED;
    if (check_alias(tables, refs, tables_out, refs_out, B * M, P)) return DCP_MLA_CACHE8_ERR_ALIAS;
    const CompactSpace ws = compact_space(P);
    if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < ws.bytes)
        return DCP_MLA_CACHE8_ERR_WORKSPACE;
    if (meet({{copies, P / 2 * 8}, {workspace, ws.bytes}},
             {{tables, B * M * 4}, {refs, P * 4}, {tables_out, B * M * 4}, {refs_out, P * 4}}))
        return DCP_MLA_CACHE8_ERR_ALIAS;
    uint8_t* const w = static_cast<uint8_t*>(workspace);
    CompactParams p;
    p.tables = tables;
    p.refs = refs;
    p.tables_out = tables_out;
    p.refs_out = refs_out;
    p.copies = copies;
    p.bits = reinterpret_cast<uint32_t*>(w + ws.bits);
    p.before = reinterpret_cast<int*>(w + ws.before);
    p.chunks = reinterpret_cast<int*>(w + ws.chunks);
    p.entries = B * M;
    p.P = (int)P;
    p.in_place = refs == refs_out;
    p.words = (int)((P + 31) / 32);
    // at most kChunksMax chunks of whole words, a word a warp where that is enough
    const int k = log2_up((p.words + kChunksMax - 1) / kChunksMax);
    p.chunk_log2 = k < 5 ? 5 : k;
    p.chunk_count = ((p.words - 1) >> p.chunk_log2) + 1;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    census_kernel<<<p.chunk_count, kThreads, 0, st>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return (int)e;
    // the second launch begins beside the first and waits for it on the device
    const int64_t work = (P > p.entries ? P : p.entries), want = (work + kMoveThreads - 1) / kMoveThreads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(want < 4 * kSms ? want : 4 * kSms));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = p.words <= kWordsShared ? (size_t)p.words * 8 : 0;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, move_kernel, p);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return (int)e;
}

extern "C" int dcp_mla_pages_copy(void* const* kv_ptrs, float* const* scale_ptrs, int pools, int64_t P, int page,
                                  int Dk, int block, const int32_t* copies, int64_t n, void* stream) {
    if (n < 0 || n > 0x7fffffff || P < 1 || P > 0x7fffffff || (Dk != 512 && Dk != 576) || pools < 1 ||
        pools > DCP_MLA_PAGES_POOLS_MAX)
        return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    if (block < 1 || block > DCP_MLA_CACHE8_BLOCK_MAX || (block & (block - 1)) != 0)
        return DCP_MLA_CACHE8_ERR_BAD_BLOCK;
    if (page_log2_of(page) < 0 || page % block != 0) return DCP_MLA_CACHE8_ERR_BAD_PAGE;
    if (kv_ptrs == nullptr || scale_ptrs == nullptr || (n > 0 && copies == nullptr))
        return DCP_MLA_CACHE8_ERR_NULL_POINTER;
    CopyParams p;
    for (int j = 0; j < pools; ++j) {
        if (kv_ptrs[j] == nullptr || scale_ptrs[j] == nullptr) return DCP_MLA_CACHE8_ERR_NULL_POINTER;
        if (!aligned(kv_ptrs[j], 16) || !aligned(scale_ptrs[j], 4)) return DCP_MLA_CACHE8_ERR_MISALIGNED;
        for (int k = 0; k < j; ++k)  // (what two pools have in common would be written by two CTAs)
            if (overlap(kv_ptrs[j], P * page * Dk, kv_ptrs[k], P * page * Dk) ||
                overlap(scale_ptrs[j], P * (page / block) * 4, scale_ptrs[k], P * (page / block) * 4))
                return DCP_MLA_CACHE8_ERR_ALIAS;
        p.kv[j] = static_cast<uint8_t*>(kv_ptrs[j]);
        p.scales[j] = scale_ptrs[j];
    }
    if (!aligned(copies, 8)) return DCP_MLA_CACHE8_ERR_MISALIGNED;
    if (n == 0) return 0;
    p.copies = reinterpret_cast<const int2*>(copies);
    p.page_bytes = (int64_t)page * Dk;
    p.P = (int)P;
    p.scale_words = page / block;
    p.parts = (int)((p.page_bytes + kCopyThreads * kCopyVecs * 16 - 1) / (kCopyThreads * kCopyVecs * 16));
    if (n * p.parts > 0x7fffffff) return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    copy_kernel<<<dim3((unsigned)(n * p.parts), (unsigned)pools), kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : (int)e;
}
