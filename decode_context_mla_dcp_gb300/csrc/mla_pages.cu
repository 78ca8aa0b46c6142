// Pages of the 8-bit latent cache, sm_103a: the step of the tables (fork, cut, end,
// grow), the compaction of a pool and the copying of pages. What they do is stated
// in include/dcp_mla_pages.h.
//
// Tables and counts are a few KB to a few MB, and every decision depends on all
// rows: one cluster of CTAs does a call, in phases between cluster barriers, so that
// a call is one launch and no count leaves the device. Sums over rows and over the
// pool give every row and every free page its rank, so nothing depends on the order
// in which CTAs or atomics come (atomics here are sums and maxima of integers).
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dcp_lse_reduce.h"
#include "dcp_mla_pages.h"

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kClusterMax = 8;
constexpr int kUnits = 8;  // entries of a lane in flight

// What phases leave for one another is read past L1: a line there may be older than the barrier.
__device__ __forceinline__ int fresh_load(const int* p) { return __ldcg(p); }

__device__ __forceinline__ int lane_sums(int x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// A shard's share of the first L positions.
__device__ __forceinline__ int64_t share_of(int64_t L, int64_t cp, int64_t shard, int64_t interleave) {
    if (L <= 0) return 0;
    if (cp == 1) return L;
    const int64_t round = cp * interleave, q = L / round;
    int64_t r = L - q * round - shard * interleave;
    r = r < 0 ? 0 : (r > interleave ? interleave : r);
    return q * interleave + r;
}

// ---- the step of the tables ------------------------------------------------------

struct alignas(16) RowPlan {
    int taken;  // pages that it takes over
    int pages;  // pages that it has afterwards
    int last;   // the page that it is about to write behind kept tokens, or -1
};

struct UpdateParams {
    const int *tables, *refs, *parents, *keeps, *wants;
    int *tables_out, *refs_out, *copies, *missing;
    RowPlan* plan;    // [B]
    int2* deal;       // [B] rank of the row's first fresh page among its CTA's; whether `last` is copied
    int *writers, *latest;  // [P], where some row has it as `last`: rows that do, the last of them
    int* fresh;       // [P] free pages by rank
    int* staged;      // [B, M] pages taken over from another row (in place)
    int* sums;        // [2][kClusterMax] fresh pages that a CTA's rows need; free pages of its part
    int64_t M;
    int B, P, page_log2, in_place;
    int cp, shard, interleave;
};

// Exclusive sum of x over the CTA's threads; *all the CTA's sum.
__device__ __forceinline__ int block_sums(int x, int* warp_s, int* all) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int incl = lane_sums(x, lane);
    __syncthreads();
    if (lane == 31) warp_s[warp] = incl;
    __syncthreads();
    const int w = warp_s[lane];  // (kWarps = 32)
    *all = __reduce_add_sync(0xffffffffu, w);
    return incl - x + __reduce_add_sync(0xffffffffu, lane < warp ? w : 0);
}

// Entries of [lo, hi) that `is` holds for, counted by warps over contiguous parts.
template <class F>
__device__ __forceinline__ int count_part(int64_t lo, int64_t hi, F is) {
    const int lane = threadIdx.x & 31;
    int n = 0;
    for (int64_t i = lo + lane; i < hi; i += 32 * kUnits) {
#pragma unroll
        for (int u = 0; u < kUnits; ++u)
            if (i + 32 * u < hi && is(i + 32 * u)) ++n;
    }
    return __reduce_add_sync(0xffffffffu, n);
}
// The same entries in order: put(rank, entry) from rank `at` on, below `end`.
template <class F, class G>
__device__ __forceinline__ void list_part(int64_t lo, int64_t hi, int64_t at, int64_t end, F is, G put) {
    const int lane = threadIdx.x & 31;
    for (int64_t i0 = lo; i0 < hi && at < end; i0 += 32 * kUnits) {
        bool here[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) here[u] = i0 + 32 * u + lane < hi && is(i0 + 32 * u + lane);
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const uint32_t m = __ballot_sync(0xffffffffu, here[u]);
            const int64_t rank = at + __popc(m & ((1u << lane) - 1));
            if (here[u] && rank < end) put(rank, i0 + 32 * u + lane);
            at += __popc(m);
        }
    }
}

__global__ void __launch_bounds__(kThreads) update_kernel(const __grid_constant__ UpdateParams p) {
    __shared__ int warp_s[kWarps], free_s[kWarps];
    const cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ctas = (int)gridDim.x, cta = (int)blockIdx.x;
    const int rows = (p.B + ctas - 1) / ctas, row0 = cta * rows, row1 = row0 + rows < p.B ? row0 + rows : p.B;
    // this warp's part of the pool
    const int64_t part = ((int64_t)p.P + ctas * kWarps - 1) / (ctas * kWarps);
    int64_t lo = (cta * kWarps + warp) * part, hi = lo + part;
    lo = lo < p.P ? lo : p.P;
    hi = hi < p.P ? hi : p.P;

    if (!p.in_place) {
        for (int64_t i = lo + lane; i < hi; i += 32) p.refs_out[i] = p.refs[i];
        cluster.sync();
    }
    // ---- what each row takes over, and the counts of pages that change hands
    const int64_t room = p.M << p.page_log2;
    for (int b = row0 + warp; b < row1; b += kWarps) {
        const int from = p.parents[b];
        const bool some = from >= 0 && from < p.B, self = from == b;
        int64_t keep = some ? share_of(p.keeps[b], p.cp, p.shard, p.interleave) : 0;
        int64_t want = share_of(p.wants[b], p.cp, p.shard, p.interleave);
        keep = keep < room ? keep : room;
        want = want < room ? want : room;
        const int64_t page_up = (1ll << p.page_log2) - 1;
        const int n_keep = (int)((keep + page_up) >> p.page_log2), n_want = (int)((want + page_up) >> p.page_log2);
        const int at = want > keep && (keep & page_up) ? (int)(keep >> p.page_log2) : -1;
        const int* const mine = p.tables + b * p.M;
        const int* const theirs = p.tables + (some ? from : b) * p.M;
        int taken = 0, last = -1;
        bool more_mine = true, more_theirs = n_keep > 0;
        for (int64_t i0 = 0; i0 < p.M && (more_mine || more_theirs); i0 += 32 * kUnits) {
            int e[kUnits], f[kUnits];
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const int64_t i = i0 + 32 * u + lane;
                e[u] = more_mine && i < p.M ? mine[i] : -1;
                f[u] = !self && more_theirs && i < n_keep ? theirs[i] : -1;
            }
#pragma unroll
            for (int u = 0; u < kUnits; ++u) {
                const int64_t i = i0 + 32 * u + lane;
                const uint32_t bad = __ballot_sync(0xffffffffu, !(e[u] >= 0 && e[u] < p.P));
                const int good = bad ? __ffs(bad) - 1 : 32;
                if (!more_mine || lane >= good) e[u] = -1;
                more_mine = more_mine && good == 32;
                if (self) {
                    f[u] = i < n_keep ? e[u] : -1;
                } else {
                    const uint32_t no = __ballot_sync(0xffffffffu, !(f[u] >= 0 && f[u] < p.P));
                    const int ok = no ? __ffs(no) - 1 : 32;
                    if (!more_theirs || lane >= ok) f[u] = -1;
                    more_theirs = more_theirs && ok == 32;
                }
                taken += __popc(__ballot_sync(0xffffffffu, f[u] >= 0));
                if (i == at) last = f[u];
                if (e[u] != f[u]) {
                    if (e[u] >= 0) atomicSub(p.refs_out + e[u], 1);
                    if (f[u] >= 0) atomicAdd(p.refs_out + f[u], 1);
                }
                if (i < p.M) {
                    if (!p.in_place) p.tables_out[b * p.M + i] = f[u];
                    else if (!self && f[u] >= 0) p.staged[b * p.M + i] = f[u];
                }
            }
            if (self) more_theirs = more_mine && i0 + 32 * kUnits < n_keep;
            if (!p.in_place && !more_mine && !more_theirs)  // the rest of the row has no pages
                for (int64_t i = i0 + 32 * kUnits + lane; i < p.M; i += 32) p.tables_out[b * p.M + i] = -1;
        }
        last = __reduce_max_sync(0xffffffffu, last);
        if (lane == 0) {
            p.plan[b] = {taken, n_keep > n_want ? n_keep : n_want, last};
            if (last >= 0) {
                p.writers[last] = 0;
                p.latest[last] = -1;
            }
        }
    }
    cluster.sync();
    // ---- who is about to write which page
    for (int b = row0 + tid; b < row1; b += kThreads) {
        const int last = fresh_load(&p.plan[b].last);
        if (last >= 0) {
            atomicAdd(p.writers + last, 1);
            atomicMax(p.latest + last, b);
        }
    }
    cluster.sync();
    // ---- how many fresh pages each row needs, and how many there are
    int need_all = 0;
    for (int b0 = row0; b0 < row1; b0 += kThreads) {
        const int b = b0 + tid;
        int need = 0, copied = 0;
        if (b < row1) {
            const int4 w = __ldcg(reinterpret_cast<const int4*>(p.plan + b));
            if (w.z >= 0)
                copied = fresh_load(p.writers + w.z) < fresh_load(p.refs_out + w.z) || fresh_load(p.latest + w.z) != b;
            need = copied + w.y - w.x;
        }
        int all;
        const int before = block_sums(need, warp_s, &all);
        if (b < row1) p.deal[b] = make_int2(need_all + before, copied);
        need_all += all;
    }
    const auto is_free = [&](int64_t i) { return fresh_load(p.refs_out + i) == 0; };
    const int n_free = count_part(lo, hi, is_free);
    if (lane == 0) free_s[warp] = n_free;
    __syncthreads();
    const int mine_free = free_s[lane];
    if (tid == 0) p.sums[cta] = need_all;
    if (warp == 0) {
        const int all = __reduce_add_sync(0xffffffffu, mine_free);
        if (lane == 0) p.sums[kClusterMax + cta] = all;
    }
    cluster.sync();
    // ---- the free pages that are dealt, by rank
    int64_t need_total = 0, free_total = 0, need_before = 0, free_before = 0;
    for (int c = 0; c < ctas; ++c) {
        const int n = fresh_load(p.sums + c), f = fresh_load(p.sums + kClusterMax + c);
        if (c < cta) {
            need_before += n;
            free_before += f;
        }
        need_total += n;
        free_total += f;
    }
    list_part(lo, hi, free_before + __reduce_add_sync(0xffffffffu, lane < warp ? mine_free : 0), need_total, is_free,
              [&](int64_t rank, int64_t i) { p.fresh[rank] = (int)i; });
    // (a page that is copied has another holder: its count stays above 0)
    for (int b = row0 + tid; b < row1; b += kThreads)
        if (p.deal[b].y) atomicSub(p.refs_out + fresh_load(&p.plan[b].last), 1);
    if (cta == 0 && tid == 0) *p.missing = need_total > free_total ? (int)(need_total - free_total) : 0;
    cluster.sync();
    // ---- the rows' new entries
    for (int b = row0 + warp; b < row1; b += kWarps) {
        const int4 w = __ldcg(reinterpret_cast<const int4*>(p.plan + b));
        const int2 deal = __ldcg(p.deal + b);
        int* const row = p.tables_out + b * p.M;
        int64_t rank = need_before + deal.x;
        if (p.in_place) {
            if (p.parents[b] != b)
                for (int i = lane; i < w.x; i += 32) row[i] = fresh_load(p.staged + b * p.M + i);
            for (int64_t i = w.y + lane; i < p.M; i += 32) row[i] = -1;  // (whatever stood behind the row's pages)
            __syncwarp();
        }
        if (deal.y) {
            const int got = rank < free_total ? fresh_load(p.fresh + rank) : -1;
            ++rank;
            if (lane == 0) {
                const int64_t keep = share_of(p.keeps[b], p.cp, p.shard, p.interleave);
                row[keep >> p.page_log2] = got;
                if (got >= 0) p.refs_out[got] = 1;
                reinterpret_cast<int2*>(p.copies)[b] = got >= 0 ? make_int2(w.z, got) : make_int2(-1, -1);
            }
        } else if (lane == 0) {
            reinterpret_cast<int2*>(p.copies)[b] = make_int2(-1, -1);
        }
        for (int i = w.x + lane; i < w.y; i += 32) {
            const int64_t r = rank + (i - w.x);
            const int got = r < free_total ? fresh_load(p.fresh + r) : -1;
            row[i] = got;
            if (got >= 0) p.refs_out[got] = 1;
        }
    }
}

// ---- compaction --------------------------------------------------------------------

struct CompactParams {
    const int *tables, *refs;
    int *tables_out, *refs_out, *copies;
    int* to;                // [P] where a page at n or beyond goes
    int *movers, *holes;    // [P / 2] by rank
    int* sums;              // [3][kClusterMax]
    int64_t entries;        // B x M
    int P, in_place;
};

__global__ void __launch_bounds__(kThreads) compact_kernel(const __grid_constant__ CompactParams p) {
    __shared__ int hole_s[kWarps], mover_s[kWarps], warp_s[kWarps];
    const cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ctas = (int)gridDim.x, cta = (int)blockIdx.x;
    const int64_t part = ((int64_t)p.P + ctas * kWarps - 1) / (ctas * kWarps);
    int64_t lo = (cta * kWarps + warp) * part, hi = lo + part;
    lo = lo < p.P ? lo : p.P;
    hi = hi < p.P ? hi : p.P;
    // ---- pages in use
    const int live = count_part(lo, hi, [&](int64_t i) { return p.refs[i] > 0; });
    if (!p.in_place)
        for (int64_t i = lo + lane; i < hi; i += 32) p.refs_out[i] = p.refs[i];
    if (lane == 0) warp_s[warp] = live;
    __syncthreads();
    if (warp == 0) {
        const int all = __reduce_add_sync(0xffffffffu, warp_s[lane]);
        if (lane == 0) p.sums[cta] = all;
    }
    cluster.sync();
    int64_t n = 0;
    for (int c = 0; c < ctas; ++c) n += fresh_load(p.sums + c);
    // ---- free ones below n, used ones from n on: as many of the one as of the other
    const auto is_hole = [&](int64_t i) { return i < n && p.refs[i] <= 0; };
    const auto is_mover = [&](int64_t i) { return i >= n && p.refs[i] > 0; };
    const int holes = count_part(lo, hi < n ? hi : n, is_hole), movers = count_part(lo > n ? lo : n, hi, is_mover);
    if (lane == 0) {
        hole_s[warp] = holes;
        mover_s[warp] = movers;
    }
    __syncthreads();
    const int my_holes = hole_s[lane], my_movers = mover_s[lane];
    if (warp == 0) {
        const int a = __reduce_add_sync(0xffffffffu, my_holes), z = __reduce_add_sync(0xffffffffu, my_movers);
        if (lane == 0) {
            p.sums[kClusterMax + cta] = a;
            p.sums[2 * kClusterMax + cta] = z;
        }
    }
    cluster.sync();
    int64_t hole_at = 0, mover_at = 0, moves = 0;
    for (int c = 0; c < ctas; ++c) {
        const int a = fresh_load(p.sums + kClusterMax + c), z = fresh_load(p.sums + 2 * kClusterMax + c);
        if (c < cta) {
            hole_at += a;
            mover_at += z;
        }
        moves += z;
    }
    hole_at += __reduce_add_sync(0xffffffffu, lane < warp ? my_holes : 0);
    mover_at += __reduce_add_sync(0xffffffffu, lane < warp ? my_movers : 0);
    list_part(lo, hi < n ? hi : n, hole_at, moves, is_hole, [&](int64_t r, int64_t i) { p.holes[r] = (int)i; });
    list_part(lo > n ? lo : n, hi, mover_at, moves, is_mover, [&](int64_t r, int64_t i) { p.movers[r] = (int)i; });
    for (int64_t i = (lo > n ? lo : n) + lane; i < hi; i += 32) p.to[i] = (int)i;
    cluster.sync();
    // ---- the moves
    const int64_t threads = (int64_t)ctas * kThreads, me = (int64_t)cta * kThreads + tid;
    for (int64_t i = me; i < p.P / 2; i += threads) {
        int2 c = make_int2(-1, -1);
        if (i < moves) {
            c = make_int2(fresh_load(p.movers + i), fresh_load(p.holes + i));
            p.to[c.x] = c.y;
            p.refs_out[c.y] = p.in_place ? fresh_load(p.refs + c.x) : p.refs[c.x];
            p.refs_out[c.x] = 0;
        }
        reinterpret_cast<int2*>(p.copies)[i] = c;
    }
    cluster.sync();
    for (int64_t i0 = me; i0 < p.entries; i0 += kUnits * threads) {
        int e[kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) e[u] = i0 + u * threads < p.entries ? p.tables[i0 + u * threads] : -1;
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            if (i0 + u * threads >= p.entries) continue;
            const bool goes = e[u] >= n && e[u] < p.P;
            const int to = goes ? fresh_load(p.to + e[u]) : e[u];
            if (!p.in_place || to != e[u]) p.tables_out[i0 + u * threads] = to;
        }
    }
}

// ---- copying pages --------------------------------------------------------------------

struct CopyParams {
    uint8_t* kv[DCP_MLA_PAGES_POOLS_MAX];
    float* scales[DCP_MLA_PAGES_POOLS_MAX];
    const int2* copies;
    int64_t n, page_bytes;
    int P, scale_words, parts;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 9;  // 16-byte pieces of a thread: a part is 36 KiB, a page of 64 tokens

// A CTA copies a part of a page of one pool, every load in flight before the first store.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyParams p) {
    const int part = (int)(blockIdx.x % (unsigned)p.parts);
    const int64_t i = blockIdx.x / (unsigned)p.parts;
    const int2 c = p.copies[i];
    if (c.x < 0 || c.x >= p.P || c.y < 0 || c.y >= p.P) return;
    const int64_t at = (int64_t)part * (kCopyThreads * kCopyVecs * 16);
    const int64_t bytes = p.page_bytes - at;
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
        if (j * 16 < bytes) dst[j] = v[k];
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
bool sizes_ok(int64_t B, int64_t M, int64_t P) {
    return B >= 0 && B <= 65535 && M >= 1 && M < 0x7fffffff && B * (M + 1) <= 0x7fffffff && P >= 1 && P <= 0x7fffffff;
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

struct UpdateSpace {
    int64_t plan, deal, writers, latest, fresh, sums, staged, bytes;
};
UpdateSpace update_space(int64_t B, int64_t M, int64_t P, bool in_place) {
    UpdateSpace w;
    w.plan = 0;
    w.deal = w.plan + round_up(B * 16);
    w.writers = w.deal + round_up(B * 8);
    w.latest = w.writers + round_up(P * 4);
    w.fresh = w.latest + round_up(P * 4);
    w.sums = w.fresh + round_up(P * 4);
    w.staged = w.sums + 256;
    w.bytes = w.staged + (in_place ? round_up(B * M * 4) : 0);
    return w;
}
struct CompactSpace {
    int64_t to, movers, holes, sums, bytes;
};
CompactSpace compact_space(int64_t P) {
    CompactSpace w;
    w.to = 0;
    w.movers = w.to + round_up(P * 4);
    w.holes = w.movers + round_up(P / 2 * 4);
    w.sums = w.holes + round_up(P / 2 * 4);
    w.bytes = w.sums + 256;
    return w;
}

template <class K, class P>
int launch_cluster(K kernel, const P& p, int ctas, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
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
    if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < ws.bytes)
        return DCP_MLA_CACHE8_ERR_WORKSPACE;
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
    p.deal = reinterpret_cast<int2*>(w + ws.deal);
    p.writers = reinterpret_cast<int*>(w + ws.writers);
    p.latest = reinterpret_cast<int*>(w + ws.latest);
    p.fresh = reinterpret_cast<int*>(w + ws.fresh);
    p.sums = reinterpret_cast<int*>(w + ws.sums);
    p.staged = reinterpret_cast<int*>(w + ws.staged);
    p.M = M;
    p.B = (int)B;
    p.P = (int)P;
    p.page_log2 = lg;
    p.in_place = in_place;
    p.cp = cp;
    p.shard = shard;
    p.interleave = interleave;
    return launch_cluster(update_kernel, p, kClusterMax, static_cast<cudaStream_t>(stream));
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
    uint8_t* const w = static_cast<uint8_t*>(workspace);
    CompactParams p;
    p.tables = tables;
    p.refs = refs;
    p.tables_out = tables_out;
    p.refs_out = refs_out;
    p.copies = copies;
    p.to = reinterpret_cast<int*>(w + ws.to);
    p.movers = reinterpret_cast<int*>(w + ws.movers);
    p.holes = reinterpret_cast<int*>(w + ws.holes);
    p.sums = reinterpret_cast<int*>(w + ws.sums);
    p.entries = B * M;
    p.P = (int)P;
    p.in_place = refs == refs_out;
    return launch_cluster(compact_kernel, p, kClusterMax, static_cast<cudaStream_t>(stream));
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
        for (int k = 0; k < j; ++k)  // (a pool that came twice would be written by two CTAs)
            if (kv_ptrs[j] == kv_ptrs[k] || scale_ptrs[j] == scale_ptrs[k]) return DCP_MLA_CACHE8_ERR_ALIAS;
        p.kv[j] = static_cast<uint8_t*>(kv_ptrs[j]);
        p.scales[j] = scale_ptrs[j];
    }
    if (!aligned(copies, 8)) return DCP_MLA_CACHE8_ERR_MISALIGNED;
    if (n == 0) return 0;
    p.copies = reinterpret_cast<const int2*>(copies);
    p.n = n;
    p.page_bytes = (int64_t)page * Dk;
    p.P = (int)P;
    p.scale_words = page / block;
    p.parts = (int)((p.page_bytes + kCopyThreads * kCopyVecs * 16 - 1) / (kCopyThreads * kCopyVecs * 16));
    if (n * p.parts > 0x7fffffff) return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    copy_kernel<<<dim3((unsigned)(n * p.parts), (unsigned)pools), kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : (int)e;
}
