// Single-token MLA attention over the 8-bit latent cache, in rows or in pages,
// sm_103a. What it computes is stated in include/dcp_mla_cache8.h and
// include/dcp_mla_pages.h.
//
// The mathematics. A tile is 128 cached tokens; the cached e4m3 codes go to the
// tensor cores as they lie in the cache. With c_t = scale * log2(e) * (scale of
// token t's block), u_t = that block's scale, and codes k_t:
//   scores, in base-2 units   s[t, h] = c_t <q_h, k_t>
//   values                    O[d, h] = sum_t 2^(s[t, h] - M_h) u_t k_t[d]
//   sums                      l[h]    = sum_t 2^(s[t, h] - M_h)
//   out = O / l, lse = M + log2 l
// * q (bf16) is two e4m3 numbers at a power-of-two scale per head, q = hi + lo:
//   8 significand bits are two of 4, so the split is exact where nothing falls
//   below e4m3's subnormals. Both parts are rows of one B operand, so the pair
//   costs what N = 2 x heads costs, and the sums add in fp32 registers.
// * The probabilities times u_t are split into hi + lo the same way. A fixed
//   scale would lose small probabilities (e4m3 spans 2^17), so each head has its
//   own power-of-two scale for each 32 tokens: with E the 32 tokens' largest
//   s + log2 u, rounded to an integer, P = 2^(s + log2 u - E + 8) in (0, 2^8.5],
//   and the tensor core multiplies by 2^(E - M - 8) (block-scaled e4m3, one ue8m0
//   scale for 32 products). What a token of 2^-14 of its block's largest loses is
//   below 2^-18 of that largest; the rest is exact to 2^-8, like bf16
//   probabilities. P itself does not depend on M.
// * The reference M is an integer per head. It begins at 0 and moves only when
//   some E exceeds it by 32, or when a segment's first ones lie 60 below it: fp32
//   sums bear both. Most segments never move it, and a move rewrites O in TMEM.
//
// Layout. The product is transposed so that the 128 tokens lie on the MMA's M:
//   S^T[128 tokens x 2 parts of the heads] = K_tile . Q^T      (18 MMAs of K = 32)
//   O^T[512 dims x heads]                 += V_tile^T . P^T    (4 row blocks)
// The cached tile serves both products: K-major for the scores, M-major (read
// along the latent dims) for the values. P lies as the softmax threads have it, a
// token's heads side by side, and is read along the heads (N-major), so that no
// bytes change lanes (153.2 -> 149.7 us against a transpose by shuffles, 64 ragged
// rows x 16K x 128 heads).
//
// What bounds it. A CTA has up to 64 heads: 2 x 64 x (576 + 512) x 2 operations a
// token (q's and P's two parts) against 576 bytes, so with 64 heads and more it is
// the tensor cores and what feeds them, with 16 the cache's way from DRAM. A tile
// of 64 heads takes some 3,800 cycles at the 1.94 GHz that the call runs at. Its MMAs
// alone take 2,958 (1,393 the scores, N = 128; 1,565 the values: N = 64 costs 55
// to 59 cycles and N = 128 77, so both parts of P go into one MMA where TMEM has room
// for them, the first 128 dims). Shared memory's port serves them all: the operands
// take 2,150 of its cycles a tile, the tile itself 580, the softmax some 900. Two
// tiles, q and P fill shared memory, S, O and the scales TMEM (456 of 512 columns), so
// there is no third stage and one CTA a multiprocessor. By the clock of the MMA warp a
// tile's turn is 930 cycles to issue the scores and 1,460 the values; the others are
// waits, each some 100 to 300: for P, for slices, for the scores' place, for what comes.
//   measured, 128 heads: 64 ragged rows of up to 16K tokens 119 to 138 us with their
//   lengths (six sets of 465,318 to 547,763 tokens), 251 to 260 us for 10^6 tokens, 512
//   wide 111 to 128 and 232 to 242; 8 rows x 4096 tokens 22.6 to 22.9 us, of which 16
//   are the main kernel (4 tiles a CTA between 10,000 cycles to begin and 6,000 to
//   end) and 6 the join; 16 heads, 200 tokens: 8.1 to 8.5 us. One shard of 8 held, 8 rows x
//   4096 of its tokens: 24.3 us.
// With 16 and 32 heads 64 ragged rows x 16K take 60 and 62 us against 45 of their
// bytes: some 16 us are the beginning, the end and the join, and the MMA warp's turn
// (46 cycles an MMA whatever its N, and the waits between) is near the rest.
//
// Pages. A tile is 128 tokens at a multiple of 128, from 1 to 4 pages: a TMA box a page
// into the tile's place (the swizzle goes by address, so that the tile is the same), and
// zeros where there is no page. The loading warps bring the tile's page numbers with its
// description; a token without a page is masked like one that is not visible. One bulk
// request a page brings the tile after next to L2. 64 ragged rows x 16K x 128 heads take
// 124 us in pages of 64 and 123 in pages of 128, the same lengths in rows 119.5 (six sets
// of lengths: pages of 64 cost 4 to 5% more than rows).
//
// Groups. Rows that share a prefix have their heads side by side in blocks of 64 over
// the prefix's tiles, so that 16 heads a row cost a quarter of the tiles' turns; what a
// row has behind the prefix, whole tiles of which are the prefix's, is a line of its own,
// and the join weighs both. 64 rows of 16 heads behind two prefixes of 16K with up to
// 1,024 tokens of their own: 55.6 us, 101 without groups; 64 rows of 16 heads behind 128
// shared tokens with up to 16K of their own 94 us, 66 without; floor of the first 20 (the products at the
// bf16 rate). Bound as above, at 2.0 us a tile: 2,464 tiles and changes of line are 16 a
// CTA, 33 us of it, and the beginning, the end and the join are the rest.
//
// Rounding to fewer bits: q's and P's parts as above. log2 u, exp2 and the division by u
// are the hardware's (two units of the last place, 2^-22, two units), far below P's
// 2^-8; the sums are those of the P that is not rounded yet, in fp32.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stddef.h>
#include <math.h>
#include <stdint.h>

#include "dcp_lse_reduce.h"
#include "dcp_mla_cache8.h"
#include "dcp_mla_decode.h"
#include "dcp_mla_pages.h"

namespace {

constexpr int kDv = 512;
constexpr int kTile = 128;                 // tokens of a tile: the MMA's M
constexpr int kSlice = kTile * 128;        // bytes of a 128-dim slice of a tile
constexpr int kSoftWarps = 16, kSoftThreads = 32 * kSoftWarps;
constexpr int kLoadWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
// Three warps load: the first slice, the next two, and the last with the rope slice (the second and third warp stand behind
// the MMA warp). A request takes its warp some 150 cycles, a tile has 5 of them, in pages up to 20, and a slice's place is
// free only shortly before its next tokens are wanted. (A fourth would leave 80 registers a thread. 64 ragged rows x 16K x
// 128 heads, when this was changed: rows 130.5 us with one, 119.5 with three; in pages of 32, 64, 128 tokens 157, 147 and
// 141, and 132, 129, 128.)
constexpr int kThreads = kSoftThreads + 128;
constexpr int kCpMax = DCP_MLA_CACHE8_CP_MAX;
constexpr int64_t kMaxInterleave = 1 << 24;
constexpr long long kWaitLimitNs = 2000000000LL;  // every wait gives up after this,
constexpr long long kTestWaitLimitNs = 20000000LL;  // or after this, with DCP_MLA_FLAG_TEST_STALL
constexpr int kLazy = 32;                  // how far an exponent may pass the reference
constexpr int kLow = 60;                   // how far below it a segment's first ones may lie

// The kernel's parameters but for what there is one of per shard. Those come in
// room for 1, 4 or 16 shards: a launch copies its parameters, and with one shard
// the compiler drops the arithmetic of several.
struct DecodeBase {
    const uint8_t* q;
    int64_t q_row, q_head;                 // bytes
    int q_wide;                            // q can be read 16 bytes at a time
    const int* seq_lens;
    float* part;                           // [2 x CTAs][heads of a block][512], normalised
    float* part_lse;                       // [2 x CTAs][heads of a block], base 2
    int2* row_info;                        // [B] a row's first range of CTAs and its segments
    uint8_t* out;
    float* lse;
    int* status;
    int64_t blocks;                        // scales of a row
    uint32_t held;                         // bit j: shard j is held
    uint32_t T, cp, interleave, window, sinks;
    int block_log2;
    int B, H, head_blocks, ranges;         // grid: head_blocks x ranges CTAs
    int row_mode;                          // a range is whole rows (no row is split)
    float scale_log2;
    float lse_scale;                       // ln 2 for a natural-log LSE, 1 for base 2
    long long wait_ns;
    int stall;                             // DCP_MLA_FLAG_TEST_STALL: a CTA's first slice waits for 16 bytes more
};
template <int kShards>
struct DecodeParams : DecodeBase {
    static constexpr bool kPaged = false;
    CUtensorMap tm_latent[kShards];        // boxes of 128 dims x 128 tokens, 128-byte swizzle
    CUtensorMap tm_rope[kShards];          // boxes of 64 dims x 128 tokens, 64-byte swizzle
    const float* scales[kShards];
    __device__ __forceinline__ uint32_t shards() const { return kShards == 1 ? 1u : cp; }
};
// A cache in pages (the maps are [P, page, Dk], their boxes a page's tokens where a page has fewer than 128), and rows
// that share a prefix. T is what a row's table has room for.
template <int kShards>
struct PagedParams : DecodeParams<kShards> {
    static constexpr bool kPaged = true;
    const uint8_t* kv[kShards];
    const int* tables[kShards];
    const int2* groups;                    // [B] first row and rows of the row's group, or NULL
    const int* shared;                     // [B] positions that they have in common
    int* lead;                             // [B] for the join: the group's first row if the row uses the prefix, or -1
    int64_t M;
    int P, page_log2;
};

// ---- PTX helpers -------------------------------------------------------------

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_launch_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
// The same without waiting (try_wait may suspend the thread for a while).
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ long long global_ns() {
    long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
// Wait for a phase, at most limit_ns: then set the CTA's abort flag and the
// status word. Returns at once when the flag is set already.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status,
                                          long long limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = global_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (*abort_flag) return false;
        if (global_ns() - t0 > limit_ns) {
            *abort_flag = 1;
            if (status != nullptr) atomicOr(status, 1);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ void mbar_drain(uint64_t* bar, uint32_t parity, long long limit_ns) {
    const long long t0 = global_ns();
    while (!mbar_try_wait(bar, parity) && global_ns() - t0 <= limit_ns) {}
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 4 bytes from global to shared memory, asynchronously; `bytes` = 0 writes zeros.
__device__ __forceinline__ void copy_word(uint32_t dst, const uint8_t* src, uint32_t bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_16(uint32_t dst, const uint8_t* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* tm, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* tm, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(reinterpret_cast<uint64_t>(tm)),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// `bytes` (a multiple of 16) from a 16-byte boundary to L2
__device__ __forceinline__ void prefetch_bulk(const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
constexpr uint32_t kSwizzle128 = 2, kSwizzle64 = 4, kSwizzle32 = 6, kSwizzleNone = 0;
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
    return (uint64_t)((addr >> 4) & 0x3fffu) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
           (1ull << 46) | ((uint64_t)swizzle << 61);
}
// D[tmem] (+)= A . B, e4m3 x e4m3, fp32
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// the same with one ue8m0 scale for 32 products of a row of A and of B
// (kKeep: A stays in the tensor core's collector; kKept: it is there from the MMA before)
enum Collect { kPlain, kKeep, kKept };
template <Collect kC>
__device__ __forceinline__ void mma_f8_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                              uint32_t sfb, uint32_t acc) {
#define DCP_MMA_SCALED(collector)                                                                                 \
    asm volatile(                                                                                                 \
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"                                                             \
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X" collector                            \
        " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),                                                        \
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)                                                  \
        : "memory")
    if constexpr (kC == kPlain) DCP_MMA_SCALED("");
    else if constexpr (kC == kKeep) DCP_MMA_SCALED(".collector::a::fill");
    else DCP_MMA_SCALED(".collector::a::lastuse");
#undef DCP_MMA_SCALED
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// 512 bytes of scales (32 rows x 16 bytes) from shared memory to 4 columns of every lane quadrant
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint32_t addr) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem),
                 "l"(smem_desc(addr, 16, 128, kSwizzleNone))
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
template <int kN>
__device__ __forceinline__ void tmem_ld(uint32_t addr, float* v) {
    uint32_t* const u = reinterpret_cast<uint32_t*>(v);
    if constexpr (kN == 4) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
                     : "r"(addr));
    } else if constexpr (kN == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                     : "r"(addr));
    } else {
        static_assert(kN == 16, "");
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
            "%15}, [%16];"
            : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
              "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
            : "r"(addr));
    }
}
__device__ __forceinline__ void tmem_st4(uint32_t addr, const float* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3]))
                 : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- which tokens a row sees ---------------------------------------------------

// Shard j's share of the first L positions: with q full rounds over the shards
// and r positions of the last one, q * interleave and what of r falls to j.
struct Prefix {
    uint32_t q, r;
};
template <class P>
__device__ __forceinline__ Prefix prefix_of(const P& p, uint32_t L) {
    if (p.shards() == 1) return {0u, L};
    const uint32_t round = p.shards() * p.interleave, q = L / round;
    return {q, L - q * round};
}
template <class P>
__device__ __forceinline__ uint32_t share(const P& p, Prefix x, uint32_t j) {
    uint32_t n = x.r;
    if (p.shards() > 1) {
        const uint32_t lo = j * p.interleave;
        n = x.r > lo ? x.r - lo : 0u;
        n = x.q * p.interleave + (n < p.interleave ? n : p.interleave);
    }
    return n < p.T ? n : p.T;
}
struct RowView {
    Prefix len, win, sink;
    bool prefix;  // (of a group: whole tiles)
};
__device__ __forceinline__ uint32_t row_length(const DecodeBase& p, int b) {
    const int n = p.seq_lens[b];
    return n < 0 ? 0u : (uint32_t)n;
}
// What is walked through. Without groups there is a line for each row, all of its positions. With groups there are 2 B:
// line b < B is the prefix of row b's group for the b-th set of that group's heads (a set is head_blocks blocks of kNH
// heads of the group's rows, one row's behind the other's), of no tile where the group has fewer sets; line B + b is
// what row b has behind the prefix. A prefix ends at a whole tile of each shard, and the rest belongs to the rows. A row
// that is shorter than its prefix takes no part, and has all its tokens in its own line.
struct Line {
    uint32_t length;  // positions [base, length)
    uint32_t base;
    uint32_t source;  // kPrefix and the set, or 0; and the heads of this CTA's block (kHeadsAt)
};
constexpr uint32_t kPrefix = 1u << 31, kHeadsAt = 16, kSetMask = 0xffffu;
template <class P>
__device__ __forceinline__ int line_count(const P& p) {
    if constexpr (P::kPaged)
        if (p.groups != nullptr) return 2 * p.B;
    return p.B;
}
// The row that a line's tokens are of.
template <class P>
__device__ __forceinline__ int line_row(const P& p, int v, uint32_t source) {
    if constexpr (P::kPaged) {
        if (p.groups == nullptr) return v;
        return source & kPrefix ? v - (int)(source & kSetMask) : v - p.B;
    }
    return v;
}
template <class P>
__device__ __forceinline__ Line line_of(const P& p, int v, int hblk, int block_heads) {
    Line r = {0u, 0u, 0u};
    if constexpr (P::kPaged) {
        const int h0 = hblk * block_heads, own = p.H - h0 < block_heads ? p.H - h0 : block_heads;
        r.source = (uint32_t)own << kHeadsAt;
        if (p.groups != nullptr) {
            const int b = v < p.B ? v : v - p.B;
            const int2 g = p.groups[b];
            const int n = p.shared[b], len = p.seq_lens[b];
            // (groups that the call does not allow have no prefix, or another one: nothing is read out of place)
            const bool is = g.x >= 0 && g.x <= b && g.y >= 2 && b - g.x < g.y && g.y <= p.B - g.x && n > 0;
            const uint32_t common = is ? (uint32_t)n : 0u;
            if (v >= p.B) {
                r.length = len < 0 ? 0u : (uint32_t)len;
                r.base = r.length >= common ? common : 0u;
                return r;
            }
            const int set = b - g.x, first = (set * p.head_blocks + hblk) * block_heads;
            const int left = is ? g.y * p.H - first : 0;
            if (is && set * p.head_blocks * block_heads < g.y * p.H) r.length = common;
            r.source = kPrefix | (uint32_t)set | ((uint32_t)max(0, min(left, block_heads)) << kHeadsAt);
            return r;
        }
    }
    r.length = row_length(p, v);
    return r;
}
template <class P>
__device__ __forceinline__ RowView row_view(const P& p, const Line& r) {
    const uint32_t L = r.length;
    const uint32_t w = p.window > 0 && L > p.window ? L - p.window : 0u;
    RowView v;
    v.len = prefix_of(p, L);
    v.win = p.window > 0 ? prefix_of(p, w) : Prefix{0u, 0u};
    v.sink = p.sinks > 0 ? prefix_of(p, p.sinks < w ? p.sinks : w) : Prefix{0u, 0u};
    if constexpr (P::kPaged) {
        if (p.groups != nullptr) {  // (there is no window with groups)
            v.win = prefix_of(p, r.base);
            v.prefix = (r.source & kPrefix) != 0;
        }
    }
    return v;
}
// A shard's visible tokens: [0, first) and [start, end); tiles of the one, then of the other. Pages want tiles that
// begin at a multiple of 128 tokens: `skip` tokens of the second part's first tile come before what is visible.
struct ShardView {
    uint32_t first, start, end, skip;
    int tiles_first, tiles;
};
template <class P>
__device__ __forceinline__ ShardView shard_view(const P& p, const RowView& v, uint32_t j) {
    ShardView s = {0u, 0u, 0u, 0u, 0, 0};
    if (!((p.held >> j) & 1u)) return s;
    s.end = share(p, v.len, j);
    if (p.window > 0) {
        s.start = share(p, v.win, j);
        s.first = p.sinks > 0 ? share(p, v.sink, j) : 0u;
        if (s.first == s.start) s.first = s.start = 0u;
    }
    if constexpr (P::kPaged) {
        if (p.groups != nullptr) {
            s.start = share(p, v.win, j) & ~(uint32_t)(kTile - 1);
            if (v.prefix) s.end &= ~(uint32_t)(kTile - 1);
        } else {
            s.skip = s.start & (kTile - 1);
            s.start -= s.skip;
        }
    }
    s.tiles_first = (int)((s.first + kTile - 1) / kTile);
    s.tiles = s.tiles_first + (int)((s.end - s.start + kTile - 1) / kTile);
    return s;
}
template <class P>
__device__ __forceinline__ int row_tiles(const P& p, const Line& r) {
    const RowView v = row_view(p, r);
    int n = 0;
#pragma unroll 1
    for (uint32_t j = 0; j < p.shards(); ++j) n += shard_view(p, v, j).tiles;
    return n;
}
// Walks a row's tiles over the shards.
struct Cursor {
    RowView row;
    ShardView s;
    uint32_t j;
    int i;  // tile of the shard
    template <class P>
    __device__ __forceinline__ void seek(const P& p, const Line& r, int tile) {
        row = row_view(p, r);
        j = 0;
        s = shard_view(p, row, 0);
        i = tile;
        settle(p);
    }
    template <class P>
    __device__ __forceinline__ void settle(const P& p) {
        while (i >= s.tiles && j + 1 < p.shards()) {
            i -= s.tiles;
            s = shard_view(p, row, ++j);
        }
    }
    template <class P>
    __device__ __forceinline__ void next(const P& p) {
        ++i;
        settle(p);
    }
    __device__ __forceinline__ uint32_t token() const {
        return i < s.tiles_first ? (uint32_t)i * kTile : s.start + (uint32_t)(i - s.tiles_first) * kTile;
    }
    __device__ __forceinline__ int valid() const {
        const uint32_t n = (i < s.tiles_first ? s.first : s.end) - token();
        return n < kTile ? (int)n : kTile;
    }
    __device__ __forceinline__ int skip() const { return i == s.tiles_first ? (int)s.skip : 0; }
};

// The CTAs' shares. All rows' tiles lie in a line that is cut evenly, but a row that begins in a share costs its CTA
// a change of segments (q, sums, output) of `change` tiles' time, so that each row is `change` places longer than its
// tiles, which come last. change is 2 with blocks of 64 heads, 1 with 32, 0 with 16. (128 heads, 64 ragged rows x 16K:
// 154 us with 0, 150 with 1, 148 with 2 and with 3; 32 rows x 4096 42, 36, 34, 34. 32 heads, 250 ragged rows x 1024:
// 40, 33, 34, 36. 16 heads, 64 rows x 16K: 66.9, 67.0, 67.9, 68.5.)
__device__ __forceinline__ int places(int tiles, int change) { return tiles > 0 ? tiles + change : 0; }

// What the join needs of a row: its first CTA range and its number of segments. Written by the CTA that has the
// row's first tile (at place pre + change); for a row without a tile by the first CTA.
template <class P>
__device__ __forceinline__ void tell_row(const P& p, int b, const Line& r, int n, int pre, int g, int g_end, int per,
                                         int range, int change) {
    pre += change;
    if (n == 0 && range == 0) p.row_info[b] = make_int2(0, 0);
    else if (n > 0 && pre >= g && pre < g_end) p.row_info[b] = make_int2(range, (pre + n - 1) / per - range + 1);
    if constexpr (P::kPaged)
        if (range == 0 && p.groups != nullptr && b >= p.B) p.lead[b - p.B] = r.base > 0 ? p.groups[b - p.B].x : -1;
}

// ---- the kernel ------------------------------------------------------------------

template <int kDk, int kNH>
struct Shape {
    static constexpr bool kHasRope = kDk > kDv;
    static constexpr int kRows = 2 * kNH;                    // Q rows: hi, then lo
    static constexpr bool kStacked = kNH <= 32;              // P's lo rows behind its hi rows in one operand
    static constexpr int kRopeSlice = kHasRope ? kTile * 64 : 0;
    static constexpr int kStage = 4 * kSlice + kRopeSlice;
    static constexpr int kQSlice = kRows * 128;
    static constexpr int kQBytes = 4 * kQSlice + (kHasRope ? kRows * 64 : 0);
    // With 64 heads P's lo part takes the rope slice of its tile, which is done with once the scores are there.
    static constexpr bool kLoInRope = !kStacked && kHasRope;
    static constexpr int kPRow = kStacked ? kRows : kNH;     // bytes of a token in P: 64, or 32 with 16 heads
    static constexpr int kPBytes = kTile * kPRow * (kStacked || kLoInRope ? 1 : 2);
    static constexpr int kMisc = 1024 + 8 * kNH * 4;
    static constexpr int kSmem = 2 * kStage + kQBytes + kPBytes + kMisc;
    static constexpr int kHW = kNH / 4;                      // heads of a thread
    // TMEM: S [0, rows), O in blocks of kNH columns, scales. A block of 128 latent dims has O's two parts side by side
    // (one MMA of both parts of P) where there is room: with 64 heads that is the first one only.
    static constexpr int kO = kRows;
    static constexpr int kOBlocks = kStacked ? 8 : 5;
    static constexpr int kSf = kO + kOBlocks * kNH;
    __device__ __forceinline__ static bool wide(int m) { return kStacked || m == 0; }
    __device__ __forceinline__ static uint32_t col(int m) {
        return (uint32_t)(kO + (kStacked ? 2 * m : m + (m > 0 ? 1 : 0)) * kNH);
    }
    static constexpr int kCols = kSf + 8 <= 256 ? 256 : 512;
    static_assert(kSmem <= 232448 && kSf + 8 <= 512, "");
};

// What the loading warp tells the others about a tile.
struct alignas(16) TileInfo {
    uint32_t token;  // first token
    int valid;       // tokens; 0: no more tiles (pages: and those to skip, from bit 8 on)
    uint32_t what;   // shard, and kFirst ...
    int row;
};
constexpr uint32_t kFirst = 256, kLast = 512;  // the first, the last tile of a segment (a run of tiles of one row)
constexpr uint32_t kWhole = 1024;              // the segment is the whole row
constexpr uint32_t kStarts = 2048;             // the segment has the row's first tile
constexpr uint32_t kFresh = 4096;              // no tile of the segment before this one has a visible token (pages)

struct Shared {  // barriers and small things, behind the scale atom
    uint64_t info_full[4];    // a tile's description is there
    uint64_t kv_full[2][4];   // a slice of a tile has landed (the last one with the rope slice)
    uint64_t kv_free[2][4];   // it has been multiplied for the last time
    uint64_t s_full, s_free;  // scores are in TMEM; they have been read
    uint64_t p_full;          // probabilities (and zeroed rows, scales) are in shared memory
    uint64_t o_done;          // a tile's values are added
    uint64_t q_full;          // a segment's q is in shared memory
    uint64_t drained;         // every MMA of the CTA is done
    uint64_t q_asked;         // the first segment's q is on its way
    uint64_t voted[4];        // a group's warps know how far their scores are above the references
    uint64_t met[4];          // a group's warps have come to the same place
    int moved[4][2];          // too far, in the group's even and odd tiles
    int armed[2][4];          // how often each slice's barrier has been armed, less one
    uint32_t tmem;
    int abort;
    int find[4];              // the CTA's first row (-1: none), its first tile there, the row's tiles
    union {
        int wsum[16];
        int pages[4][4];      // of a tile, by fours of 32 tokens at most; negative: none
    };
    TileInfo info[4];
    uint32_t source[4];       // of a tile's line (pages)
};
static_assert(sizeof(Shared) <= 512 && offsetof(Shared, s_full) == 160, "");

// Scores ride on 1.5 * 2^23: x + kMagic rounds x to an integer that the low bits
// of the sum hold, so that integer maxima and differences of the sums' bits are
// those of the rounded scores (for |x| < 2^22).
constexpr float kMagic = 12582912.f;
constexpr int kMagicBits = 0x4B400000;
constexpr int kRange = 1 << 21;  // scores beyond this (base-2 units) give NaN
constexpr int kBias = 127 - 8;   // P is 2^8 at the block's largest
// A token's weight in the sums is 2^(s - M) = P (1 / u) 2^(E - M - 8), of which the last two factors are taken 2^-kEven
// and 2^kEven times. So no token whose score is within 29 of the row's largest is lost below fp32, whatever scales of
// 2^-60 to 2^32 stand side by side: M is at most 93 above that score (kLow, and the largest scale), a factor of 0 has
// E - M < -182, and s is at most E + 60.5.
constexpr int kEven = 64;
__device__ __forceinline__ float weight_of(int d) {  // (d is at most kLazy)
    return __int_as_float(max(d + kBias + kEven, 0) << 23);
}
// 2^-x, for x > 126 zero (x >= -127)
__device__ __forceinline__ float down_by(int x) { return __int_as_float(max(127 - x, 0) << 23); }

using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
    f32x2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ void unpack2(f32x2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ __nv_bfloat162 as_bf16x2(uint32_t x) { return *reinterpret_cast<__nv_bfloat162*>(&x); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 x) { return *reinterpret_cast<uint32_t*>(&x); }
// Two e4m3 codes of a pair of bf16, in its order.
__device__ __forceinline__ uint32_t codes2(uint32_t x) {
    return __nv_cvt_float2_to_fp8x2(make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u)),
                                    __NV_SATFINITE, __NV_E4M3);
}
// Four e4m3 codes, the first in the low byte.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
// A vote of all softmax warps (and a barrier).
__device__ __forceinline__ bool soft_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 q, %2, 0;\n barrier.cta.red.or.pred.aligned p, 5, %1, q;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(r)
        : "n"(kSoftThreads), "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
    return r != 0;
}

// The scores' MMAs over slice s of the tile at `ka`, with the last slice those over the rope slice.
// (Loops are kept rolled where code runs once or rarely: a call is short, its
// instructions come from L2, and unrolled they cost more than they compute.)
template <class S>
__device__ __forceinline__ void issue_scores(uint32_t ka, uint32_t qa, uint32_t tmem, uint32_t idesc, int s,
                                             uint64_t* done) {
    if (elect_one()) {
        const uint64_t a0 = smem_desc(ka + s * kSlice, 16, 1024, kSwizzle128);
        const uint64_t b0 = smem_desc(qa + s * S::kQSlice, 16, 1024, kSwizzle128);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f8(tmem, a0 + (uint32_t)(2 * k), b0 + (uint32_t)(2 * k), idesc, s | k);
        if (s == 3) {
            if constexpr (S::kHasRope) {
                const uint64_t a1 = smem_desc(ka + 4 * kSlice, 16, 512, kSwizzle64);
                const uint64_t b1 = smem_desc(qa + 4 * S::kQSlice, 16, 512, kSwizzle64);
                mma_f8(tmem, a1, b1, idesc, 1);
                mma_f8(tmem, a1 + 2, b1 + 2, idesc, 1);
            }
            mma_commit(done);
        }
    }
    __syncwarp();
}

// Its values: per 128 latent dims 4 MMAs with both parts of P side by side, or 8 with one part each (the cached tile
// then stays in the collector for the second); each slice of the tile is given back as soon as it has been used.
// (Blocks kM0 to kM1 of the four.)
template <class S, int kM0, int kM1>
__device__ __forceinline__ void issue_values(uint32_t ka, uint32_t pa, uint32_t tmem, uint32_t go_on,
                                             uint64_t* slice_free, uint64_t* done) {
    // ue8m0 scales, A read M-major, B N-major
    constexpr uint32_t kId = (1u << 23) | (8u << 24) | (1u << 15) | (1u << 16);
    constexpr uint32_t kIdBoth = kId | ((uint32_t)(S::kRows >> 3) << 17);
    constexpr uint32_t kIdPart = kId | ((uint32_t)(S::kRows >> 4) << 17);
    constexpr uint32_t kSw = S::kPRow == 64 ? kSwizzle64 : kSwizzle32, kStep = 2 * S::kPRow;
    if (elect_one()) {
        // the parts of P: in one row per token, or the low one in its tile's rope slice, or behind the other
        const uint32_t lo = S::kLoInRope ? ka + 4 * kSlice : pa + kTile * S::kPRow;
        const uint64_t a0 = smem_desc(ka, kSlice, 1024, kSwizzle128);
        const uint64_t hi = smem_desc(pa, 16, 8 * S::kPRow, kSw), b1 = smem_desc(lo, 16, 8 * S::kPRow, kSw);
        const uint64_t both = S::kStacked ? hi : (S::kLoInRope ? smem_desc(lo, pa - lo, 8 * S::kPRow, kSw)
                                                               : smem_desc(pa, lo - pa, 8 * S::kPRow, kSw));
        if (kM0 == 0) copy_scales(tmem + S::kSf + 4, pa + S::kPBytes);
#pragma unroll 1
        for (int m = kM0; m < kM1; ++m) {
            const uint32_t d = tmem + S::col(m);
            const uint64_t am = a0 + (uint32_t)(m * (kSlice >> 4));
            if (S::wide(m)) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    mma_f8_scaled<kPlain>(d, am + (uint32_t)(256 * k), both + kStep * k,
                                          kIdBoth | ((uint32_t)k << 4) | ((uint32_t)k << 29), tmem + S::kSf,
                                          tmem + S::kSf + 4, k > 0 ? 1u : go_on);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t id = kIdPart | ((uint32_t)k << 4) | ((uint32_t)k << 29);
                    mma_f8_scaled<kKeep>(d, am + (uint32_t)(256 * k), hi + kStep * k, id, tmem + S::kSf,
                                         tmem + S::kSf + 4, k > 0 ? 1u : go_on);
                    mma_f8_scaled<kKept>(d, am + (uint32_t)(256 * k), b1 + kStep * k, id, tmem + S::kSf,
                                         tmem + S::kSf + 4, 1u);
                }
            }
            mma_commit(slice_free + m);
        }
        if (kM1 == 4) mma_commit(done);
    }
    __syncwarp();
}

// Roles. Sixteen warps do the softmax, in four groups of four: a group has a
// quarter of the heads, a warp of it 32 of the tile's tokens (its TMEM lanes), a
// thread one token. Three warps walk the tiles and load them (TMA, two stages, each
// slice as soon as the values of the tile before last have used it, and the tile
// after next into L2), one issues the MMAs in a fixed turn: a tile's scores, slice
// by slice, then the values of the tile before, so that scores and softmax of one
// tile run beside the values of another. (Polling for whichever was ready first
// was slower, 170 against 164 us at 64 ragged rows x 16K; so was a slice of values
// put between two of scores, 161 against 153.) Where a segment begins the values
// come first, for its q and its sums must wait for them.
//
// Shares. All rows' tiles are cut evenly over the CTAs (a row's parts are joined by
// the second kernel), each head block for itself; a call whose rows have at most two
// tiles gives whole rows to a CTA and needs no second kernel.
template <int kDk, int kNH, class P>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const __grid_constant__ P p) {
    using S = Shape<kDk, kNH>;
    constexpr bool kPaged = P::kPaged;
    constexpr int kHW = S::kHW, kChange = kNH / 32;
    constexpr uint32_t kIdS = (1u << 4) | ((uint32_t)(S::kRows >> 3) << 17) | (8u << 24);
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* const q_s = smem + 2 * S::kStage;
    uint8_t* const p_s = q_s + S::kQBytes;
    uint8_t* const sf_s = p_s + S::kPBytes;                       // a 512-byte scale atom
    Shared* const sh = reinterpret_cast<Shared*>(sf_s + 512);
    int* const m_s = reinterpret_cast<int*>(sf_s + 1024);         // reference exponents (as bits of x + kMagic)
    float* const g_s = reinterpret_cast<float*>(m_s + kNH);       // q's scales
    float* const a_s = g_s + kNH;                                 // factors of a moved reference, 1 / sums
    int* const up_s = reinterpret_cast<int*>(a_s + kNH);          // how far it moved
    float* const red = a_s + 2 * kNH;                             // [4][kNH]: a warp's own words
    int* const red_i = reinterpret_cast<int*>(red);
    volatile int* const abort_flag = &sh->abort;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool loads = warp == kLoadWarp || warp > kMmaWarp;
    const int hblk = blockIdx.x % p.head_blocks, range = blockIdx.x / p.head_blocks;
    const int h0 = hblk * kNH;
    const int nh = p.H - h0 < kNH ? p.H - h0 : kNH;

    if (warp == kLoadWarp) {
        // barriers, one per lane: those that one thread or one MMA completes, then those of 16 warps, then of 4
        if (lane < 24) mbar_init(&sh->info_full[0] + lane, lane == 21 || lane == 22 ? kSoftWarps : 1);
        else if (lane == 24) mbar_init(&sh->q_full, kSoftWarps);
        else if (lane == 25) mbar_init(&sh->drained, 1);
        else if (lane == 26) mbar_init(&sh->q_asked, kSoftWarps);
        if (lane < 8) mbar_init(&sh->voted[0] + lane, 4);
        if (lane >= 24) (&sh->moved[0][0])[lane - 24] = 0;
        if (lane >= 16 && lane < 24) (&sh->armed[0][0])[lane - 16] = -1;
        if (lane == 0) {
            *abort_flag = 0;
            sh->find[0] = p.row_mode ? range : -1;
            if constexpr (kPaged) sh->find[3] = nh << kHeadsAt;
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh->tmem)),
                     "r"(S::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid < 128) reinterpret_cast<uint32_t*>(sf_s)[tid] = 0;

    pdl_wait();
    pdl_launch_dependents();
    const int lines = line_count(p);
    Line line = {0u, 0u, 0u};  // the loading warp's; with few lines, first a lane's own
    if (loads && lane < lines) line = line_of(p, lane, hblk, kNH);

    // ---- this CTA's tiles: [g, g_end) of all rows' tiles, from tile `tile` of row `row` (or whole rows)
    int row = range, tile = 0, n_row = 0, g = 0, g_end = 0;
    if (!p.row_mode && lines <= 32) {
        if (loads) {  // few rows: a lane a row, beside the others' set-up
            const int n = lane < lines ? row_tiles(p, line) : 0;
            int x = places(n, kChange);
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            const int total = __shfl_sync(0xffffffffu, x, 31), pre = x - places(n, kChange);
            const int per = max((total + p.ranges - 1) / p.ranges, 1);
            const int64_t lo = (int64_t)range * per, hi = lo + per;
            g = lo < total ? (int)lo : total;
            g_end = hi < total ? (int)hi : total;
            const uint32_t here = __ballot_sync(0xffffffffu, pre <= g && g < x);
            row = here ? __ffs(here) - 1 : 0;
            tile = g - __shfl_sync(0xffffffffu, pre, row) - kChange;
            n_row = __shfl_sync(0xffffffffu, n, row);
            const Line own = line;
            line.length = __shfl_sync(0xffffffffu, line.length, row);
            if constexpr (kPaged) {
                line.base = __shfl_sync(0xffffffffu, line.base, row);
                line.source = __shfl_sync(0xffffffffu, line.source, row);
            }
            if (lane == 0 && here && warp == kLoadWarp) {
                sh->find[0] = row;
                if constexpr (kPaged) sh->find[3] = (int)line.source;
            }
            // (told before the shuffles, the rows' kernel of 64 heads spills: 145.6 us for 64 ragged rows x 16K, not 142)
            if (hblk == 0 && lane < lines && warp == kLoadWarp) tell_row(p, lane, own, n, pre, g, g_end, per, range, kChange);
        }
    } else if (!p.row_mode) {
        int total = 0, n_mine = 0, pre_mine = 0, per_cta = 0;
        Line mine = {0u, 0u, 0u};
        for (int pass = 0; pass < 2; ++pass) {
            int base = 0;
            if (pass == 1) {
                const int per = max((total + p.ranges - 1) / p.ranges, 1);
                const int64_t lo = (int64_t)range * per, hi = lo + per;
                g = lo < total ? (int)lo : total;
                g_end = hi < total ? (int)hi : total;
                per_cta = per;
            }
            for (int b0 = 0; b0 < lines; b0 += kSoftThreads) {
                if (pass == 0 || lines > kSoftThreads) {
                    const bool is = tid < kSoftThreads && b0 + tid < lines;
                    if (is) mine = line_of(p, b0 + tid, hblk, kNH);
                    const int n = is ? row_tiles(p, mine) : 0;
                    int x = places(n, kChange);
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int y = __shfl_up_sync(0xffffffffu, x, o);
                        if (lane >= o) x += y;
                    }
                    if (lane == 31 && warp < kSoftWarps) sh->wsum[warp] = x;
                    __syncthreads();
                    const int ws = lane < kSoftWarps ? sh->wsum[lane] : 0;
                    const int before = __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0);
                    const int all = __reduce_add_sync(0xffffffffu, ws);
                    __syncthreads();
                    n_mine = n;
                    pre_mine = base + before + x - places(n, kChange);
                    base += all;
                }
                if (pass == 1) {
                    if (pre_mine <= g && g < pre_mine + places(n_mine, kChange) && g < g_end) {
                        sh->find[0] = b0 + tid;
                        sh->find[1] = g - pre_mine - kChange;
                        sh->find[2] = n_mine;
                        if constexpr (kPaged) sh->find[3] = (int)mine.source;
                    }
                    if (hblk == 0 && tid < kSoftThreads && b0 + tid < lines)
                        tell_row(p, b0 + tid, mine, n_mine, pre_mine, g, g_end, per_cta, range, kChange);
                }
            }
            if (pass == 0) total = base;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;

    if (loads) {
        // ---- loads (a warp walks together over all tiles and loads its slices, lane 0, or a lane a page)
        const int my_slice = warp > kMmaWarp ? 2 * (warp - kMmaWarp) - 1 : 0, end_slice = my_slice == 1 ? 3 : my_slice + 1;
        if (!p.row_mode && lines > 32) {
            row = lines;
            if (g < g_end) {  // (a range of no tiles has found no row)
                row = sh->find[0];
                tile = sh->find[1];
                n_row = sh->find[2];
                line = line_of(p, row, hblk, kNH);
            }
        }
        // the pages of a tile: a lane has that of its 32, 64 or 128 tokens
        int box_log2 = 7, boxes = 1;
        uint32_t page_mask = ~0u;
        if constexpr (kPaged) {
            page_mask = (1u << p.page_log2) - 1;
            box_log2 = p.page_log2 < 7 ? p.page_log2 : 7;
            boxes = kTile >> box_log2;
        }
        const auto page_at = [&](const Cursor& c, int table_row) {
            int id = -1;
            if constexpr (kPaged) {
                const int64_t slot = (int64_t)(c.token() >> p.page_log2) + lane;
                if (lane < boxes && slot < p.M) id = p.tables[c.j][table_row * p.M + slot];
                if (id >= p.P) id = -1;
            }
            return id < 0 ? -1 : id;
        };
        uint32_t t = 0;
        bool ok = true, known = !p.row_mode;
        while (ok && row < lines && (p.row_mode || g < g_end)) {
            if (kPaged && !p.row_mode && !known) {  // the next line with tiles: many may have none, so a lane a line
                uint32_t some = 0;
                for (; row < lines && !some; row += some ? 0 : 32) {
                    n_row = 0;
                    if (row + lane < lines) {
                        line = line_of(p, row + lane, hblk, kNH);
                        n_row = row_tiles(p, line);
                    }
                    some = __ballot_sync(0xffffffffu, n_row > 0);
                }
                if (!some) break;
                const int at = __ffs(some) - 1;
                row += at;
                n_row = __shfl_sync(0xffffffffu, n_row, at);
                line = {__shfl_sync(0xffffffffu, line.length, at), __shfl_sync(0xffffffffu, line.base, at),
                        __shfl_sync(0xffffffffu, line.source, at)};
            } else if (!known) {
                line = line_of(p, row, hblk, kNH);
                n_row = row_tiles(p, line);
            }
            known = false;
            if (n_row == 0 && p.row_mode && my_slice == 0) {  // a row that sees nothing
                uint4* const o = reinterpret_cast<uint4*>(p.out + ((int64_t)row * p.H + h0) * (kDv * 2));
                for (int i = lane; i < nh * (kDv / 8); i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
                if (p.lse != nullptr)
                    for (int i = lane; i < nh; i += 32) p.lse[(int64_t)row * p.H + h0 + i] = -INFINITY;
            }
            if (!p.row_mode && tile < 0) {  // (places of no tile)
                g -= n_row > 0 ? tile : 0;
                tile = 0;
            }
            const int n = p.row_mode || n_row - tile < g_end - g ? n_row - tile : g_end - g;
            if (n > 0) {
                Cursor c;
                c.seek(p, line, tile);
                const bool alone = !kPaged || (line.base == 0 && !(line.source & kPrefix));  // (nothing joins it)
                const uint32_t about = (tile == 0 ? kStarts : 0u) | (tile == 0 && n == n_row && alone ? kWhole : 0u);
                int table_row = line_row(p, row, line.source);
                if constexpr (kPaged) {
                    // a prefix is read through the first of the group's rows that has all of it (a shorter one may have
                    // been cut back, or have ended)
                    if (line.source & kPrefix) {
                        const int rows = p.groups[row].y, first = table_row;
                        for (int k = 0; k < rows; k += 32) {
                            const uint32_t has = __ballot_sync(
                                0xffffffffu, k + lane < rows && row_length(p, first + k + lane) >= line.length);
                            if (has) {
                                table_row = first + k + __ffs(has) - 1;
                                break;
                            }
                        }
                    }
                }
                int id = page_at(c, table_row);
                bool fresh = true;
                for (int i = 0; i < n; ++i, ++t) {
                    const uint32_t st = t & 1, par = ((t >> 1) + 1) & 1;
                    uint8_t* const kv = smem + st * S::kStage;
                    const int tok0 = (int)c.token();
                    uint32_t what = c.j | about | (i == 0 ? kFirst : 0u) | (i == n - 1 ? kLast : 0u);
                    int valid = c.valid();
                    if (kPaged && my_slice == 0) {
                        if (lane < 4) sh->pages[t & 3][lane] = id;
                        const int lo = lane << box_log2;
                        const bool seen = id >= 0 && lo < valid && lo + (1 << box_log2) > c.skip();
                        what |= fresh ? kFresh : 0u;
                        fresh = fresh && !__any_sync(0xffffffffu, seen);
                        valid |= c.skip() << 8;
                        __syncwarp();
                    }
                    if (lane == 0 && my_slice == 0) {
                        sh->info[t & 3] = {(uint32_t)tok0, valid, what, row};
                        if constexpr (kPaged) sh->source[t & 3] = line.source;
                        mbar_arrive(&sh->info_full[t & 3]);
                    }
                    // (q is needed first: the first tile's loads stand behind it)
                    if (t == 0)
                        ok = __all_sync(0xffffffffu, mbar_wait(&sh->q_asked, 0, abort_flag, p.status, p.wait_ns));
                    if (!ok) break;
                    const int id0 = kPaged ? __shfl_sync(0xffffffffu, id, 0) : row, y = tok0 & (int)page_mask;
#pragma unroll 1
                    for (int a = my_slice; a < end_slice; ++a) {
                        if (t >= 2) ok = mbar_wait(&sh->kv_free[st][a], par, abort_flag, p.status, p.wait_ns);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        uint64_t* const bar = &sh->kv_full[st][a];
                        if (lane == 0) {
                            mbar_expect_tx(bar, kSlice + (a == 3 ? S::kRopeSlice : 0) +
                                                    (p.stall && t == 0 && a == 0 ? 16 : 0));
                            if (!kPaged || boxes == 1) {  // (what is the same in every lane is cheaper)
                                tma_load_3d(kv + a * kSlice, &p.tm_latent[c.j], a * 128, y, id0, bar);
                                if (S::kHasRope && a == 3)
                                    tma_load_3d(kv + 4 * kSlice, &p.tm_rope[c.j], kDv, y, id0, bar);
                            }
                            sh->armed[st][a] = (int)(t >> 1);
                        }
                        if constexpr (kPaged) {
                            // a lane a page (of none, it lies outside the map: zeros), in no order with lane 0's arrival:
                            // the phase waits for that and for all of its bytes
                            if (boxes > 1 && lane < boxes) {
                                tma_load_3d(kv + a * kSlice + (lane << (box_log2 + 7)), &p.tm_latent[c.j], a * 128, 0,
                                            id, bar);
                                if (S::kHasRope && a == 3)
                                    tma_load_3d(kv + 4 * kSlice + (lane << (box_log2 + 6)), &p.tm_rope[c.j], kDv, 0,
                                                id, bar);
                            }
                            __syncwarp();
                        }
                    }
                    if (!ok) break;
                    c.next(p);
                    if constexpr (kPaged) {
                        if (i + 1 < n) {
                            id = page_at(c, table_row);
                            // the next tile's stage is still in use: to L2 meanwhile (a page's tokens lie side by side,
                            // so one request a page instead of one a slice)
                            if (my_slice == 3 && t >= 1 && lane < boxes && id >= 0) {
                                const int64_t at = ((int64_t)id << p.page_log2) + (boxes == 1 ? c.token() & page_mask : 0u);
                                prefetch_bulk(p.kv[c.j] + at * kDk, (uint32_t)kDk << box_log2);
                            }
                            __syncwarp();
                        }
                    }
                    if (kPaged) continue;
                    // the next tile's stage is still in use: to L2 meanwhile
                    if (my_slice == 3 && i + 1 < n && t >= 1 && lane == 0) {
#pragma unroll 1
                        for (int a = 0; a < 4; ++a) tma_prefetch_3d(&p.tm_latent[c.j], a * 128, (int)c.token(), row);
                        if constexpr (S::kHasRope) tma_prefetch_3d(&p.tm_rope[c.j], kDv, (int)c.token(), row);
                    }
                }
            }
            g += n > 0 ? n : 0;
            row += p.row_mode ? p.ranges : 1;
            tile = p.row_mode ? 0 : -kChange;
        }
        if (lane == 0 && my_slice == 0) {
            // no more tiles: a tile of no tokens. (A description's place is free as soon as any slice of the tile three
            // before has been used: the softmax warps are then done with the one before that. The MMA warp looks for the
            // next tile while it has half of the values before to issue, so that no description waits for those.)
            if (ok) {
                sh->info[t & 3] = {0u, 0, 0u, 0};
                mbar_arrive(&sh->info_full[t & 3]);
            }
        }
    } else if (warp == kMmaWarp) {
        // ---- MMAs, in turn: the scores of a tile, slice by slice as they land, then the values of the tile before.
        // The whole warp walks the loop on values that are the same in every lane (so that descriptors live in
        // uniform registers, and an MMA costs one instruction), and one elected lane issues.
        uint32_t t = 0, segs = 0;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), base = smem_u32(smem);
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            return (bool)__all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, p.wait_ns));
        };
        bool began = false;  // tile t - 1 is the first of a segment
        // What tile n is: the first of a segment, one at all.
        auto describe = [&](uint32_t n, bool* first, bool* is) {
            if (!wait(&sh->info_full[n & 3], (n >> 2) & 1)) return false;
            *first = (__shfl_sync(0xffffffffu, sh->info[n & 3].what, 0) & kFirst) != 0;
            *is = __shfl_sync(0xffffffffu, sh->info[n & 3].valid, 0) != 0;
            return true;
        };
        // The values of tile v, and `beside`, what the next tile is: with blocks of 16 or 32 heads that is asked for between
        // their halves, while the first one is at work. (64 ragged rows x 16K: 16 heads 59.7 us, 62.5 with it behind; 32
        // heads 62 and 66; in pages of 64 63 and 66, 64 and 70; where the tiles come from L2, 64 rows behind two prefixes
        // of 16K alone, 102 and 98; 8 rows x 4096 x 16 heads 13.3 and 13.2. 128 heads in pages 132 us, and 124 behind:
        // there the second half comes too late.)
        auto values = [&](uint32_t v, auto beside) {
            if (!wait(&sh->p_full, v & 1)) return false;
            tc_fence_after();
            constexpr int kHalf = S::kStacked ? 2 : 4;
            const uint32_t ka = base + (v & 1) * S::kStage, pa = base + 2 * S::kStage + S::kQBytes;
            issue_values<S, 0, kHalf>(ka, pa, tm, began ? 0u : 1u, sh->kv_free[v & 1], &sh->o_done);
            const bool ok = beside();
            if (kHalf < 4) issue_values<S, kHalf, 4>(ka, pa, tm, began ? 0u : 1u, sh->kv_free[v & 1], &sh->o_done);
            return ok;
        };
        bool first = true, more = false, going = describe(0, &first, &more);
        while (going) {
            // (a new segment's q comes after the sums of the last one, and they after its values)
            const bool turn = t > 0 && (first || !more);
            if (turn && !values(t - 1, [] { return true; })) break;
            if (!more) break;
            if (t > 0 && !wait(&sh->s_free, (t - 1) & 1)) break;
            if (first && !wait(&sh->q_full, segs++ & 1)) break;
            // (whether the next slice is there is asked before this one's MMAs are issued)
            uint64_t* const full = sh->kv_full[t & 1];
            const uint32_t par = (t >> 1) & 1;
            bool ok = true, there = mbar_test(full, par);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (!__all_sync(0xffffffffu, there)) ok = wait(full + s, par);
                if (!ok) break;
                if (s < 3) there = mbar_test(full + s + 1, par);
                tc_fence_after();
                issue_scores<S>(base + (t & 1) * S::kStage, base + 2 * S::kStage, tm, kIdS, s, &sh->s_full);
            }
            if (!ok) break;
            bool next_first = false, next_more = false;
            const auto next = [&] { return describe(t + 1, &next_first, &next_more); };
            going = t > 0 && !turn ? values(t - 1, next) : next();
            began = first;
            first = next_first;
            more = next_more;
            ++t;
        }
        if (elect_one()) mma_commit(&sh->drained);
        mbar_drain(&sh->drained, 0, p.wait_ns);
    } else {
        // ---- softmax
        const int group = warp >> 2, quad = warp & 3, tok = quad * 32 + lane, hb = group * kHW;
        const uint32_t tlane = tmem + ((uint32_t)(32 * quad) << 16);
        if (warp < 4) {  // the cached tile's scale is 1 everywhere: its own scale goes into the probabilities
            const float one[4] = {__uint_as_float(0x7f7f7f7fu), __uint_as_float(0x7f7f7f7fu),
                                  __uint_as_float(0x7f7f7f7fu), __uint_as_float(0x7f7f7f7fu)};
            tmem_st4(tlane + S::kSf, one);
            tmem_wait_st();  // (ordered before the first values by the probabilities' barrier)
        }
        uint32_t t = 0, met = 0;
        bool aborted = false;
        // the four warps of the group meet (a bounded wait, as every wait of this kernel)
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->met[group]);
            return (bool)__all_sync(0xffffffffu,
                                    mbar_wait(&sh->met[group], met++ & 1, abort_flag, p.status, p.wait_ns));
        };
        // A segment's q, raw: a head's bf16 values into the place of its two parts (128 dims of a slice are 256 bytes
        // either way), all of a warp's heads (a quarter of its group's) in flight at once.
        constexpr int kPer = kHW / 4;
        const int hq = hb + quad * kPer;
        auto fetch_q = [&](int v, uint32_t source) {
            const int row = line_row(p, v, source);
            const uint8_t* const src = p.q + row * p.q_row + (h0 + hq) * p.q_head;
            const uint32_t to = smem_u32(q_s);
            const int heads = kPaged ? (int)(source >> kHeadsAt) & 127 : nh;
            // head k of the warp's: of one row, or of a group's rows one behind the other
            const auto head_at = [&](int k) {
                if constexpr (kPaged) {
                    if (source & kPrefix) {
                        const uint32_t r = ((source & kSetMask) * p.head_blocks + hblk) * kNH + hq + k, m = r / p.H;
                        return p.q + (int64_t)(row + (int)m) * p.q_row + (int64_t)(r - m * p.H) * p.q_head;
                    }
                }
                return src + k * p.q_head;
            };
            if (p.q_wide) {
                constexpr int kC = kDk / 8;  // 16-byte pieces of a head
#pragma unroll 1
                for (int i = lane; i < kPer * kC; i += 32) {
                    const int k = i / kC, j = i - k * kC;
                    const uint32_t dst =
                        j < 64 ? (j >> 4) * S::kQSlice + (hq + k + ((j >> 3) & 1) * kNH) * 128 + (j & 7) * 16
                               : 4 * S::kQSlice + (hq + k + ((j - 64) >> 2) * kNH) * 64 + (j & 3) * 16;
                    const bool is = hq + k < heads;
                    copy_16(to + dst, is ? head_at(k) + 16 * j : p.q, is ? 16u : 0u);
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < kPer; ++k) {
                    const bool is = hq + k < heads;
                    const uint8_t* const from = is ? head_at(k) + 4 * lane : p.q;
                    const uint32_t dst = to + (hq + k) * 128 + 4 * lane, step = is ? 128u : 0u, bytes = is ? 4u : 0u;
#pragma unroll 1
                    for (int i = 0; i < 8; ++i)
                        copy_word(dst + (i >> 1) * S::kQSlice + (i & 1) * kNH * 128, from + i * step, bytes);
                    if constexpr (S::kHasRope)
                        copy_word(to + 4 * S::kQSlice + (hq + k + (lane >> 4) * kNH) * 64 + 4 * (lane & 15),
                                  from + 8 * step, bytes);
                }
            }
        };
        // hi and lo e4m3 parts of each head at its own power-of-two scale. A lane has dims 4l .. 4l + 3 of each slice
        // and 2l, 2l + 1 of the rotary part; the arithmetic is on pairs of bf16, and exact.
        auto split_q = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            constexpr int kWords = kDk / 64;
#pragma unroll 1
            for (int h = hq; h < hq + kPer; ++h) {
                uint32_t w[kWords];
                const uint8_t* const raw = q_s + (h + (lane >> 4) * kNH) * 128 + 8 * (lane & 15);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint2 v = *reinterpret_cast<const uint2*>(raw + i * S::kQSlice);
                    w[2 * i] = v.x;
                    w[2 * i + 1] = v.y;
                }
                if constexpr (S::kHasRope)
                    w[8] = *reinterpret_cast<const uint32_t*>(q_s + 4 * S::kQSlice + (h + (lane >> 4) * kNH) * 64 +
                                                              4 * (lane & 15));
                __syncwarp();
                __nv_bfloat162 top = __habs2(as_bf16x2(w[0]));  // (the larger of two numbers: a NaN is passed over)
#pragma unroll
                for (int i = 1; i < kWords; ++i) top = __hmax2(top, __habs2(as_bf16x2(w[i])));
                uint32_t u = as_u32(top);
                u = __reduce_max_sync(0xffffffffu, max(u & 0xffff0000u, u << 16));
                int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // top <= 448 * 2^e
                e = e < -120 ? -120 : e;
                const bool bad = u >= 0x7f800000u;  // an infinity: the whole head is NaN (a NaN stays one by itself)
                const uint32_t inv = bad ? 0x7fff7fffu : (uint32_t)(127 - e) * 0x00800080u;
                if (lane == 0) g_s[h] = bad ? 1.f : __uint_as_float((uint32_t)(127 + e) << 23);
                uint32_t hi[kWords], lo[kWords];
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    // hi: to 4 significand bits (halves away from zero); lo: the rest, at most 4 bits
                    const __nv_bfloat162 x = __hmul2(as_bf16x2(w[i]), as_bf16x2(inv));
                    const uint32_t xh = (as_u32(x) + 0x00080008u) & 0xfff0fff0u;
                    hi[i] = codes2(xh);
                    lo[i] = codes2(as_u32(__hsub2(x, as_bf16x2(xh))));
                }
                // (kNH is a multiple of 8: the rows of both parts are swizzled alike)
                uint8_t* const at = q_s + h * 128 + (((lane >> 2) ^ (h & 7)) << 4) + ((4 * lane) & 15);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    *reinterpret_cast<uint32_t*>(at + i * S::kQSlice) = hi[2 * i] | (hi[2 * i + 1] << 16);
                    *reinterpret_cast<uint32_t*>(at + i * S::kQSlice + kNH * 128) = lo[2 * i] | (lo[2 * i + 1] << 16);
                }
                if constexpr (S::kHasRope) {
                    uint8_t* const ar = q_s + 4 * S::kQSlice + h * 64 + (((lane >> 3) ^ ((h >> 1) & 3)) << 4) +
                                        ((2 * lane) & 15);
                    *reinterpret_cast<uint16_t*>(ar) = (uint16_t)hi[8];
                    *reinterpret_cast<uint16_t*>(ar + kNH * 64) = (uint16_t)lo[8];
                }
            }
            if (lane < kPer) m_s[hq + lane] = kMagicBits;
            async_fence();
            const bool ok = meet();  // (the group's warps use each other's heads)
            if (lane == 0) mbar_arrive(&sh->q_full);
            return ok;
        };
        // The next tile's description; a tile of no tokens ends the loop, and so does a wait that gave up in any
        // warp: all warps agree here.
        TileInfo ti = {0u, 0, 0u, 0};
        uint32_t source = 0;
        auto next_segment = [&](bool good) {
            const bool ok = mbar_wait(&sh->info_full[t & 3], (t >> 2) & 1, abort_flag, p.status, p.wait_ns);
            ti = sh->info[t & 3];
            if constexpr (kPaged) source = sh->source[t & 3];
            return !soft_any(!(ok && good)) && ti.valid > 0;
        };
        // q of the CTA's first row is asked for at once (with whole rows that row may turn out to see nothing)
        const int asked = sh->find[0];
        if (asked >= 0) fetch_q(asked, kPaged ? (uint32_t)sh->find[3] : 0u);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->q_asked);
        bool going = next_segment(true);
        if (going) {
            if (ti.row != asked) {
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                fetch_q(ti.row, source);
            }
            aborted = !split_q();
        }
        while (going) {  // segments
            const int line_now = ti.row, row = line_row(p, ti.row, source);
            const int heads = kPaged ? (int)(source >> kHeadsAt) & 127 : nh;
            f32x2 l2[kHW / 2];
#pragma unroll
            for (int h = 0; h < kHW / 2; ++h) l2[h] = 0ull;

            const uint32_t about = ti.what;  // (of the first tile: how the segment lies in its row)
            // Of a tile: whether this thread's token is visible, and its block's scale, which is asked for one tile ahead.
            const auto look = [&](const TileInfo& i, uint32_t at, bool ok, bool* visible) {
                const int valid = kPaged ? i.valid & 255 : i.valid;
                float u = 1.f;
                bool is = tok < valid;
                if constexpr (kPaged) {
                    const int box = tok >> (p.page_log2 < 7 ? p.page_log2 : 7);
                    const int id = ok ? *(volatile int*)&sh->pages[at & 3][box] : -1;
                    is = is && tok >= (i.valid >> 8) && id >= 0;
                    const uint32_t in_page = (i.token + (uint32_t)tok) & ((1u << p.page_log2) - 1);
                    if (is) u = p.scales[i.what & 255u][(((int64_t)id << p.page_log2) + in_page) >> p.block_log2];
                } else if (ok) {
                    const uint32_t loc = i.token + (uint32_t)(is ? tok : valid - 1);
                    u = p.scales[i.what & 255u][(int64_t)row * p.blocks + (loc >> p.block_log2)];
                }
                *visible = is;
                return u;
            };
            bool seen;
            float u = look(ti, t, true, &seen);
            for (bool first = true;; first = false, ++t) {
                const int valid = kPaged ? ti.valid & 255 : ti.valid;
                bool ok = mbar_wait(&sh->s_full, t & 1, abort_flag, p.status, p.wait_ns);
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
                float sv[kHW];
                f32x2 ru2;
                {
                    float lo[kHW];
                    tmem_ld<kHW>(tlane + hb, sv);
                    tmem_ld<kHW>(tlane + kNH + hb, lo);
                    tmem_wait_ld();
                    tc_fence_before();
                    if (lane == 0) mbar_arrive(&sh->s_free);
                    // a scale of 0 is that of zeros, and counts as the smallest: a weight is at most 2^(kLazy + 60.5),
                    // and fp32 holds the sum of as many as there can be tokens (a NaN stays one)
                    if (u < 7.888609e-31f) u = 8.6736174e-19f;  // 2^-100, 2^-60
                    const float c = u * p.scale_log2, lu = __log2f(u);
                    const float ru = __fdividef(5.421010862e-20f, u);  // 2^-kEven / u
                    ru2 = pack2(ru, ru);
                    const f32x2 c2 = pack2(c, c), lu2 = pack2(lu, lu);
#pragma unroll
                    for (int h = 0; h < kHW; h += 4) {
                        const float4 g = *reinterpret_cast<const float4*>(g_s + hb + h);
                        unpack2(fma2(add2(pack2(sv[h], sv[h + 1]), pack2(lo[h], lo[h + 1])),
                                     mul2(pack2(g.x, g.y), c2), lu2),
                                sv[h], sv[h + 1]);
                        unpack2(fma2(add2(pack2(sv[h + 2], sv[h + 3]), pack2(lo[h + 2], lo[h + 3])),
                                     mul2(pack2(g.z, g.w), c2), lu2),
                                sv[h + 2], sv[h + 3]);
                    }
                }
                if (kPaged ? !seen : valid < kTile && tok >= valid) {
                    // a token that is not visible may hold anything: probability 0 (2^-kRange, and with a whole
                    // warp of them scale 2^-127), and a value row of zeros (0 x NaN)
#pragma unroll
                    for (int h = 0; h < kHW; ++h) sv[h] = -(float)kRange;
                    uint4* const r = reinterpret_cast<uint4*>(smem + (t & 1) * S::kStage + group * kSlice + tok * 128);
#pragma unroll
                    for (int k = 0; k < 8; ++k) r[(k + tok) & 7] = make_uint4(0u, 0u, 0u, 0u);
                }
                // E, the 32 tokens' largest score rounded to an integer, per head, and P = 2^(s - E + 8) in (0, 2^8.5],
                // which does not depend on the reference
                int* const mine = red_i + quad * kNH + hb;  // this warp's words
                int top[kHW];
                uint32_t wh[kHW / 4], wl[kHW / 4];
                const f32x2 neg = pack2(-1.f, -1.f);
#pragma unroll
                for (int h = 0; h < kHW; h += kHW < 8 ? 4 : 8) {
                    constexpr int kB = kHW < 8 ? 4 : 8;
                    float hi[kB], lo[kB];
#pragma unroll
                    for (int k = 0; k < kB; k += 2) {
                        const f32x2 s2 = pack2(sv[h + k], sv[h + k + 1]);
                        float e0, e1;
                        unpack2(add2(s2, pack2(kMagic, kMagic)), e0, e1);
                        top[h + k] = __reduce_max_sync(0xffffffffu, __float_as_int(e0));
                        top[h + k + 1] = __reduce_max_sync(0xffffffffu, __float_as_int(e1));
                        const f32x2 e8 = fma2(pack2(__int_as_float(top[h + k]), __int_as_float(top[h + k + 1])), neg,
                                              pack2(kMagic + 8.f, kMagic + 8.f));
                        float x, y;
                        unpack2(add2(s2, e8), x, y);
                        sv[h + k] = ex2(x);
                        sv[h + k + 1] = ex2(y);
                        // the nearest numbers of 4 significand bits, and the rest
                        hi[k] = __uint_as_float((__float_as_uint(sv[h + k]) + 0x80000u) & 0xfff00000u);
                        hi[k + 1] = __uint_as_float((__float_as_uint(sv[h + k + 1]) + 0x80000u) & 0xfff00000u);
                        unpack2(fma2(pack2(hi[k], hi[k + 1]), neg, pack2(sv[h + k], sv[h + k + 1])), lo[k], lo[k + 1]);
                    }
#pragma unroll
                    for (int k = 0; k < kB; k += 4) {
                        wh[(h + k) / 4] = codes4(hi[k], hi[k + 1], hi[k + 2], hi[k + 3]);
                        wl[(h + k) / 4] = codes4(lo[k], lo[k + 1], lo[k + 2], lo[k + 3]);
                    }
                }
                // Does the reference of some head have to move? Up when a score passes it by 2^kLazy; down only at
                // once, when a segment's first scores lie far below the 0 that it begins at (sums would lose
                // themselves below fp32's range). Each warp says so now and hears the others below. If it moves by
                // `up`, the scales 2^(E - M - 8) and what has been summed are multiplied by 2^-up. P's share of the
                // sums waits for the reference that holds: M follows s + log2 u and the sums s alone, so that at the
                // old one a token with a small scale can lie beyond fp32, and after a move by a large scale the sums
                // before it can still count.
                // (How far E lies from the reference, `d`, and what follows from it is the same for the whole warp: a lane a
                // head, through the warp's words, instead of all heads in every lane.)
                if (lane == 0) {
#pragma unroll
                    for (int h = 0; h < kHW; h += 4)
                        *reinterpret_cast<int4*>(mine + h) = make_int4(top[h], top[h + 1], top[h + 2], top[h + 3]);
                }
                __syncwarp();
                int d = lane < kHW ? mine[lane] - m_s[hb + lane] : INT_MIN;
                bool move = __reduce_max_sync(0xffffffffu, d) > kLazy;
                if (kPaged ? (ti.what & kFresh) && __any_sync(0xffffffffu, seen) : first && quad * 32 < valid)
                    move |= __reduce_min_sync(0xffffffffu, lane < kHW ? d : INT_MAX) < -kLow;
                if (lane == 0) {
                    if (move) sh->moved[group][t & 1] = 1;
                    mbar_arrive(&sh->voted[group]);
                }
                // Beside the vote: the next tile's description, and P, whose place is free once the values before are
                // added. (Both behind it, and the scale asked for with its tile's scores: 64 ragged rows x
                // 16K x 128 heads in pages of 64 125.2 us, 123.6 so.)
                TileInfo next = ti;
                float next_u = 1.f;
                bool next_seen = false;
                if (!(ti.what & kLast)) {
                    const uint32_t n = t + 1;
                    const bool is = mbar_wait(&sh->info_full[n & 3], (n >> 2) & 1, abort_flag, p.status, p.wait_ns);
                    ok = ok && is;
                    next = sh->info[n & 3];
                    next_u = look(next, n, is, &next_seen);
                }
                if (t > 0) ok = mbar_wait(&sh->o_done, (t - 1) & 1, abort_flag, p.status, p.wait_ns) && ok;
                {
                    // A token's heads side by side, as they lie in this thread (the MMA reads P along the heads).
                    uint8_t* const p_lo = S::kLoInRope ? smem + (t & 1) * S::kStage + 4 * kSlice
                                                       : p_s + (S::kStacked ? 0 : kTile * S::kPRow);
                    const int swz = S::kPRow == 64 ? (tok >> 1) & 3 : (tok >> 2) & 1;
                    const int at_h = tok * S::kPRow + (((hb >> 4) ^ swz) << 4) + (hb & 15);
                    const int lo_c = (S::kStacked ? kNH >> 4 : 0) + (hb >> 4);
                    const int at_l = tok * S::kPRow + ((lo_c ^ swz) << 4) + (hb & 15);
                    if constexpr (kHW == 16) {
                        *reinterpret_cast<uint4*>(p_s + at_h) = make_uint4(wh[0], wh[1], wh[2], wh[3]);
                        *reinterpret_cast<uint4*>(p_lo + at_l) = make_uint4(wl[0], wl[1], wl[2], wl[3]);
                    } else if constexpr (kHW == 8) {
                        *reinterpret_cast<uint2*>(p_s + at_h) = make_uint2(wh[0], wh[1]);
                        *reinterpret_cast<uint2*>(p_lo + at_l) = make_uint2(wl[0], wl[1]);
                    } else {
                        *reinterpret_cast<uint32_t*>(p_s + at_h) = wh[0];
                        *reinterpret_cast<uint32_t*>(p_lo + at_l) = wl[0];
                    }
                }
                const bool heard =
                    __all_sync(0xffffffffu, mbar_wait(&sh->voted[group], t & 1, abort_flag, p.status, p.wait_ns));
                ok = ok && heard;
                if (heard && *(volatile int*)&sh->moved[group][t & 1]) {
                    if (lane < kHW) mine[lane] = d;
                    ok = meet() && ok;
                    if (quad == 0 && lane < kHW) {
                        const int r = hb + lane;
                        int up = INT_MIN;
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) up = max(up, red_i[k * kNH + r]);
                        // (each head by its own scores: none is rounded differently for another's)
                        up = up > kLazy || ((kPaged ? (ti.what & kFresh) != 0 : first) && up < -kLow) ? up : 0;
                        const int m = m_s[r] + up;
                        // out of range, or NaN: the head's sums become NaN
                        const bool bad = m >= kMagicBits + kRange || m <= kMagicBits - kRange;
                        a_s[r] = bad ? __int_as_float(0x7fffffff) : down_by(max(up, 0));
                        m_s[r] = m;
                        up_s[r] = up;
                        if (lane == 0) sh->moved[group][t & 1] = 0;
                    }
                    ok = meet() && ok;
                    if (lane < kHW) d -= up_s[hb + lane];
#pragma unroll
                    for (int h = 0; h < kHW; h += 2) {
                        // in two factors, for sums can be 2^93 and a move more than 2^126; a_s adds a NaN, or nothing
                        // (a first tile has no sums before it)
                        const float2 f = *reinterpret_cast<const float2*>(a_s + hb + h);
                        const int2 up = *reinterpret_cast<const int2*>(up_s + hb + h);
                        const int x = max(up.x, 0), y = max(up.y, 0);
                        l2[h / 2] = fma2(pack2(f.x, f.y), 0ull,
                                         mul2(mul2(l2[h / 2], pack2(down_by(x >> 1), down_by(y >> 1))),
                                              pack2(down_by(x - (x >> 1)), down_by(y - (y >> 1)))));
                    }
                    if (!first) {  // O as well (the values before are added)
                        __syncwarp();
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < S::kOBlocks * (kHW / 4); ++c) {
                            const int h = (c % (kHW / 4)) * 4, b = c / (kHW / 4);
                            const uint32_t col = tlane + S::kO + b * kNH + hb + h;
                            float o[4];
                            tmem_ld<4>(col, o);
                            const float4 f = *reinterpret_cast<const float4*>(a_s + hb + h);
                            tmem_wait_ld();
                            o[0] *= f.x;
                            o[1] *= f.y;
                            o[2] *= f.z;
                            o[3] *= f.w;
                            tmem_st4(col, o);
                        }
                        tmem_wait_st();
                    }
                }
                float* const weight = reinterpret_cast<float*>(mine);
                if (lane < kHW) weight[lane] = weight_of(d);
                __syncwarp();
#pragma unroll
                for (int h = 0; h < kHW; h += 4) {
                    const float4 w = *reinterpret_cast<const float4*>(weight + h);
                    l2[h / 2] = fma2(mul2(pack2(sv[h], sv[h + 1]), ru2), pack2(w.x, w.y), l2[h / 2]);
                    l2[h / 2 + 1] = fma2(mul2(pack2(sv[h + 2], sv[h + 3]), ru2), pack2(w.z, w.w), l2[h / 2 + 1]);
                }
                // (warps of a group leave at one place: at the end of a tile, when a wait gave up anywhere)
                if (lane < kHW) {
                    const int r = hb + lane;
                    const int sf = max(d + kBias, 0);
                    sf_s[(r & 31) * 16 + (r >> 5) * 4 + quad] = (uint8_t)sf;
                    sf_s[((r + kNH) & 31) * 16 + ((r + kNH) >> 5) * 4 + quad] = (uint8_t)sf;
                }
                async_fence();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->p_full);
                aborted = aborted || __any_sync(0xffffffffu, !ok);
                if (aborted || (ti.what & kLast)) break;
                ti = next;
                u = next_u;
                seen = next_seen;
            }
            ++t;
            // ---- the segment's end. The next one's q comes in meanwhile (this one's scores are all done: q's place
            // is free) and is split before this one's output leaves, so that its first scores run beside that.
            going = next_segment(!aborted);
            if (going) fetch_q(ti.row, source);
            if (!aborted) {
                // sums over the warp's tokens: halves of the heads to halves of the lanes until a lane has one head
                float l[kHW];
#pragma unroll
                for (int h = 0; h < kHW; h += 2) unpack2(l2[h / 2], l[h], l[h + 1]);
                int off = 16;
#pragma unroll
                for (int k = kHW / 2; k >= 1; k /= 2, off /= 2) {
                    const bool upper = (lane & off) != 0;
#pragma unroll
                    for (int h = 0; h < k; ++h) {
                        const float give = upper ? l[h] : l[h + k], keep = upper ? l[h + k] : l[h];
                        l[h] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                    }
                }
#pragma unroll
                for (; off >= 1; off /= 2) l[0] += __shfl_xor_sync(0xffffffffu, l[0], off);
                if ((lane & (32 / kHW - 1)) == 0) red[quad * kNH + hb + lane / (32 / kHW)] = l[0];
                aborted = !meet();
                const bool whole = (about & kWhole) != 0;  // the row's only segment
                int64_t slot = (int64_t)blockIdx.x * 2 + ((about & kStarts) ? 1 : 0);
                if constexpr (kPaged)  // with groups a CTA can have many lines that begin here and are joined
                    if (p.groups != nullptr)
                        slot = (about & kStarts) ? gridDim.x + (int64_t)line_now * p.head_blocks + hblk : blockIdx.x;
                if (quad == 0 && lane < kHW) {
                    const int r = hb + lane;
                    const float l = (red[r] + red[kNH + r]) + (red[2 * kNH + r] + red[3 * kNH + r]);
                    a_s[r] = kPaged && l == 0.f ? 0.f : __fdividef(1.0f, l);  // (no visible token has a page)
                    const float lse2 = (float)(m_s[r] - kMagicBits) + log2f(l);
                    if (!whole) p.part_lse[slot * kNH + r] = lse2;
                    else if (p.lse != nullptr && r < heads) p.lse[(int64_t)row * p.H + h0 + r] = lse2 * p.lse_scale;
                }
                aborted = !meet() || aborted;
                float inv[kHW];
#pragma unroll
                for (int h = 0; h < kHW; h += 4) {
                    const float4 x = *reinterpret_cast<const float4*>(a_s + hb + h);
                    inv[h] = x.x;
                    inv[h + 1] = x.y;
                    inv[h + 2] = x.z;
                    inv[h + 3] = x.w;
                }
                if (going) aborted = !split_q() || aborted;
                aborted = !__all_sync(0xffffffffu, mbar_wait(&sh->o_done, (t - 1) & 1, abort_flag, p.status,
                                                             p.wait_ns)) || aborted;
                tc_fence_after();
#pragma unroll 1
                for (int m = 0; m < 4; ++m) {
                    float o[kHW];
                    tmem_ld<kHW>(tlane + S::col(m) + hb, o);
                    if (S::wide(m)) {
                        float lo[kHW];
                        tmem_ld<kHW>(tlane + S::col(m) + kNH + hb, lo);
                        tmem_wait_ld();
#pragma unroll
                        for (int h = 0; h < kHW; ++h) o[h] += lo[h];
                    }
                    tmem_wait_ld();
                    const int d = 128 * m + tok;  // lane = latent dim: a warp's store is contiguous
                    if (whole) {
                        __nv_bfloat16* const dst =
                            reinterpret_cast<__nv_bfloat16*>(p.out) + ((int64_t)row * p.H + h0 + hb) * kDv + d;
#pragma unroll
                        for (int h = 0; h < kHW; ++h)
                            if (hb + h < heads) dst[h * kDv] = __float2bfloat16_rn(o[h] * inv[h]);
                    } else {
                        float* const dst = p.part + slot * (kNH * kDv) + hb * kDv + d;
#pragma unroll
                        for (int h = 0; h < kHW; ++h)
                            if (!kPaged || hb + h < heads) dst[h * kDv] = o[h] * inv[h];
                    }
                }
                tc_fence_before();
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");  // (of a segment that was given up)
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    // after a wait that gave up, what was armed still lands before the CTA leaves
    if (warp == kLoadWarp && lane < 8 && *abort_flag) {
        const int n = sh->armed[lane >> 2][lane & 3];
        if (n >= 0) mbar_drain(&sh->kv_full[lane >> 2][lane & 3], (uint32_t)(n & 1), p.wait_ns);
    }
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kCols) : "memory");
}

// ---- the rows that were split ---------------------------------------------------------

struct JoinParams {
    static constexpr bool kPaged = false;
    const float* part;
    const float* part_lse;
    const int2* row_info;
    uint8_t* out;
    float* lse;
    int64_t units;       // rows x heads
    int H, head_blocks, block_heads;
    float lse_scale;
};
struct PagedJoinParams : JoinParams {
    static constexpr bool kPaged = true;
    const int* lead;     // [B], or NULL: no groups
    int B, ctas;
};

// One warp per (row, head), eight of them a CTA; or a CTA of kWarps warps, where there are few rows and many segments
// of each (its 1024 CTAs for 8 rows x 128 heads are resident at once with four warps, not with eight). The segments'
// outputs are weighted by 2^(lse - max), and the row's LSE comes of the same weights. Rows with one segment have been
// written; rows without a tile get zeros. Bound by the partials' way from L2, so a warp asks for two segments at once,
// together with the LSEs: two round trips, the first for what the row has.
// Rows with a prefix have its segments first, those of the group's set of heads that has this head, then their own.
template <int kWarps, class Q>
__global__ void __launch_bounds__(kWarps > 1 ? 32 * kWarps : 256) join_kernel(const __grid_constant__ Q p) {
    constexpr bool kPaged = Q::kPaged;
    __shared__ float acc_s[kWarps > 1 ? kWarps : 1][kDv];
    __shared__ float sum_s[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = kWarps > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 8 + warp;
    const int b = (int)(unit / p.H), h = (int)(unit - (int64_t)b * p.H);
    const int hblk = h / p.block_heads, hh = h - hblk * p.block_heads, w = kWarps > 1 ? warp : 0;
    pdl_wait();
    pdl_launch_dependents();
    if (unit >= p.units) return;
    // the places of its segments, in heads: the first prefix one, then from `pre_at` on; the first own one, then from
    // `own_at` on (with `step` each)
    const int step = p.head_blocks * p.block_heads;
    int2 row, pre = {0, 0};
    int pre_first = 0, pre_at = 0, own_first = 0, own_at = 0;
    bool grouped = false;
    if constexpr (kPaged) {
        grouped = p.lead != nullptr;
        row = p.row_info[grouped ? p.B + b : b];
        const int lead = grouped ? p.lead[b] : -1;
        if (lead < 0) {
            if (row.y == 1) return;
        } else {
            const int r = (b - lead) * p.H + h, chunk = r / p.block_heads, head = r - chunk * p.block_heads;
            const int set = chunk / p.head_blocks, block = chunk - set * p.head_blocks;
            pre = p.row_info[lead + set];
            pre_first = (p.ctas + (lead + set) * p.head_blocks + block) * p.block_heads + head;
            pre_at = (pre.x * p.head_blocks + block) * p.block_heads + head;
        }
        own_first = (p.ctas + (p.B + b) * p.head_blocks + hblk) * p.block_heads + hh;
        own_at = ((row.x - pre.y) * p.head_blocks + hblk) * p.block_heads + hh;
    } else {
        row = p.row_info[b];
        if (row.y == 1) return;
    }
    const int n = pre.y + row.y;
    uint4* const out = reinterpret_cast<uint4*>(p.out + unit * (kDv * 2));
    if (n == 0) {
        if (w == 0) {
            out[lane] = make_uint4(0u, 0u, 0u, 0u);
            out[32 + lane] = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse != nullptr && lane == 0) p.lse[unit] = -INFINITY;
        }
        return;
    }
    // segment i of the row: the first one is its CTA's last, the others are their CTAs' first
    const auto place = [&](int i) {
        if constexpr (kPaged) {
            if (grouped) {
                if (i < pre.y) return (int64_t)(i == 0 ? pre_first : pre_at + i * step);
                return (int64_t)(i == pre.y ? own_first : own_at + i * step);
            }
        }
        return (((int64_t)(row.x + i) * p.head_blocks + hblk) * 2 + (i == 0 ? 1 : 0)) * p.block_heads + hh;
    };
    float acc[16], sum = 0.f, m = -INFINITY;
    bool nan = false;
    float4 x[2][4];
    const auto load = [&](int i, float4* to) {
        const float4* const src = reinterpret_cast<const float4*>(p.part + place(i) * kDv);
#pragma unroll
        for (int k = 0; k < 4; ++k) to[k] = src[k * 32 + lane];
    };
    if (w < n) load(w, x[0]);
    if (w + kWarps < n) load(w + kWarps, x[1]);
    for (int i = lane; i < n; i += 32) {
        const float l = p.part_lse[place(i)];
        nan |= isnan(l);
        m = fmaxf(m, l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (__any_sync(0xffffffffu, nan)) m = __uint_as_float(0x7fffffffu);
    const bool none = kPaged && m == -INFINITY;  // (no visible token has a page)
    if (none) m = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll 1
    for (int i0 = w; i0 < n; i0 += 2 * kWarps) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = i0 + u * kWarps;
            if (i >= n) break;
            const float f = ex2(p.part_lse[place(i)] - m);
            sum += f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[4 * k] = fmaf(f, x[u][k].x, acc[4 * k]);
                acc[4 * k + 1] = fmaf(f, x[u][k].y, acc[4 * k + 1]);
                acc[4 * k + 2] = fmaf(f, x[u][k].z, acc[4 * k + 2]);
                acc[4 * k + 3] = fmaf(f, x[u][k].w, acc[4 * k + 3]);
            }
            if (i + 2 * kWarps < n) load(i + 2 * kWarps, x[u]);
        }
    }
    if constexpr (kWarps > 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4*>(acc_s[warp])[i * 32 + lane] =
                make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
        if (lane == 0) sum_s[warp] = sum;
        __syncthreads();  // (the whole CTA is one unit: no thread has left)
        sum = 0.f;
        float4 a = {0.f, 0.f, 0.f, 0.f};
        static_assert(kWarps == 1 || kDv == 128 * kWarps, "");
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
            const float4 y = *reinterpret_cast<const float4*>(&acc_s[v][4 * threadIdx.x]);
            sum += sum_s[v];
            a.x += y.x;
            a.y += y.y;
            a.z += y.z;
            a.w += y.w;
        }
        acc[0] = a.x;
        acc[1] = a.y;
        acc[2] = a.z;
        acc[3] = a.w;
    }
    const float inv = none ? 0.f : 1.0f / sum;
#pragma unroll
    for (int i = 0; i < (kWarps > 1 ? 1 : 4); ++i) {
        uint2 v;
        const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[4 * i] * inv, acc[4 * i + 1] * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[4 * i + 2] * inv, acc[4 * i + 3] * inv);
        v.x = *reinterpret_cast<const uint32_t*>(&lo);
        v.y = *reinterpret_cast<const uint32_t*>(&hi);
        reinterpret_cast<uint2*>(out)[kWarps > 1 ? (int)threadIdx.x : i * 32 + lane] = v;
    }
    if (p.lse != nullptr && lane == 0 && w == 0) p.lse[unit] = (m + log2f(sum)) * p.lse_scale;
}

// ---- host side -------------------------------------------------------------------------

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// A [B, T, Dk] byte cache (a pool: [P, page, Dk]) read in boxes of `width` dims x `tokens` tokens; tokens past T, and
// rows outside [0, B), read as 0.
bool encode_cache(CUtensorMap* tm, const void* base, int Dk, int64_t T, int64_t B, uint32_t width, int tokens,
                  CUtensorMapSwizzle swizzle) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    cuuint64_t dim[3] = {(cuuint64_t)Dk, (cuuint64_t)T, (cuuint64_t)B};
    cuuint64_t stride[2] = {(cuuint64_t)Dk, (cuuint64_t)Dk * (cuuint64_t)T};
    cuuint32_t box[3] = {width, (cuuint32_t)tokens, 1u};
    cuuint32_t step[3] = {1u, 1u, 1u};
    return enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dim, stride, box, step,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Heads of a CTA: the smallest block that holds them all, else 64. (16 heads, 8 rows x 4096: 13.0 us in a block of 16,
// 14.4 in 32, 18.4 in 64; 64 rows x 16K: 66, 70, 81. 32 heads: 14.5 us in 32, 15.5 in 16, 18.6 in 64; 70, 113, 82. 128
// heads: 23.4 us in 64, 26.2 in 32; 145, 231. Only 64 heads over few tokens are 8% better in 32, and not over many.)
int head_block(int H) { return H <= 16 ? 16 : (H <= 32 ? 32 : 64); }

// CTAs of a call: one per multiprocessor, shared out between the head blocks.
int grid_ranges(int H, int heads, int num_sms) {
    const int blocks = (H + heads - 1) / heads;
    const int r = num_sms / blocks;
    return r < 1 ? 1 : r;
}

int64_t round_up(int64_t x) { return (x + 255) / 256 * 256; }

struct Workspace {
    int64_t part, part_lse, row_info, lead, bytes;
};
// heads: of a block, from head_block(). With groups each line that begins somewhere has a place, besides those that go on.
Workspace workspace_of(int64_t B, int H, int heads, bool grouped, int num_sms) {
    const int64_t blocks = (H + heads - 1) / heads, ctas = grid_ranges(H, heads, num_sms) * blocks;
    const int64_t slots = grouped ? ctas + 2 * B * blocks : 2 * ctas;
    Workspace w;
    w.part = 0;
    w.part_lse = w.part + round_up(slots * heads * kDv * 4);
    w.row_info = w.part_lse + round_up(slots * heads * 4);
    w.lead = w.row_info + round_up((grouped ? 2 : 1) * B * 8);
    w.bytes = w.lead + (grouped ? round_up(B * 4) : 0);
    return w;
}

// Multiprocessors of the current device, looked up once a device.
int multiprocessors() {
    static int known[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return -1;
    if (dev >= 0 && dev < 64) {
        const int n = __atomic_load_n(&known[dev], __ATOMIC_ACQUIRE);
        if (n > 0) return n;
    }
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return -1;
    if (dev >= 0 && dev < 64) __atomic_store_n(&known[dev], n, __ATOMIC_RELEASE);
    return n;
}

template <class P>
bool grouped_rows(const P& p) {
    if constexpr (P::kPaged) return p.groups != nullptr;
    return false;
}

template <int kDk, int kNH, class P>
cudaError_t launch_decode(const P& p, unsigned flags, cudaStream_t st) {
    constexpr int bytes = Shape<kDk, kNH>::kSmem;
    static int configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(decode_kernel<kDk, kNH, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.ranges * p.head_blocks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (flags & DCP_FLAG_PDL) ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, decode_kernel<kDk, kNH, P>, p);
    if (e != cudaSuccess || p.row_mode) return e;
    // the join overlaps its launch with the decode's tail and waits for it on the device
    const int64_t units = (int64_t)p.B * p.H;
    // four warps a (row, head) where a row has four segments or more on average and the CTAs of all (row, head) are
    // resident in about one turn, else one (128 heads: 8 rows x 4096 23.4 us with four, 25.7 with one; 19 rows 38.2 and
    // 36.5; 64 ragged rows x 16K 152 and 145; 16 heads, 32 rows x 4096 26.2 and 27.3), and with groups, whose prefixes
    // have many (64 rows of 16 heads behind two prefixes of 16K: 61.6 and 63.4)
    const bool few = (p.ranges >= 4 * p.B || grouped_rows(p)) && units <= 8 * (int64_t)p.ranges * p.head_blocks;
    cfg.gridDim = dim3((unsigned)(few ? units : (units + 7) / 8));
    cfg.blockDim = dim3(few ? 128 : 256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    const JoinParams j = {p.part, p.part_lse, p.row_info, p.out, p.lse, units, p.H, p.head_blocks, kNH, p.lse_scale};
    if constexpr (P::kPaged) {
        const PagedJoinParams pj = {j, p.groups != nullptr ? p.lead : nullptr, p.B, p.ranges * p.head_blocks};
        return few ? cudaLaunchKernelEx(&cfg, join_kernel<4, PagedJoinParams>, pj)
                   : cudaLaunchKernelEx(&cfg, join_kernel<1, PagedJoinParams>, pj);
    } else {
        return few ? cudaLaunchKernelEx(&cfg, join_kernel<4, JoinParams>, j)
                   : cudaLaunchKernelEx(&cfg, join_kernel<1, JoinParams>, j);
    }
}

template <class P>
cudaError_t launch_heads(const P& p, int Dk, int heads, unsigned flags, cudaStream_t st) {
    if (Dk > kDv)
        return heads == 16 ? launch_decode<576, 16>(p, flags, st)
                           : (heads == 32 ? launch_decode<576, 32>(p, flags, st) : launch_decode<576, 64>(p, flags, st));
    return heads == 16 ? launch_decode<512, 16>(p, flags, st)
                       : (heads == 32 ? launch_decode<512, 32>(p, flags, st) : launch_decode<512, 64>(p, flags, st));
}

// Encode the shards' tensor maps (of caches of `rows` rows of `tokens` tokens, in boxes of `box`) and launch. Returns the
// call's status.
template <int kShards, class P>
int run_decode(P& p, const DecodeBase& base, const void* const* kv, const float* const* scales, int64_t rows,
               int64_t tokens, int box, int Dk, int heads, unsigned flags, cudaStream_t st) {
    static_cast<DecodeBase&>(p) = base;
    for (uint32_t j = 0; j < (uint32_t)kShards; ++j) {
        p.scales[j] = j < base.cp ? scales[j] : nullptr;
        if (!((base.held >> j) & 1u)) continue;
        if (!encode_cache(&p.tm_latent[j], kv[j], Dk, tokens, rows, 128, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
            (Dk > kDv && !encode_cache(&p.tm_rope[j], kv[j], Dk, tokens, rows, 64, box, CU_TENSOR_MAP_SWIZZLE_64B)))
            return DCP_MLA_CACHE8_ERR_TENSOR_MAP;
    }
    const cudaError_t e = launch_heads(p, Dk, heads, flags, st);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return (int)e;
}
template <int kShards>
int run_rows(const DecodeBase& base, const void* const* kv, const float* const* scales, int Dk, int heads,
             unsigned flags, cudaStream_t st) {
    DecodeParams<kShards> p;
    return run_decode<kShards>(p, base, kv, scales, base.B, base.T, kTile, Dk, heads, flags, st);
}

// What a paged call has besides.
struct Pages {
    const int32_t* const* tables;
    int64_t P, M;
    int page, page_log2;
    const int32_t *groups, *shared;
    int32_t* lead;
};
template <int kShards>
int run_paged(const DecodeBase& base, const Pages& pages, const void* const* kv, const float* const* scales, int Dk,
              int heads, unsigned flags, cudaStream_t st) {
    PagedParams<kShards> p;
    for (uint32_t j = 0; j < (uint32_t)kShards; ++j) {
        p.kv[j] = j < base.cp ? static_cast<const uint8_t*>(kv[j]) : nullptr;
        p.tables[j] = j < base.cp ? pages.tables[j] : nullptr;
    }
    p.groups = reinterpret_cast<const int2*>(pages.groups);
    p.shared = pages.shared;
    p.lead = pages.lead;
    p.M = pages.M;
    p.P = (int)pages.P;
    p.page_log2 = pages.page_log2;
    return run_decode<kShards>(p, base, kv, scales, pages.P, pages.page, pages.page < kTile ? pages.page : kTile, Dk,
                               heads, flags, st);
}

// Every count of tiles stays in 32 bits, for `lines` lines of T tokens a shard (with groups there are two a row).
bool few_tiles(int cp, int64_t lines, int64_t T) { return lines * cp * (T / kTile + 2) <= 1 << 30; }

// Rows of at most two tiles are not worth splitting: a join costs as much. (128 heads x 256 tokens: 12.6 us whole, 15.3
// split for 8 rows, 34 and 41 for 200. Of four tiles: 16.6 whole and 15.7 split for 8 rows x 512, 17.8 and 20.4 for 64;
// the lengths are on the device, and a call with uneven ones wants the split.) Shards that are not held count too: one
// of 8 with 256 tokens a row is split, 16.2 us for 8 rows and 41.9 for 200, where the same tokens alone take 12.0 and
// 33.1.
int64_t most_tiles(int cp, int64_t T, int64_t window, int64_t sinks) {
    const int64_t seen = window > 0 && window < T ? window : T, first = sinks < T ? sinks : T;
    return cp * ((seen + kTile - 1) / kTile + (window > 0 ? (first + kTile - 1) / kTile : 0));
}
bool whole_rows(int cp, int64_t T, int64_t window, int64_t sinks) { return most_tiles(cp, T, window, sinks) <= 2; }
// With pages three tiles neither: it saves a workspace and a second launch as well. (Pages of 64, whole and split. Three
// tiles: 16 heads, 1 row 10.6 and 10.4 us, 128 rows 11.6 and 13.7; 128 heads, 8 rows 14.6 and 16.6. Four tiles: 16 heads, 8
// rows 12.2 and 11.1, 32 rows 12.5 and 11.8; 128 heads, 8 rows 16.6 and 17.0.)
bool whole_paged_rows(int cp, int64_t T, int64_t window, int64_t sinks) {
    return most_tiles(cp, T, window, sinks) <= 3;
}

int page_log2_of(int page) {
    for (int k = 0; (1 << k) <= DCP_MLA_PAGE_MAX; ++k)
        if (page == 1 << k) return (1 << k) >= DCP_MLA_PAGE_MIN ? k : -1;
    return -1;
}

// Groups are of use where a row's heads leave room in a block of 64: then several rows' heads fill it, and a prefix's
// tile is multiplied for all of them at once. (A multiple of 64 heads fills its blocks alone: every block takes the
// prefix's tiles for itself either way, and finds them in L2 without groups too.) And where there are tiles enough: blocks
// of 64 heads, places and a join cost some 5 us more than 16 heads a row alone. (16 heads, one group, with groups and
// without: 8 rows x 2,048 tokens, 144 tiles, 18.8 us and 12.9; 16 x 8,192, 1,056 tiles, 24.0 and 22.8; 8 x 32,768, 2,064
// tiles, 31.2 and 33.5; 32 x 32,768, 8,256 tiles, 51.4 and 93.1. 40 heads, 16 x 8,192: 30.4 and 31.4.) The rows' own tokens
// are in blocks of 64 heads then too, and long ones cost what is saved and more: 64 rows of 16 heads behind 128, 4,096 and
// 8,192 shared tokens with up to 16,384, 12,288 and 8,192 of their own 93.8, 77.1 and 64.6 us with groups, 66.0, 74.4 and
// 82.9 without; of 32 heads 102.8, 82.1, 80.4, and 69.0, 78.0, 88.4. What is known here is what rows have room for, not
// their lengths nor the prefix's: the header says when a caller should leave groups out. Each row takes places for partial results, so that there is a limit; and
// where the tiles of twice as many lines could not be counted, a call goes without.
bool uses_groups(bool grouped, int cp, int64_t B, int H, int64_t T) {
    return grouped && B >= 2 && B <= 2048 && H % 64 != 0 && B * cp * ((T + kTile - 1) / kTile) >= 1024 &&
           few_tiles(cp, 2 * B, T);
}
int group_block(int64_t B, int H) { return head_block(B * H < 64 ? (int)(B * H) : 64); }

}  // namespace

extern "C" int64_t dcp_mla_cache8_decode_workspace_bytes(int cp, int64_t B, int H, int64_t T, int64_t window,
                                                         int64_t sinks, int num_sms) {
    if (cp < 1 || cp > kCpMax || B < 0 || B > 65535 || H < 1 || H > 1024 || T < 0 || T > 0x7fffffff || window < 0 ||
        sinks < 0 || num_sms < 1 || num_sms > 4096 || !few_tiles(cp, B, T))
        return -1;
    return B == 0 || whole_rows(cp, T, window, sinks) ? 0 : workspace_of(B, H, head_block(H), false, num_sms).bytes;
}

extern "C" int64_t dcp_mla_cache8_decode_paged_workspace_bytes(int cp, int64_t B, int H, int page, int64_t M,
                                                               int64_t window, int64_t sinks, int grouped,
                                                               int num_sms) {
    if (page_log2_of(page) < 0 || M < 1 || M > 0x7fffffff || M * page > 0x7fffffff) return -1;
    const int64_t bytes = dcp_mla_cache8_decode_workspace_bytes(cp, B, H, M * page, window, sinks, num_sms);
    if (bytes < 0 || B == 0) return bytes;
    if (uses_groups(grouped != 0, cp, B, H, M * page))
        return workspace_of(B, H, group_block(B, H), true, num_sms).bytes;
    return whole_paged_rows(cp, M * page, window, sinks) ? 0 : bytes;
}

// Both forms. T: what a row has room for; pages: NULL for rows one after the other.
static int decode_call(const void* q, int64_t q_row, int64_t q_head, const void* const* kv_ptrs,
                       const float* const* scale_ptrs, Pages* pages, const int32_t* seq_lens, int cp, int64_t B, int H,
                       int Dk, int Dv, int64_t T, int block, int interleave, int64_t window, int64_t sinks, float scale,
                       int lse_base_e, void* workspace, int64_t workspace_bytes, void* out, float* lse, int32_t* status,
                       unsigned flags, void* stream) {
    if (B < 0 || B > 65535 || H < 1 || H > 1024 || (Dk != 512 && Dk != 576) || Dv != kDv || T < 0 || T > 0x7fffffff)
        return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    int lg = -1;
    for (int k = 0; (1 << k) <= DCP_MLA_CACHE8_BLOCK_MAX; ++k)
        if (block == 1 << k) lg = k;
    if (lg < 0) return DCP_MLA_CACHE8_ERR_BAD_BLOCK;
    if (cp < 1 || cp > kCpMax || interleave < 1 || interleave > kMaxInterleave) return DCP_MLA_CACHE8_ERR_BAD_CP;
    if (window < 0 || sinks < 0 || (sinks > 0 && window == 0)) return DCP_MLA_CACHE8_ERR_BAD_WINDOW;
    if ((flags & ~(DCP_FLAG_PDL | DCP_MLA_FLAG_TEST_STALL)) != 0) return DCP_MLA_CACHE8_ERR_BAD_FLAGS;
    if (kv_ptrs == nullptr || scale_ptrs == nullptr ||
        (B > 0 && (q == nullptr || seq_lens == nullptr || out == nullptr)))
        return DCP_MLA_CACHE8_ERR_NULL_POINTER;
    if (!aligned(q, 4) || q_row % 2 != 0 || q_head % 2 != 0 || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(seq_lens, 4) || !aligned(status, 4))
        return DCP_MLA_CACHE8_ERR_MISALIGNED;
    DecodeBase p;
    int some = -1;
    p.held = 0;
    for (int j = 0; j < cp; ++j) {
        if ((kv_ptrs[j] == nullptr) != (scale_ptrs[j] == nullptr)) return DCP_MLA_CACHE8_ERR_NULL_POINTER;
        if (!aligned(kv_ptrs[j], 16) || !aligned(scale_ptrs[j], 4)) return DCP_MLA_CACHE8_ERR_MISALIGNED;
        if (kv_ptrs[j] != nullptr) {
            if (pages != nullptr && B > 0 && pages->tables[j] == nullptr) return DCP_MLA_CACHE8_ERR_NULL_POINTER;
            if (pages != nullptr && !aligned(pages->tables[j], 4)) return DCP_MLA_CACHE8_ERR_MISALIGNED;
            p.held |= 1u << j;
            some = j;
        }
    }
    if (some < 0) return DCP_MLA_CACHE8_ERR_NULL_POINTER;
    if (!few_tiles(cp, B, T)) return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    const bool grouped = pages != nullptr && uses_groups(pages->groups != nullptr, cp, B, H, T);
    if (B == 0) return 0;
    const int sms = multiprocessors();
    if (sms < 1) {
        (void)cudaGetLastError();
        return DCP_ERR_DEVICE;
    }
    const int heads = grouped ? group_block(B, H) : head_block(H);
    const Workspace ws = workspace_of(B, H, heads, grouped, sms);
    p.row_mode = grouped            ? 0
                 : pages != nullptr ? whole_paged_rows(cp, T, window, sinks)
                                    : whole_rows(cp, T, window, sinks);
    if (!p.row_mode && (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < ws.bytes))
        return DCP_MLA_CACHE8_ERR_WORKSPACE;
    if (T == 0 || (pages != nullptr && pages->P == 0)) p.held = 0;  // nothing is cached: every row is empty
    uint8_t* const w = static_cast<uint8_t*>(workspace);
    p.q = static_cast<const uint8_t*>(q);
    p.q_row = q_row * 2;
    p.q_head = q_head * 2;
    p.q_wide = aligned(q, 16) && q_row % 8 == 0 && q_head % 8 == 0;
    p.seq_lens = seq_lens;
    p.part = reinterpret_cast<float*>(w + ws.part);
    p.part_lse = reinterpret_cast<float*>(w + ws.part_lse);
    p.row_info = reinterpret_cast<int2*>(w + ws.row_info);
    p.out = static_cast<uint8_t*>(out);
    p.lse = lse;
    p.status = status;
    p.blocks = (T + block - 1) / block;
    p.T = (uint32_t)T;
    p.cp = (uint32_t)cp;
    p.interleave = (uint32_t)interleave;
    p.window = window > 0x7fffffff ? 0x7fffffffu : (uint32_t)window;
    p.sinks = sinks > 0x7fffffff ? 0x7fffffffu : (uint32_t)sinks;
    p.block_log2 = lg;
    p.B = (int)B;
    p.H = H;
    p.head_blocks = (H + heads - 1) / heads;
    p.ranges = grid_ranges(H, heads, sms);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.lse_scale = lse_base_e ? 0.6931471805599453f : 1.0f;
    p.stall = (flags & DCP_MLA_FLAG_TEST_STALL) ? 1 : 0;
    p.wait_ns = p.stall ? kTestWaitLimitNs : kWaitLimitNs;
    if (p.row_mode && p.ranges > B) p.ranges = (int)B;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (pages != nullptr) {
        if (grouped) pages->lead = reinterpret_cast<int32_t*>(w + ws.lead);
        else pages->groups = nullptr;
        return cp == 1 ? run_paged<1>(p, *pages, kv_ptrs, scale_ptrs, Dk, heads, flags, st)
                       : run_paged<kCpMax>(p, *pages, kv_ptrs, scale_ptrs, Dk, heads, flags, st);
    }
    if (cp == 1) return run_rows<1>(p, kv_ptrs, scale_ptrs, Dk, heads, flags, st);
    if (cp <= 4) return run_rows<4>(p, kv_ptrs, scale_ptrs, Dk, heads, flags, st);
    return run_rows<kCpMax>(p, kv_ptrs, scale_ptrs, Dk, heads, flags, st);
}

extern "C" int dcp_mla_cache8_decode(const void* q, int64_t q_row, int64_t q_head, const void* const* kv_ptrs,
                                     const float* const* scale_ptrs, const int32_t* seq_lens, int cp, int64_t B,
                                     int H, int Dk, int Dv, int64_t T, int block, int interleave, int64_t window,
                                     int64_t sinks, float scale, int lse_base_e, void* workspace,
                                     int64_t workspace_bytes, void* out, float* lse, int32_t* status, unsigned flags,
                                     void* stream) {
    return decode_call(q, q_row, q_head, kv_ptrs, scale_ptrs, nullptr, seq_lens, cp, B, H, Dk, Dv, T, block, interleave,
                       window, sinks, scale, lse_base_e, workspace, workspace_bytes, out, lse, status, flags, stream);
}

extern "C" int dcp_mla_cache8_decode_paged(const void* q, int64_t q_row, int64_t q_head, const void* const* kv_ptrs,
                                           const float* const* scale_ptrs, const int32_t* const* table_ptrs,
                                           const int32_t* seq_lens, const int32_t* groups, const int32_t* shared,
                                           int cp, int64_t B, int H, int Dk, int Dv, int64_t P, int page, int64_t M,
                                           int block, int interleave, int64_t window, int64_t sinks, float scale,
                                           int lse_base_e, void* workspace, int64_t workspace_bytes, void* out,
                                           float* lse, int32_t* status, unsigned flags, void* stream) {
    Pages pages = {table_ptrs, P, M, page, page_log2_of(page), groups, shared, nullptr};
    if (P < 0 || P > 0x7fffffff || M < 1 || M > 0x7fffffff || B < 0 || B > 65535 || B * M > 0x7fffffff)
        return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    if (block < 1 || block > DCP_MLA_CACHE8_BLOCK_MAX || (block & (block - 1)) != 0)
        return DCP_MLA_CACHE8_ERR_BAD_BLOCK;
    if (pages.page_log2 < 0 || page % block != 0) return DCP_MLA_CACHE8_ERR_BAD_PAGE;
    if (M * page > 0x7fffffff) return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    if (table_ptrs == nullptr || (groups == nullptr) != (shared == nullptr)) return DCP_MLA_CACHE8_ERR_NULL_POINTER;
    if (!aligned(groups, 8) || !aligned(shared, 4)) return DCP_MLA_CACHE8_ERR_MISALIGNED;
    if (groups != nullptr && window > 0) return DCP_MLA_CACHE8_ERR_BAD_WINDOW;
    return decode_call(q, q_row, q_head, kv_ptrs, scale_ptrs, &pages, seq_lens, cp, B, H, Dk, Dv, M * page, block,
                       interleave, window, sinks, scale, lse_base_e, workspace, workspace_bytes, out, lse, status,
                       flags, stream);
}
