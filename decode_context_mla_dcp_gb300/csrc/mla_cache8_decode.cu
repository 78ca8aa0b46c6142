// Single-token MLA attention over the 8-bit latent cache, sm_103a. What it
// computes is stated in include/dcp_mla_cache8.h.
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
// of 64 heads takes 4,230 cycles at the 1.94 GHz that the call runs at. Its MMAs
// alone take 2,958 (1,393 the scores, N = 128; 1,565 the values: N = 64 costs 55
// to 59 cycles and N = 128 77, so both parts of P go into one MMA where TMEM has room
// for them, the first 128 dims). Shared memory's port is what they wait for: the
// operands take 2,150 of its cycles a tile, the tile itself 580, the softmax some
// 900. Two tiles, q and P fill shared memory, S, O and the scales TMEM (456 of 512
// columns), so there is no third stage and one CTA a multiprocessor.
//   measured, 128 heads: 64 ragged rows of up to 16K tokens 142 to 151 us with their
//   lengths, 280 to 286 us for 10^6 tokens (146.3 us, 1.00 PFLOP/s as the operator
//   counts them, twice that on the tensor cores, over three sets of lengths; 148 for
//   seconds on end, at the power limit); 8 rows x 4096 tokens 23.5 us, of which 16.4
//   are the main kernel (4 tiles a CTA between 10,000 cycles to begin and 6,000 to
//   end) and 6 the join; 16 heads, 200 tokens: 8.1 to 8.4 us. One shard of 8 held,
//   8 rows x 4096 of its tokens: 24.0 us.
// With 16 and 32 heads 64 ragged rows x 16K take 67 and 71 us against 45 of their
// bytes; where the rest goes has not been measured.
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

namespace {

constexpr int kDv = 512;
constexpr int kTile = 128;                 // tokens of a tile: the MMA's M
constexpr int kSlice = kTile * 128;        // bytes of a 128-dim slice of a tile
constexpr int kSoftWarps = 16, kSoftThreads = 32 * kSoftWarps;
constexpr int kLoadWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
constexpr int kThreads = kSoftThreads + 64;
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
    CUtensorMap tm_latent[kShards];        // boxes of 128 dims x 128 tokens, 128-byte swizzle
    CUtensorMap tm_rope[kShards];          // boxes of 64 dims x 128 tokens, 64-byte swizzle
    const float* scales[kShards];
    __device__ __forceinline__ uint32_t shards() const { return kShards == 1 ? 1u : cp; }
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
};
__device__ __forceinline__ uint32_t row_length(const DecodeBase& p, int b) {
    const int n = p.seq_lens[b];
    return n < 0 ? 0u : (uint32_t)n;
}
template <class P>
__device__ __forceinline__ RowView row_view(const P& p, uint32_t L) {
    const uint32_t w = p.window > 0 && L > p.window ? L - p.window : 0u;
    RowView v;
    v.len = prefix_of(p, L);
    v.win = p.window > 0 ? prefix_of(p, w) : Prefix{0u, 0u};
    v.sink = p.sinks > 0 ? prefix_of(p, p.sinks < w ? p.sinks : w) : Prefix{0u, 0u};
    return v;
}
// A shard's visible tokens: [0, first) and [start, end); tiles of the one, then of the other.
struct ShardView {
    uint32_t first, start, end;
    int tiles_first, tiles;
};
template <class P>
__device__ __forceinline__ ShardView shard_view(const P& p, const RowView& v, uint32_t j) {
    ShardView s = {0u, 0u, 0u, 0, 0};
    if (!((p.held >> j) & 1u)) return s;
    s.end = share(p, v.len, j);
    if (p.window > 0) {
        s.start = share(p, v.win, j);
        s.first = p.sinks > 0 ? share(p, v.sink, j) : 0u;
        if (s.first == s.start) s.first = s.start = 0u;
    }
    s.tiles_first = (int)((s.first + kTile - 1) / kTile);
    s.tiles = s.tiles_first + (int)((s.end - s.start + kTile - 1) / kTile);
    return s;
}
template <class P>
__device__ __forceinline__ int row_tiles(const P& p, uint32_t L) {
    const RowView v = row_view(p, L);
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
    __device__ __forceinline__ void seek(const P& p, uint32_t L, int tile) {
        row = row_view(p, L);
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
};

// The CTAs' shares. All rows' tiles lie in a line that is cut evenly, but a row that begins in a share costs its CTA
// a change of segments (q, sums, output) of `change` tiles' time, so that each row is `change` places longer than its
// tiles, which come last. change is 2 with blocks of 64 heads, 1 with 32, 0 with 16. (128 heads, 64 ragged rows x 16K:
// 154 us with 0, 150 with 1, 148 with 2 and with 3; 32 rows x 4096 42, 36, 34, 34. 32 heads, 250 ragged rows x 1024:
// 40, 33, 34, 36. 16 heads, 64 rows x 16K: 66.9, 67.0, 67.9, 68.5.)
__device__ __forceinline__ int places(int tiles, int change) { return tiles > 0 ? tiles + change : 0; }

// What the join needs of a row: its first CTA range and its number of segments. Written by the CTA that has the
// row's first tile (at place pre + change); for a row without a tile by the first CTA.
__device__ __forceinline__ void tell_row(const DecodeBase& p, int b, int n, int pre, int g, int g_end, int per,
                                         int range, int change) {
    pre += change;
    if (n == 0 && range == 0) p.row_info[b] = make_int2(0, 0);
    else if (n > 0 && pre >= g && pre < g_end) p.row_info[b] = make_int2(range, (pre + n - 1) / per - range + 1);
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
    int valid;       // tokens; 0: no more tiles
    uint32_t what;   // shard, and kFirst ...
    int row;
};
constexpr uint32_t kFirst = 256, kLast = 512;  // the first, the last tile of a segment (a run of tiles of one row)
constexpr uint32_t kWhole = 1024;              // the segment is the whole row
constexpr uint32_t kStarts = 2048;             // the segment has the row's first tile

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
    int wsum[16];
    TileInfo info[4];
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
template <class S>
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
        copy_scales(tmem + S::kSf + 4, pa + S::kPBytes);
#pragma unroll 1
        for (int m = 0; m < 4; ++m) {
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
        mma_commit(done);
    }
    __syncwarp();
}

// Roles. Sixteen warps do the softmax, in four groups of four: a group has a
// quarter of the heads, a warp of it 32 of the tile's tokens (its TMEM lanes), a
// thread one token. One warp walks the tiles and loads them (TMA, two stages, each
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
template <int kDk, int kNH, int kShards>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const __grid_constant__ DecodeParams<kShards> p) {
    using S = Shape<kDk, kNH>;
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
    uint32_t length = 0;  // the loading warp's row's; with few rows, first a lane's row's
    if (warp == kLoadWarp && lane < p.B) length = row_length(p, lane);

    // ---- this CTA's tiles: [g, g_end) of all rows' tiles, from tile `tile` of row `row` (or whole rows)
    int row = range, tile = 0, n_row = 0, g = 0, g_end = 0;
    if (!p.row_mode && p.B <= 32) {
        if (warp == kLoadWarp) {  // few rows: a lane a row, beside the others' set-up
            const int n = lane < p.B ? row_tiles(p, length) : 0;
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
            length = __shfl_sync(0xffffffffu, length, row);
            if (lane == 0 && here) sh->find[0] = row;
            if (hblk == 0 && lane < p.B) tell_row(p, lane, n, pre, g, g_end, per, range, kChange);
        }
    } else if (!p.row_mode) {
        int total = 0, n_mine = 0, pre_mine = 0, per_cta = 0;
        for (int pass = 0; pass < 2; ++pass) {
            int base = 0;
            if (pass == 1) {
                const int per = max((total + p.ranges - 1) / p.ranges, 1);
                const int64_t lo = (int64_t)range * per, hi = lo + per;
                g = lo < total ? (int)lo : total;
                g_end = hi < total ? (int)hi : total;
                per_cta = per;
            }
            for (int b0 = 0; b0 < p.B; b0 += kSoftThreads) {
                if (pass == 0 || p.B > kSoftThreads) {
                    const int n = tid < kSoftThreads && b0 + tid < p.B ? row_tiles(p, row_length(p, b0 + tid)) : 0;
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
                    }
                    if (hblk == 0 && tid < kSoftThreads && b0 + tid < p.B)
                        tell_row(p, b0 + tid, n_mine, pre_mine, g, g_end, per_cta, range, kChange);
                }
            }
            if (pass == 0) total = base;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;

    if (warp == kLoadWarp) {
        // ---- loads (the warp walks together, lane 0 issues)
        if (!p.row_mode && p.B > 32) {
            row = p.B;
            if (g < g_end) {  // (a range of no tiles has found no row)
                row = sh->find[0];
                tile = sh->find[1];
                n_row = sh->find[2];
                length = row_length(p, row);
            }
        }
        uint32_t t = 0;
        bool ok = true, known = !p.row_mode;
        while (ok && row < p.B && (p.row_mode || g < g_end)) {
            if (!known) {
                length = row_length(p, row);
                n_row = row_tiles(p, length);
            }
            known = false;
            if (n_row == 0 && p.row_mode) {  // a row that sees nothing
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
                c.seek(p, length, tile);
                const uint32_t about = (tile == 0 ? kStarts : 0u) | (tile == 0 && n == n_row ? kWhole : 0u);
                for (int i = 0; i < n; ++i, ++t) {
                    const uint32_t st = t & 1, par = ((t >> 1) + 1) & 1;
                    uint8_t* const kv = smem + st * S::kStage;
                    const int tok0 = (int)c.token();
                    if (lane == 0) {
                        sh->info[t & 3] = {(uint32_t)tok0, c.valid(),
                                           c.j | about | (i == 0 ? kFirst : 0u) | (i == n - 1 ? kLast : 0u), row};
                        mbar_arrive(&sh->info_full[t & 3]);
                    }
                    // (q is needed first: the first tile's loads stand behind it)
                    if (t == 0)
                        ok = __all_sync(0xffffffffu, mbar_wait(&sh->q_asked, 0, abort_flag, p.status, p.wait_ns));
                    if (!ok) break;
#pragma unroll 1
                    for (int a = 0; a < 4; ++a) {
                        if (t >= 2) ok = mbar_wait(&sh->kv_free[st][a], par, abort_flag, p.status, p.wait_ns);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        if (lane == 0) {
                            uint64_t* const bar = &sh->kv_full[st][a];
                            mbar_expect_tx(bar, kSlice + (a == 3 ? S::kRopeSlice : 0) +
                                                    (p.stall && t == 0 && a == 0 ? 16 : 0));
                            tma_load_3d(kv + a * kSlice, &p.tm_latent[c.j], a * 128, tok0, row, bar);
                            if (S::kHasRope && a == 3)
                                tma_load_3d(kv + 4 * kSlice, &p.tm_rope[c.j], kDv, tok0, row, bar);
                            sh->armed[st][a] = (int)(t >> 1);
                        }
                    }
                    if (!ok) break;
                    c.next(p);
                    if (i + 1 < n && t >= 1 && lane == 0) {  // the next tile's stage is still in use: to L2 meanwhile
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
        if (lane == 0) {
            if (ok) {  // no more tiles: a tile of no tokens
                if (t >= 4) ok = mbar_wait(&sh->kv_free[t & 1][3], ((t >> 1) + 1) & 1, abort_flag, p.status, p.wait_ns);
                sh->info[t & 3] = {0u, 0, 0u, 0};
                mbar_arrive(&sh->info_full[t & 3]);
            }
        }
    } else if (warp == kMmaWarp) {
        // ---- MMAs, in turn: the scores of a tile, slice by slice as they land, then the values of the tile before.
        // The whole warp walks the loop on values that are the same in every lane (so that descriptors live in
        // uniform registers, and an MMA costs one instruction), and one elected lane issues.
        uint32_t t = 0, segs = 0;
        bool more = true;
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), base = smem_u32(smem);
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            return (bool)__all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, p.wait_ns));
        };
        bool began = false;  // tile t - 1 is the first of a segment
        auto values = [&](uint32_t v) {
            if (!wait(&sh->p_full, v & 1)) return false;
            tc_fence_after();
            issue_values<S>(base + (v & 1) * S::kStage, base + 2 * S::kStage + S::kQBytes, tm, began ? 0u : 1u,
                            sh->kv_free[v & 1], &sh->o_done);
            return true;
        };
        while (more) {
            if (!wait(&sh->info_full[t & 3], (t >> 2) & 1)) break;
            const bool first = (__shfl_sync(0xffffffffu, sh->info[t & 3].what, 0) & kFirst) != 0;
            more = __shfl_sync(0xffffffffu, sh->info[t & 3].valid, 0) != 0;
            // (a new segment's q comes after the sums of the last one, and they after its values)
            const bool turn = t > 0 && (first || !more);
            if (turn && !values(t - 1)) break;
            if (more) {
                if (t > 0 && !wait(&sh->s_free, (t - 1) & 1)) break;
                if (first && !wait(&sh->q_full, segs++ & 1)) break;
                // (whether the next slice is there is asked before this one's MMAs are issued)
                uint64_t* const full = sh->kv_full[t & 1];
                const uint32_t par = (t >> 1) & 1;
                bool ok = true, there = mbar_try_wait(full, par);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    if (!__all_sync(0xffffffffu, there)) ok = wait(full + s, par);
                    if (!ok) break;
                    if (s < 3) there = mbar_try_wait(full + s + 1, par);
                    tc_fence_after();
                    issue_scores<S>(base + (t & 1) * S::kStage, base + 2 * S::kStage, tm, kIdS, s, &sh->s_full);
                }
                if (!ok || (t > 0 && !turn && !values(t - 1))) break;
            }
            began = first;
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
        auto fetch_q = [&](int row) {
            const uint8_t* const src = p.q + row * p.q_row + (h0 + hq) * p.q_head;
            const uint32_t to = smem_u32(q_s);
            if (p.q_wide) {
                constexpr int kC = kDk / 8;  // 16-byte pieces of a head
#pragma unroll 1
                for (int i = lane; i < kPer * kC; i += 32) {
                    const int k = i / kC, j = i - k * kC;
                    const uint32_t dst =
                        j < 64 ? (j >> 4) * S::kQSlice + (hq + k + ((j >> 3) & 1) * kNH) * 128 + (j & 7) * 16
                               : 4 * S::kQSlice + (hq + k + ((j - 64) >> 2) * kNH) * 64 + (j & 3) * 16;
                    const bool is = hq + k < nh;
                    copy_16(to + dst, is ? src + k * p.q_head + 16 * j : p.q, is ? 16u : 0u);
                }
            } else {
#pragma unroll 1
                for (int k = 0; k < kPer; ++k) {
                    const bool is = hq + k < nh;
                    const uint8_t* const from = is ? src + k * p.q_head + 4 * lane : p.q;
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
        auto next_segment = [&](bool good) {
            const bool ok = mbar_wait(&sh->info_full[t & 3], (t >> 2) & 1, abort_flag, p.status, p.wait_ns);
            ti = sh->info[t & 3];
            return !soft_any(!(ok && good)) && ti.valid > 0;
        };
        // q of the CTA's first row is asked for at once (with whole rows that row may turn out to see nothing)
        const int asked = sh->find[0];
        if (asked >= 0) fetch_q(asked);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->q_asked);
        bool going = next_segment(true);
        if (going) {
            if (ti.row != asked) {
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                fetch_q(ti.row);
            }
            aborted = !split_q();
        }
        while (going) {  // segments
            const int row = ti.row;
            f32x2 l2[kHW / 2];
#pragma unroll
            for (int h = 0; h < kHW / 2; ++h) l2[h] = 0ull;

            const uint32_t about = ti.what;  // (of the first tile: how the segment lies in its row)
            for (bool first = true;; first = false, ++t) {
                bool ok = mbar_wait(&sh->info_full[t & 3], (t >> 2) & 1, abort_flag, p.status, p.wait_ns);
                ti = sh->info[t & 3];
                // this thread's token's scale, in flight beside the scores
                float u = 1.f;
                const int valid = ti.valid;
                if (ok) {
                    const uint32_t loc = ti.token + (uint32_t)(tok < valid ? tok : valid - 1);
                    u = p.scales[ti.what & 255u][(int64_t)row * p.blocks + (loc >> p.block_log2)];
                }
                ok = ok && mbar_wait(&sh->s_full, t & 1, abort_flag, p.status, p.wait_ns);
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
                if (valid < kTile && tok >= valid) {
                    // a token that is not visible may hold anything: probability 0 (2^-kRange, and with a whole
                    // warp of them scale 2^-127), and a value row of zeros (0 x NaN)
#pragma unroll
                    for (int h = 0; h < kHW; ++h) sv[h] = -(float)kRange;
                    uint4* const r = reinterpret_cast<uint4*>(smem + (t & 1) * S::kStage + group * kSlice + tok * 128);
#pragma unroll
                    for (int k = 0; k < 8; ++k) r[(k + tok) & 7] = make_uint4(0u, 0u, 0u, 0u);
                }
                // E, the 32 tokens' largest score rounded to an integer, per head; how far it lies from the reference;
                // and P = 2^(s - E + 8) in (0, 2^8.5], which does not depend on the reference
                int d[kHW], far = INT_MIN;
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
                        const int i0 = __reduce_max_sync(0xffffffffu, __float_as_int(e0));
                        const int i1 = __reduce_max_sync(0xffffffffu, __float_as_int(e1));
                        const int2 m = *reinterpret_cast<const int2*>(m_s + hb + h + k);
                        d[h + k] = i0 - m.x;
                        d[h + k + 1] = i1 - m.y;
                        far = max(far, max(d[h + k], d[h + k + 1]));
                        const f32x2 e8 = fma2(pack2(__int_as_float(i0), __int_as_float(i1)), neg,
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
                bool move = far > kLazy;
                if (first && quad * 32 < valid) {
#pragma unroll
                    for (int h = 0; h < kHW; ++h) move |= d[h] < -kLow;
                }
                if (lane == 0) {
                    if (move) sh->moved[group][t & 1] = 1;
                    mbar_arrive(&sh->voted[group]);
                }
                int* const mine = red_i + quad * kNH + hb;  // this warp's words
                if (lane == 0) {
#pragma unroll
                    for (int h = 0; h < kHW; h += 4)
                        *reinterpret_cast<int4*>(mine + h) = make_int4(d[h], d[h + 1], d[h + 2], d[h + 3]);
                }
                __syncwarp();
                int sf = lane < kHW ? mine[lane] : 0;
                const bool heard =
                    __all_sync(0xffffffffu, mbar_wait(&sh->voted[group], t & 1, abort_flag, p.status, p.wait_ns));
                ok = ok && heard;
                if (heard && *(volatile int*)&sh->moved[group][t & 1]) {
                    ok = meet() && ok;
                    if (quad == 0 && lane < kHW) {
                        const int r = hb + lane;
                        int up = INT_MIN;
#pragma unroll 1
                        for (int k = 0; k < 4; ++k) up = max(up, red_i[k * kNH + r]);
                        // (each head by its own scores: none is rounded differently for another's)
                        up = up > kLazy || (first && up < -kLow) ? up : 0;
                        const int m = m_s[r] + up;
                        // out of range, or NaN: the head's sums become NaN
                        const bool bad = m >= kMagicBits + kRange || m <= kMagicBits - kRange;
                        a_s[r] = bad ? __int_as_float(0x7fffffff) : down_by(max(up, 0));
                        m_s[r] = m;
                        up_s[r] = up;
                        if (lane == 0) sh->moved[group][t & 1] = 0;
                    }
                    ok = meet() && ok;
                    if (lane < kHW) sf -= up_s[hb + lane];
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
                        d[h] -= up.x;
                        d[h + 1] -= up.y;
                    }
                    if (!first) {  // O as well, once the values before are added
                        ok = mbar_wait(&sh->o_done, (t - 1) & 1, abort_flag, p.status, p.wait_ns) && ok;
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
#pragma unroll
                for (int h = 0; h < kHW; h += 2)
                    l2[h / 2] = fma2(mul2(pack2(sv[h], sv[h + 1]), ru2), pack2(weight_of(d[h]), weight_of(d[h + 1])),
                                     l2[h / 2]);
                // the buffer of P is free once the values before are added
                if (t > 0) ok = mbar_wait(&sh->o_done, (t - 1) & 1, abort_flag, p.status, p.wait_ns) && ok;
                // (warps of a group leave at one place: at the end of a tile, when a wait gave up anywhere)
                // A token's heads side by side, as they lie in this thread (the MMA reads P along the heads).
                uint8_t* const p_lo =
                    S::kLoInRope ? smem + (t & 1) * S::kStage + 4 * kSlice : p_s + (S::kStacked ? 0 : kTile * S::kPRow);
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
                if (lane < kHW) {
                    const int r = hb + lane;
                    sf = max(sf + kBias, 0);
                    sf_s[(r & 31) * 16 + (r >> 5) * 4 + quad] = (uint8_t)sf;
                    sf_s[((r + kNH) & 31) * 16 + ((r + kNH) >> 5) * 4 + quad] = (uint8_t)sf;
                }
                async_fence();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->p_full);
                aborted = aborted || __any_sync(0xffffffffu, !ok);
                if (aborted || (ti.what & kLast)) break;
            }
            ++t;
            // ---- the segment's end. The next one's q comes in meanwhile (this one's scores are all done: q's place
            // is free) and is split before this one's output leaves, so that its first scores run beside that.
            going = next_segment(!aborted);
            if (going) fetch_q(ti.row);
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
                const int64_t slot = (int64_t)blockIdx.x * 2 + ((about & kStarts) ? 1 : 0);
                if (quad == 0 && lane < kHW) {
                    const int r = hb + lane;
                    const float l = (red[r] + red[kNH + r]) + (red[2 * kNH + r] + red[3 * kNH + r]);
                    a_s[r] = __fdividef(1.0f, l);
                    const float lse2 = (float)(m_s[r] - kMagicBits) + log2f(l);
                    if (!whole) p.part_lse[slot * kNH + r] = lse2;
                    else if (p.lse != nullptr && r < nh) p.lse[(int64_t)row * p.H + h0 + r] = lse2 * p.lse_scale;
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
                            if (hb + h < nh) dst[h * kDv] = __float2bfloat16_rn(o[h] * inv[h]);
                    } else {
                        float* const dst = p.part + slot * (kNH * kDv) + hb * kDv + d;
#pragma unroll
                        for (int h = 0; h < kHW; ++h) dst[h * kDv] = o[h] * inv[h];
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
    const float* part;
    const float* part_lse;
    const int2* row_info;
    uint8_t* out;
    float* lse;
    int64_t units;       // rows x heads
    int H, head_blocks, block_heads;
    float lse_scale;
};

// One warp per (row, head), eight of them a CTA; or a CTA of kWarps warps, where there are few rows and many segments
// of each (its 1024 CTAs for 8 rows x 128 heads are resident at once with four warps, not with eight). The segments'
// outputs are weighted by 2^(lse - max), and the row's LSE comes of the same weights. Rows with one segment have been
// written; rows without a tile get zeros. Bound by the partials' way from L2, so a warp asks for two segments at once,
// together with the LSEs: two round trips, the first for what the row has.
template <int kWarps>
__global__ void __launch_bounds__(kWarps > 1 ? 32 * kWarps : 256) join_kernel(const __grid_constant__ JoinParams p) {
    __shared__ float acc_s[kWarps > 1 ? kWarps : 1][kDv];
    __shared__ float sum_s[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = kWarps > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 8 + warp;
    const int b = (int)(unit / p.H), h = (int)(unit - (int64_t)b * p.H);
    const int hblk = h / p.block_heads, hh = h - hblk * p.block_heads, w = kWarps > 1 ? warp : 0;
    pdl_wait();
    pdl_launch_dependents();
    if (unit >= p.units) return;
    const int2 row = p.row_info[b];
    if (row.y == 1) return;
    uint4* const out = reinterpret_cast<uint4*>(p.out + unit * (kDv * 2));
    if (row.y == 0) {
        if (w == 0) {
            out[lane] = make_uint4(0u, 0u, 0u, 0u);
            out[32 + lane] = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse != nullptr && lane == 0) p.lse[unit] = -INFINITY;
        }
        return;
    }
    // segment i of the row: the first one is its CTA's last, the others are their CTAs' first
    const auto place = [&](int i) {
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
    if (w < row.y) load(w, x[0]);
    if (w + kWarps < row.y) load(w + kWarps, x[1]);
    for (int i = lane; i < row.y; i += 32) {
        const float l = p.part_lse[place(i)];
        nan |= isnan(l);
        m = fmaxf(m, l);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (__any_sync(0xffffffffu, nan)) m = __uint_as_float(0x7fffffffu);
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll 1
    for (int i0 = w; i0 < row.y; i0 += 2 * kWarps) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = i0 + u * kWarps;
            if (i >= row.y) break;
            const float f = ex2(p.part_lse[place(i)] - m);
            sum += f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                acc[4 * k] = fmaf(f, x[u][k].x, acc[4 * k]);
                acc[4 * k + 1] = fmaf(f, x[u][k].y, acc[4 * k + 1]);
                acc[4 * k + 2] = fmaf(f, x[u][k].z, acc[4 * k + 2]);
                acc[4 * k + 3] = fmaf(f, x[u][k].w, acc[4 * k + 3]);
            }
            if (i + 2 * kWarps < row.y) load(i + 2 * kWarps, x[u]);
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
    const float inv = 1.0f / sum;
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

// A [B, T, Dk] byte cache read in boxes of `width` dims x 128 tokens; tokens past T read as 0.
bool encode_cache(CUtensorMap* tm, const void* base, int Dk, int64_t T, int64_t B, uint32_t width,
                  CUtensorMapSwizzle swizzle) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (enc == nullptr) return false;
    cuuint64_t dim[3] = {(cuuint64_t)Dk, (cuuint64_t)T, (cuuint64_t)B};
    cuuint64_t stride[2] = {(cuuint64_t)Dk, (cuuint64_t)Dk * (cuuint64_t)T};
    cuuint32_t box[3] = {width, (cuuint32_t)kTile, 1u};
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
int grid_ranges(int H, int num_sms) {
    const int blocks = (H + head_block(H) - 1) / head_block(H);
    const int r = num_sms / blocks;
    return r < 1 ? 1 : r;
}

int64_t round_up(int64_t x) { return (x + 255) / 256 * 256; }

struct Workspace {
    int64_t part, part_lse, row_info, bytes;
};
Workspace workspace_of(int64_t B, int H, int num_sms) {
    const int nh = head_block(H);
    const int64_t ctas = (int64_t)grid_ranges(H, num_sms) * ((H + nh - 1) / nh);
    Workspace w;
    w.part = 0;
    w.part_lse = w.part + round_up(2 * ctas * nh * kDv * 4);
    w.row_info = w.part_lse + round_up(2 * ctas * nh * 4);
    w.bytes = w.row_info + round_up(B * 8);
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

template <int kDk, int kNH, int kShards>
cudaError_t launch_decode(const DecodeParams<kShards>& p, unsigned flags, cudaStream_t st) {
    constexpr int bytes = Shape<kDk, kNH>::kSmem;
    static int configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(decode_kernel<kDk, kNH, kShards>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
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
    e = cudaLaunchKernelEx(&cfg, decode_kernel<kDk, kNH, kShards>, p);
    if (e != cudaSuccess || p.row_mode) return e;
    // the join overlaps its launch with the decode's tail and waits for it on the device
    const int64_t units = (int64_t)p.B * p.H;
    // four warps a (row, head) where a row has four segments or more on average and the CTAs of all (row, head) are
    // resident in about one turn, else one (128 heads: 8 rows x 4096 23.4 us with four, 25.7 with one; 19 rows 38.2 and
    // 36.5; 64 ragged rows x 16K 152 and 145; 16 heads, 32 rows x 4096 26.2 and 27.3)
    const bool few = p.ranges >= 4 * p.B && units <= 8 * (int64_t)p.ranges * p.head_blocks;
    cfg.gridDim = dim3((unsigned)(few ? units : (units + 7) / 8));
    cfg.blockDim = dim3(few ? 128 : 256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    const JoinParams j = {p.part, p.part_lse, p.row_info, p.out, p.lse, units, p.H, p.head_blocks, kNH, p.lse_scale};
    return few ? cudaLaunchKernelEx(&cfg, join_kernel<4>, j) : cudaLaunchKernelEx(&cfg, join_kernel<1>, j);
}

// Encode the shards' tensor maps and launch. Returns the call's status.
template <int kShards>
int run_decode(const DecodeBase& base, const void* const* kv, const float* const* scales, int Dk, unsigned flags,
               cudaStream_t st) {
    DecodeParams<kShards> p;
    static_cast<DecodeBase&>(p) = base;
    for (uint32_t j = 0; j < (uint32_t)kShards; ++j) {
        p.scales[j] = j < base.cp ? scales[j] : nullptr;
        if (!((base.held >> j) & 1u)) continue;
        if (!encode_cache(&p.tm_latent[j], kv[j], Dk, base.T, base.B, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
            (Dk > kDv && !encode_cache(&p.tm_rope[j], kv[j], Dk, base.T, base.B, 64, CU_TENSOR_MAP_SWIZZLE_64B)))
            return DCP_MLA_CACHE8_ERR_TENSOR_MAP;
    }
    const int nh = head_block(base.H);
    cudaError_t e;
    if (Dk > kDv) {
        e = nh == 16 ? launch_decode<576, 16>(p, flags, st)
                     : (nh == 32 ? launch_decode<576, 32>(p, flags, st) : launch_decode<576, 64>(p, flags, st));
    } else {
        e = nh == 16 ? launch_decode<512, 16>(p, flags, st)
                     : (nh == 32 ? launch_decode<512, 32>(p, flags, st) : launch_decode<512, 64>(p, flags, st));
    }
    if (e != cudaSuccess) (void)cudaGetLastError();
    return (int)e;
}

// Rows of at most two tiles are not worth splitting: a join costs as much. (128 heads x 256 tokens: 12.6 us whole, 15.3
// split for 8 rows, 34 and 41 for 200. Of four tiles: 16.6 whole and 15.7 split for 8 rows x 512, 17.8 and 20.4 for 64;
// the lengths are on the device, and a call with uneven ones wants the split.) Shards that are not held count too: one
// of 8 with 256 tokens a row is split, 16.2 us for 8 rows and 41.9 for 200, where the same tokens alone take 12.0 and
// 33.1.
bool whole_rows(int cp, int64_t T, int64_t window, int64_t sinks) {
    const int64_t seen = window > 0 && window < T ? window : T, first = sinks < T ? sinks : T;
    const int64_t most = (seen + kTile - 1) / kTile + (window > 0 ? (first + kTile - 1) / kTile : 0);
    return cp * most <= 2;
}

}  // namespace

extern "C" int64_t dcp_mla_cache8_decode_workspace_bytes(int cp, int64_t B, int H, int64_t T, int64_t window,
                                                         int64_t sinks, int num_sms) {
    if (cp < 1 || cp > kCpMax || B < 0 || B > 65535 || H < 1 || H > 1024 || T < 0 || T > 0x7fffffff || window < 0 ||
        sinks < 0 || num_sms < 1 || num_sms > 4096)
        return -1;
    return B == 0 || whole_rows(cp, T, window, sinks) ? 0 : workspace_of(B, H, num_sms).bytes;
}

extern "C" int dcp_mla_cache8_decode(const void* q, int64_t q_row, int64_t q_head, const void* const* kv_ptrs,
                                     const float* const* scale_ptrs, const int32_t* seq_lens, int cp, int64_t B,
                                     int H, int Dk, int Dv, int64_t T, int block, int interleave, int64_t window,
                                     int64_t sinks, float scale, int lse_base_e, void* workspace,
                                     int64_t workspace_bytes, void* out, float* lse, int32_t* status, unsigned flags,
                                     void* stream) {
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
            p.held |= 1u << j;
            some = j;
        }
    }
    if (some < 0) return DCP_MLA_CACHE8_ERR_NULL_POINTER;
    // every tile count stays in 32 bits
    const int64_t shard_tiles = T / kTile + 2;
    if (B * cp * shard_tiles > 0x40000000) return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    if (B == 0) return 0;
    const int sms = multiprocessors();
    if (sms < 1) {
        (void)cudaGetLastError();
        return DCP_ERR_DEVICE;
    }
    const Workspace ws = workspace_of(B, H, sms);
    p.row_mode = whole_rows(cp, T, window, sinks) ? 1 : 0;
    if (!p.row_mode && (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < ws.bytes))
        return DCP_MLA_CACHE8_ERR_WORKSPACE;
    if (T == 0) p.held = 0;  // nothing is cached: every row is empty
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
    p.head_blocks = (H + head_block(H) - 1) / head_block(H);
    p.ranges = grid_ranges(H, sms);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.lse_scale = lse_base_e ? 0.6931471805599453f : 1.0f;
    p.stall = (flags & DCP_MLA_FLAG_TEST_STALL) ? 1 : 0;
    p.wait_ns = p.stall ? kTestWaitLimitNs : kWaitLimitNs;
    if (p.row_mode && p.ranges > B) p.ranges = (int)B;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (cp == 1) return run_decode<1>(p, kv_ptrs, scale_ptrs, Dk, flags, st);
    if (cp <= 4) return run_decode<4>(p, kv_ptrs, scale_ptrs, Dk, flags, st);
    return run_decode<kCpMax>(p, kv_ptrs, scale_ptrs, Dk, flags, st);
}
