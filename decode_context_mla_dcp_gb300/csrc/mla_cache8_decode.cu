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
//   own power-of-two scale for each 32 tokens: E = ceil(max over the 32 tokens of
//   s + log2 u), P = 2^(s + log2 u - E + 8) in (0, 256], and the tensor core
//   multiplies by 2^(E - M - 8) (block-scaled e4m3, one ue8m0 scale for 32
//   products). What a token of 2^-14 of its block's largest loses is below 2^-18
//   of that largest; the rest is exact to 2^-8, like bf16 probabilities.
// * The reference M is an integer per head that follows the largest E lazily:
//   it moves only when some E exceeds it by 32, which fp32 sums bear.
//
// Layout. The product is transposed so that the 128 tokens lie on the MMA's M:
//   S^T[128 tokens x 2 heads-blocks] = K_tile . Q^T      (18 MMAs of K = 32)
//   O^T[512 dims x heads]           += V_tile^T . P^T    (4 row blocks)
// The cached tile serves both products: K-major for the scores, M-major (read
// along the latent dims) for the values.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "dcp_lse_reduce.h"
#include "dcp_mla_cache8.h"

namespace {

constexpr int kDv = 512;
constexpr int kTile = 128;                 // tokens of a tile: the MMA's M
constexpr int kSlice = kTile * 128;        // bytes of a 128-dim slice of a tile
constexpr int kThreads = 512;
constexpr int kCpMax = DCP_MLA_CACHE8_CP_MAX;
constexpr int64_t kMaxInterleave = 1 << 24;
constexpr long long kWaitLimitNs = 2000000000LL;  // every wait gives up after this
constexpr int kFar = 1 << 28;              // beyond every exponent
constexpr int kLazy = 32;                  // how far an exponent may pass the reference

struct DecodeParams {
    CUtensorMap tm_latent[kCpMax];         // boxes of 128 dims x 128 tokens, 128-byte swizzle
    CUtensorMap tm_rope[kCpMax];           // boxes of 64 dims x 128 tokens, 64-byte swizzle
    const float* scales[kCpMax];
    const uint8_t* q;
    int64_t q_row, q_head;                 // bytes
    const int* seq_lens;
    float* part;                           // [2 x CTAs][heads of a block][512], normalised
    float* part_lse;                       // [2 x CTAs][heads of a block], base 2
    int* row_info;                         // [B] tiles before the row; [B]: tiles of a CTA
    uint8_t* out;
    float* lse;
    int* status;
    int64_t blocks;                        // scales of a row
    uint32_t held;                         // bit j: shard j is held
    uint32_t T, cp, interleave, window, sinks;
    int block_log2;
    int B, H, head_blocks, ranges;         // grid: head_blocks x ranges CTAs
    int min_tiles;
    int row_mode;                          // a range is whole rows (no row is split)
    float scale_log2;
    float lse_scale;                       // ln 2 for a natural-log LSE, 1 for base 2
    long long wait_ns;
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
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* tm, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
constexpr uint32_t kSwizzle128 = 2, kSwizzle64 = 4, kSwizzleNone = 0;
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
__device__ __forceinline__ void mma_f8_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                              uint32_t sfb, uint32_t acc) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
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
__device__ __forceinline__ Prefix prefix_of(const DecodeParams& p, uint32_t L) {
    if (p.cp == 1) return {0u, L};
    const uint32_t round = p.cp * p.interleave, q = L / round;
    return {q, L - q * round};
}
__device__ __forceinline__ uint32_t share(const DecodeParams& p, Prefix x, uint32_t j) {
    uint32_t n = x.r;
    if (p.cp > 1) {
        const uint32_t lo = j * p.interleave;
        n = x.r > lo ? x.r - lo : 0u;
        n = x.q * p.interleave + (n < p.interleave ? n : p.interleave);
    }
    return n < p.T ? n : p.T;
}
struct RowView {
    Prefix len, win, sink;
};
__device__ __forceinline__ RowView row_view(const DecodeParams& p, int b) {
    const int n = p.seq_lens[b];
    const uint32_t L = n < 0 ? 0u : (uint32_t)n;
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
__device__ __forceinline__ ShardView shard_view(const DecodeParams& p, const RowView& v, uint32_t j) {
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
__device__ __forceinline__ int row_tiles(const DecodeParams& p, int b) {
    const RowView v = row_view(p, b);
    int n = 0;
    for (uint32_t j = 0; j < p.cp; ++j) n += shard_view(p, v, j).tiles;
    return n;
}
// Walks a row's tiles over the shards.
struct Cursor {
    RowView row;
    ShardView s;
    uint32_t j;
    int i;  // tile of the shard
    __device__ __forceinline__ void seek(const DecodeParams& p, int b, int tile) {
        row = row_view(p, b);
        j = 0;
        s = shard_view(p, row, 0);
        i = tile;
        settle(p);
    }
    __device__ __forceinline__ void settle(const DecodeParams& p) {
        while (i >= s.tiles && j + 1 < p.cp) {
            i -= s.tiles;
            s = shard_view(p, row, ++j);
        }
    }
    __device__ __forceinline__ void next(const DecodeParams& p) {
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
    static constexpr int kPBytes = kStacked || !kLoInRope ? kRows * 128 : kNH * 128;
    static constexpr int kMisc = 1024 + 128 + 4 * kNH * 4;
    static constexpr int kSmem = 2 * kStage + kQBytes + kPBytes + kMisc;
    static constexpr int kHW = kNH / 4;                      // heads of a thread
    static constexpr int kO = kRows;                         // TMEM: S [0, rows), O 4 x kOB columns, scales
    static constexpr int kOB = kStacked ? kRows : kNH;
    static constexpr int kSf = kO + 4 * kOB;
    static constexpr int kCols = kSf + 12 <= 256 ? 256 : 512;
    static_assert(kSmem <= 232448 && kSf + 12 <= 512, "");
};

template <int kDk, int kNH>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const __grid_constant__ DecodeParams p) {
    using S = Shape<kDk, kNH>;
    constexpr int kHW = S::kHW;
    constexpr uint32_t kIdS = (1u << 4) | ((uint32_t)(S::kRows >> 3) << 17) | (8u << 24);
    constexpr uint32_t kIdO = ((uint32_t)((S::kStacked ? S::kRows : kNH) >> 3) << 17) | (1u << 23) | (8u << 24) |
                              (1u << 15);  // ue8m0 scales, A read M-major
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* const q_s = smem + 2 * S::kStage;
    uint8_t* const p_s = q_s + S::kQBytes;
    uint8_t* const sf_s = p_s + S::kPBytes;                       // two 512-byte scale atoms
    uint64_t* const bar_kv = reinterpret_cast<uint64_t*>(sf_s + 1024);  // [2] a tile has landed
    uint64_t* const bar_s = bar_kv + 2;                           // a tile's scores are there
    uint64_t* const bar_o = bar_kv + 3;                           // a tile's values are added
    uint32_t* const tslot = reinterpret_cast<uint32_t*>(bar_kv + 4);
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
    int* const find_s = reinterpret_cast<int*>(tslot + 2);        // [4]
    int* const wsum = reinterpret_cast<int*>(tslot + 6);          // [16]
    int* const m_s = reinterpret_cast<int*>(sf_s + 1024 + 128);   // reference exponents
    int* const mn_s = m_s + kNH;
    float* const a_s = reinterpret_cast<float*>(mn_s + kNH);      // rescale factors, then 1 / sums
    float* const g_s = a_s + kNH;                                 // q's scales

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int hblk = blockIdx.x % p.head_blocks, range = blockIdx.x / p.head_blocks;
    const int h0 = hblk * kNH;
    const int nh = p.H - h0 < kNH ? p.H - h0 : kNH;

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) mbar_init(bar_kv + i, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort_flag = 0;
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tslot)),
                     "r"(S::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    for (int i = tid; i < 256; i += kThreads) reinterpret_cast<uint32_t*>(sf_s)[i] = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const int quad = warp & 3, tok = quad * 32 + lane, hb = (warp >> 2) * kHW;
    const uint32_t tlane = tmem + ((uint32_t)(32 * quad) << 16);
    if (warp < 4) {  // the cached tile's scale is 1 everywhere: its own scale went into the probabilities
        const float one[4] = {__uint_as_float(0x7f7f7f7fu), __uint_as_float(0x7f7f7f7fu), __uint_as_float(0x7f7f7f7fu),
                              __uint_as_float(0x7f7f7f7fu)};
        tmem_st4(tlane + S::kSf, one);
        tmem_wait_st();
    }

    pdl_wait();
    pdl_launch_dependents();

    // ---- this CTA's tiles: [g, g_end) of all rows' tiles, from tile `tile` of row `row`
    int row = range, tile = 0, g = 0, g_end = 0;
    if (!p.row_mode) {
        int total = 0, n_mine = 0, pre_mine = 0;
        for (int pass = 0; pass < 2; ++pass) {
            int base = 0;
            if (pass == 1) {
                int per = (total + p.ranges - 1) / p.ranges;
                if (per < p.min_tiles) per = p.min_tiles;
                const int64_t lo = (int64_t)range * per, hi = lo + per;
                g = lo < total ? (int)lo : total;
                g_end = hi < total ? (int)hi : total;
                if (blockIdx.x == 0 && tid == 0) p.row_info[p.B] = per;
                if (tid == 0) find_s[0] = p.B;
                __syncthreads();
            }
            for (int b0 = 0; b0 < p.B; b0 += kThreads) {
                if (pass == 0 || p.B > kThreads) {
                    const int n = b0 + tid < p.B ? row_tiles(p, b0 + tid) : 0;
                    int x = n;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int y = __shfl_up_sync(0xffffffffu, x, o);
                        if (lane >= o) x += y;
                    }
                    if (lane == 31) wsum[warp] = x;
                    __syncthreads();
                    int before = 0, all = 0;
                    for (int w = 0; w < kThreads / 32; ++w) {
                        before += w < warp ? wsum[w] : 0;
                        all += wsum[w];
                    }
                    __syncthreads();
                    n_mine = n;
                    pre_mine = base + before + x - n;
                    base += all;
                }
                if (pass == 1) {
                    if (n_mine > 0 && pre_mine <= g && g < pre_mine + n_mine && g < g_end) {
                        find_s[0] = b0 + tid;
                        find_s[1] = g - pre_mine;
                    }
                    // the CTA that has a row's first tile says where the row lies
                    if (n_mine > 0 && hblk == 0 && pre_mine >= g && pre_mine < g_end)
                        p.row_info[b0 + tid] = pre_mine;
                }
            }
            if (pass == 0) total = base;
        }
        __syncthreads();
        row = find_s[0];
        tile = find_s[1];
    }

    uint32_t it = 0;        // tiles of this CTA so far: stage it & 1
    bool aborted = false;
    while (row < p.B && (p.row_mode || g < g_end)) {
        // ---- a segment: tiles [tile, tile + n) of this row
        const int n_row = row_tiles(p, row);
        const int n = p.row_mode || n_row - tile < g_end - g ? n_row - tile : g_end - g;
        if (n_row == 0) {
            if (p.row_mode) {
                uint4* const o = reinterpret_cast<uint4*>(p.out + ((int64_t)row * p.H + h0) * (kDv * 2));
                for (int i = tid; i < nh * (kDv / 8); i += kThreads) o[i] = make_uint4(0u, 0u, 0u, 0u);
                if (p.lse != nullptr && tid < nh) p.lse[(int64_t)row * p.H + h0 + tid] = -INFINITY;
            }
            row += p.row_mode ? p.ranges : 1;
            tile = 0;
            continue;
        }
        Cursor cur, ahead;
        cur.seek(p, row, tile);
        ahead = cur;
        auto load = [&](const Cursor& c, uint32_t k) {  // one thread: tile k of this CTA into its stage
            uint8_t* const kv = smem + (k & 1) * S::kStage;
            uint64_t* const bar = bar_kv + (k & 1);
            const int t0 = (int)c.token();
            mbar_expect_tx(bar, S::kStage);
#pragma unroll
            for (int a = 0; a < 4; ++a) tma_load_3d(kv + a * kSlice, &p.tm_latent[c.j], a * 128, t0, row, bar);
            if constexpr (S::kHasRope) tma_load_3d(kv + 4 * kSlice, &p.tm_rope[c.j], kDv, t0, row, bar);
        };
        if (tid == 0) load(ahead, it);

        // ---- q: hi and lo e4m3 parts of each head at its own power-of-two scale
        for (int h = warp; h < kNH; h += kThreads / 32) {
            uint32_t w[kDk / 64];
            const uint32_t* const src = reinterpret_cast<const uint32_t*>(p.q + row * p.q_row + (h0 + h) * p.q_head);
#pragma unroll
            for (int i = 0; i < kDk / 64; ++i) w[i] = h < nh ? __ldg(src + i * 32 + lane) : 0u;
            float top = 0.f;
#pragma unroll
            for (int i = 0; i < kDk / 64; ++i)
                top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const uint32_t u = __float_as_uint(top);
            int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // top <= 448 * 2^e
            e = e < -120 ? -120 : e;
            const bool bad = u >= 0x7f800000u;  // an infinity: the whole head is NaN (a NaN stays one by itself)
            const float inv = bad ? __uint_as_float(0x7fffffffu) : __uint_as_float((uint32_t)(127 - e) << 23);
            if (lane == 0) g_s[h] = bad ? 1.f : __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int i = 0; i < kDk / 64; ++i) {
                const float x = __uint_as_float(w[i] << 16) * inv, y = __uint_as_float(w[i] & 0xffff0000u) * inv;
                const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
                const float2 back = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(hi, __NV_E4M3)));
                const __nv_fp8x2_storage_t lo =
                    __nv_cvt_float2_to_fp8x2(make_float2(x - back.x, y - back.y), __NV_SATFINITE, __NV_E4M3);
                const int d = 64 * i + 2 * lane, c = (d & 127) >> 4;
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const int r = h + part * kNH;
                    uint8_t* dst;
                    if (S::kHasRope && i == kDv / 64)
                        dst = q_s + 4 * S::kQSlice + r * 64 + ((c ^ ((r >> 1) & 3)) << 4) + (d & 15);
                    else
                        dst = q_s + (d >> 7) * S::kQSlice + r * 128 + ((c ^ (r & 7)) << 4) + (d & 15);
                    *reinterpret_cast<__nv_fp8x2_storage_t*>(dst) = part ? lo : hi;
                }
            }
        }
        if (tid < kNH) m_s[tid] = -kFar;
        if (tid < kNH) mn_s[tid] = -kFar;
        async_fence();
        __syncthreads();

        float l_part[kHW];
#pragma unroll
        for (int h = 0; h < kHW; ++h) l_part[h] = 0.f;

        for (int i = 0; i < n; ++i, ++it) {
            if (__syncthreads_or(*abort_flag != 0)) {
                aborted = true;
                break;
            }
            uint8_t* const kv = smem + (it & 1) * S::kStage;
            const int valid = cur.valid();
            // this thread's token's scale, in flight beside the tile
            const uint32_t t_loc = cur.token() + (uint32_t)(tok < valid ? tok : valid - 1);
            const float u = fmaxf(p.scales[cur.j][(int64_t)row * p.blocks + (t_loc >> p.block_log2)], 7.888609e-31f);
            (void)mbar_wait(bar_kv + (it & 1), (it >> 1) & 1, abort_flag, p.status, p.wait_ns);
            if (tid == 0 && !*abort_flag) {  // scores
                tc_fence_after();
                const uint32_t ka = smem_u32(kv), qa = smem_u32(q_s);
#pragma unroll
                for (int a = 0; a < 4; ++a)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f8(tmem, smem_desc(ka + a * kSlice + k * 32, 16, 1024, kSwizzle128),
                               smem_desc(qa + a * S::kQSlice + k * 32, 16, 1024, kSwizzle128), kIdS, (a | k) != 0);
                if constexpr (S::kHasRope) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        mma_f8(tmem, smem_desc(ka + 4 * kSlice + k * 32, 16, 512, kSwizzle64),
                               smem_desc(qa + 4 * S::kQSlice + k * 32, 16, 512, kSwizzle64), kIdS, 1);
                }
                mma_commit(bar_s);
            }
            (void)mbar_wait(bar_s, it & 1, abort_flag, p.status, p.wait_ns);
            tc_fence_after();
            // (every MMA before these is done too: the other stage is free)
            if (tid == 0 && i + 1 < n && !*abort_flag) {
                ahead.next(p);
                load(ahead, it + 1);
            }

            float sv[kHW];
            {
                float lo[kHW];
                tmem_ld<kHW>(tlane + hb, sv);
                tmem_ld<kHW>(tlane + kNH + hb, lo);
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < kHW; ++h) sv[h] += lo[h];
            }
            const bool live = tok < valid;
            const float c = u * p.scale_log2, lu = log2f(u), ru = 1.0f / u;
            int e[kHW];
            bool over = false;
#pragma unroll
            for (int h = 0; h < kHW; ++h) {
                sv[h] = live ? fmaf(sv[h] * g_s[hb + h], c, lu) : -INFINITY;
                int x = __float2int_ru(sv[h]);
                x = __reduce_max_sync(0xffffffffu, x < -kFar ? -kFar : (x > kFar ? kFar : x));
                e[h] = x;
                over |= x - m_s[hb + h] > kLazy;
            }
            // a token that is not visible may hold anything: its value row must not (0 x NaN)
            if (!live) {
                uint4* const r = reinterpret_cast<uint4*>(kv + (warp >> 2) * kSlice + tok * 128);
#pragma unroll
                for (int k = 0; k < 8; ++k) r[(k + tok) & 7] = make_uint4(0u, 0u, 0u, 0u);
            }
            const bool move = __syncthreads_or(over);
            if (move) {
#pragma unroll
                for (int h = 0; h < kHW; ++h)
                    if (lane == 0) atomicMax(&mn_s[hb + h], e[h]);
                __syncthreads();
                if (tid < kNH) {
                    const int m = m_s[tid], mn = mn_s[tid] > m ? mn_s[tid] : m;
                    a_s[tid] = ex2((float)(m - mn));
                    m_s[tid] = mn;
                }
                __syncthreads();
#pragma unroll
                for (int h = 0; h < kHW; ++h) l_part[h] *= a_s[hb + h];
                if (i > 0) {
#pragma unroll 1
                    for (int b = 0; b < 4 * (S::kStacked ? 2 : 1); ++b) {
                        const uint32_t col = tlane + S::kO + (S::kStacked ? (b >> 1) * S::kOB + (b & 1) * kNH : b * S::kOB) + hb;
#pragma unroll
                        for (int h = 0; h < kHW; h += 4) {
                            float o[4];
                            tmem_ld<4>(col + h, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 4; ++k) o[k] *= a_s[hb + h + k];
                            tmem_st4(col + h, o);
                        }
                    }
                    tmem_wait_st();
                }
            }
            uint8_t* const p_lo = S::kStacked ? p_s + kNH * 128 : (S::kLoInRope ? kv + 4 * kSlice : p_s + kNH * 128);
            int sf = 0;
#pragma unroll
            for (int h = 0; h < kHW; h += 2) {
                float hi[2], lo[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float x = ex2(sv[h + k] - (float)(e[h + k] - 8));
                    int f = e[h + k] - m_s[hb + h + k] - 8 + 127;
                    f = f < 0 ? 0 : f;
                    if (lane == h + k) sf = f;
                    l_part[h + k] = fmaf(x * ru, __int_as_float(f << 23), l_part[h + k]);
                    // the nearest number of 4 significand bits, and the rest
                    hi[k] = __uint_as_float((__float_as_uint(x) + 0x80000u) & 0xfff00000u);
                    lo[k] = (x - hi[k]) * 32.f;
                }
                const uint32_t ch = __nv_cvt_float2_to_fp8x2(make_float2(hi[0], hi[1]), __NV_SATFINITE, __NV_E4M3);
                const uint32_t cl = __nv_cvt_float2_to_fp8x2(make_float2(lo[0], lo[1]), __NV_SATFINITE, __NV_E4M3);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int r = hb + h + k;
                    const int at = r * 128 + (((tok >> 4) ^ (r & 7)) << 4) + (tok & 15);
                    const int at_lo = S::kStacked ? r * 128 + (((tok >> 4) ^ ((r + kNH) & 7)) << 4) + (tok & 15) : at;
                    p_s[at] = (uint8_t)(ch >> (8 * k));
                    p_lo[at_lo] = (uint8_t)(cl >> (8 * k));
                }
            }
            if (lane < kHW) {
                const int r = hb + lane, r2 = S::kStacked ? r + kNH : r;
                const int lo = sf - 5;
                sf_s[(r & 31) * 16 + (r >> 5) * 4 + quad] = (uint8_t)sf;
                sf_s[(S::kStacked ? 0 : 512) + (r2 & 31) * 16 + (r2 >> 5) * 4 + quad] = (uint8_t)(lo < 0 ? 0 : lo);
            }
            async_fence();
            tc_fence_before();
            __syncthreads();
            if (tid == 0 && !*abort_flag) {  // values
                tc_fence_after();
                copy_scales(tmem + S::kSf + 4, smem_u32(sf_s));
                if constexpr (!S::kStacked) copy_scales(tmem + S::kSf + 8, smem_u32(sf_s + 512));
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int part = 0; part < (S::kStacked ? 1 : 2); ++part)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_f8_scaled(tmem + S::kO + m * S::kOB,
                                          smem_desc(smem_u32(kv + m * kSlice) + k * 4096, kSlice, 1024, kSwizzle128),
                                          smem_desc(smem_u32(part ? p_lo : p_s) + k * 32, 16, 1024, kSwizzle128),
                                          kIdO | ((uint32_t)k << 4) | ((uint32_t)k << 29), tmem + S::kSf,
                                          tmem + S::kSf + 4 + 4 * part, (i > 0 || part > 0 || k > 0) ? 1u : 0u);
                mma_commit(bar_o);
            }
            cur.next(p);
        }
        if (aborted) break;

        // ---- the segment's end: sums, then O / l
        (void)mbar_wait(bar_o, (it - 1) & 1, abort_flag, p.status, p.wait_ns);
        if (__syncthreads_or(*abort_flag != 0)) {
            aborted = true;
            break;
        }
        tc_fence_after();
        float* const red = reinterpret_cast<float*>(p_s);  // [4][kNH]
#pragma unroll
        for (int h = 0; h < kHW; ++h) {
            float x = l_part[h];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            if (lane == 0) red[quad * kNH + hb + h] = x;
        }
        __syncthreads();
        const bool whole = tile == 0 && n == n_row;  // the row's only segment
        const int64_t slot = (int64_t)blockIdx.x * 2 + (tile == 0 ? 1 : 0);
        if (tid < kNH) {
            const float l = (red[tid] + red[kNH + tid]) + (red[2 * kNH + tid] + red[3 * kNH + tid]);
            a_s[tid] = 1.0f / l;
            const float lse2 = (float)m_s[tid] + log2f(l);
            if (!whole) p.part_lse[slot * kNH + tid] = lse2;
            else if (p.lse != nullptr && tid < nh) p.lse[(int64_t)row * p.H + h0 + tid] = lse2 * p.lse_scale;
        }
        __syncthreads();
#pragma unroll 1
        for (int m = 0; m < 4; ++m) {
            float o[kHW];
            tmem_ld<kHW>(tlane + S::kO + m * S::kOB + hb, o);
            if constexpr (S::kStacked) {
                float lo[kHW];
                tmem_ld<kHW>(tlane + S::kO + m * S::kOB + kNH + hb, lo);
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < kHW; ++h) o[h] += lo[h];
            }
            tmem_wait_ld();
            const int d = 128 * m + tok;  // lane = latent dim
#pragma unroll
            for (int h = 0; h < kHW; ++h) {
                const float x = o[h] * a_s[hb + h];
                if (whole) reinterpret_cast<__nv_bfloat16*>(smem)[(hb + h) * kDv + d] = __float2bfloat16_rn(x);
                else reinterpret_cast<float*>(smem)[(hb + h) * kDv + d] = x;
            }
        }
        async_fence();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (tid == 0) {
            void* const dst = whole ? static_cast<void*>(p.out + ((int64_t)row * p.H + h0) * (kDv * 2))
                                    : static_cast<void*>(p.part + slot * (kNH * kDv));
            asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                         "r"(smem_u32(smem)), "r"((uint32_t)(nh * kDv * (whole ? 2 : 4)))
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        }
        __syncthreads();
        g += n;
        row += p.row_mode ? p.ranges : 1;
        tile = 0;
    }
    if (aborted) {
        // A wait gave up. Before the CTA leaves, wait (bounded) for what may still
        // be in flight: the tile loads and MMAs of the last two tiles.
        __syncthreads();
        if (tid == 0) {
            for (uint32_t k = 0; k < 2; ++k) {
                mbar_drain(bar_kv + k, 0, p.wait_ns);
                mbar_drain(bar_kv + k, 1, p.wait_ns);
            }
            mbar_drain(bar_s, it & 1, p.wait_ns);
            mbar_drain(bar_o, it & 1, p.wait_ns);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kCols) : "memory");
}

// ---- the rows that were split ---------------------------------------------------------

// One warp (or kWarps warps, where there are few rows and many segments of each)
// per (row, head): the segments' outputs weighted by 2^(lse - max), and the row's
// LSE. Rows with one segment have been written; rows without a tile get zeros.
template <int kWarps>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ DecodeParams p, int heads_of_block) {
    __shared__ float acc_s[8][kDv];
    __shared__ float sum_s[8];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * (8 / kWarps) + warp / kWarps;
    if (unit >= (int64_t)p.B * p.H) return;
    const int b = (int)(unit / p.H), h = (int)(unit - (int64_t)b * p.H);
    const int n = row_tiles(p, b);
    uint4* const out = reinterpret_cast<uint4*>(p.out + unit * (kDv * 2));
    const int w = warp % kWarps;
    if (n == 0) {
        if (w == 0) {
            out[lane] = make_uint4(0u, 0u, 0u, 0u);
            out[32 + lane] = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse != nullptr && lane == 0) p.lse[unit] = -INFINITY;
        }
        return;
    }
    const int per = p.row_info[p.B], pre = p.row_info[b];
    const int k0 = pre / per, k1 = (pre + n - 1) / per;
    if (k0 == k1) return;
    const int hblk = h / heads_of_block, hh = h - hblk * heads_of_block;
    auto slot = [&](int k) { return ((int64_t)k * p.head_blocks + hblk) * 2 + (k == k0 ? 1 : 0); };
    float m = -INFINITY;
    bool nan = false;
    for (int k = k0 + lane; k <= k1; k += 32) {
        const float x = p.part_lse[slot(k) * heads_of_block + hh];
        nan |= isnan(x);
        m = fmaxf(m, x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (__any_sync(0xffffffffu, nan)) m = __uint_as_float(0x7fffffffu);
    float acc[16], sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
#pragma unroll 2
    for (int k = k0 + w; k <= k1; k += kWarps) {
        const int64_t s = slot(k);
        const float4* const src = reinterpret_cast<const float4*>(p.part + (s * heads_of_block + hh) * kDv);
        float4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = src[i * 32 + lane];
        const float f = ex2(p.part_lse[s * heads_of_block + hh] - m);
        sum += f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            acc[4 * i] = fmaf(f, x[i].x, acc[4 * i]);
            acc[4 * i + 1] = fmaf(f, x[i].y, acc[4 * i + 1]);
            acc[4 * i + 2] = fmaf(f, x[i].z, acc[4 * i + 2]);
            acc[4 * i + 3] = fmaf(f, x[i].w, acc[4 * i + 3]);
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
        for (int v = 0; v < kWarps; ++v) sum += sum_s[v];
        const float inv = 1.0f / sum;
        const int d = threadIdx.x * 2;
        float a = 0.f, c = 0.f;
        for (int v = 0; v < kWarps; ++v) {
            a += acc_s[v][d];
            c += acc_s[v][d + 1];
        }
        reinterpret_cast<__nv_bfloat162*>(out)[threadIdx.x] = __floats2bfloat162_rn(a * inv, c * inv);
        if (p.lse != nullptr && threadIdx.x == 0) p.lse[unit] = (m + log2f(sum)) * p.lse_scale;
    } else {
        const float inv = 1.0f / sum;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint2 v;
            const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[4 * i] * inv, acc[4 * i + 1] * inv);
            const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[4 * i + 2] * inv, acc[4 * i + 3] * inv);
            v.x = *reinterpret_cast<const uint32_t*>(&lo);
            v.y = *reinterpret_cast<const uint32_t*>(&hi);
            reinterpret_cast<uint2*>(out)[i * 32 + lane] = v;
        }
        if (p.lse != nullptr && lane == 0) p.lse[unit] = (m + log2f(sum)) * p.lse_scale;
    }
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
    w.bytes = w.row_info + round_up((B + 1) * 4);
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

template <int kDk, int kNH>
cudaError_t launch_decode(const DecodeParams& p, unsigned flags, cudaStream_t st) {
    constexpr int bytes = Shape<kDk, kNH>::kSmem;
    static int configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
        e = cudaFuncSetAttribute(decode_kernel<kDk, kNH>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
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
    e = cudaLaunchKernelEx(&cfg, decode_kernel<kDk, kNH>, p);
    if (e != cudaSuccess || p.row_mode) return e;
    // the join overlaps its launch with the decode's tail and waits for it on the device
    const int64_t units = (int64_t)p.B * p.H;
    const bool few = units <= 512;
    cfg.gridDim = dim3((unsigned)(few ? units : (units + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return few ? cudaLaunchKernelEx(&cfg, join_kernel<8>, p, (int)kNH)
               : cudaLaunchKernelEx(&cfg, join_kernel<1>, p, (int)kNH);
}

template <int kDk>
cudaError_t launch_decode_dk(const DecodeParams& p, unsigned flags, cudaStream_t st) {
    const int nh = head_block(p.H);
    if (nh == 16) return launch_decode<kDk, 16>(p, flags, st);
    if (nh == 32) return launch_decode<kDk, 32>(p, flags, st);
    return launch_decode<kDk, 64>(p, flags, st);
}

}  // namespace

extern "C" int64_t dcp_mla_cache8_decode_workspace_bytes(int64_t B, int H, int num_sms) {
    if (B < 0 || B > 65535 || H < 1 || H > 1024 || num_sms < 1 || num_sms > 4096) return -1;
    return workspace_of(B, H, num_sms).bytes;
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
    if ((flags & ~(unsigned)DCP_FLAG_PDL) != 0) return DCP_MLA_CACHE8_ERR_BAD_FLAGS;
    if (q == nullptr || kv_ptrs == nullptr || scale_ptrs == nullptr || seq_lens == nullptr || out == nullptr)
        return DCP_MLA_CACHE8_ERR_NULL_POINTER;
    if (!aligned(q, 4) || q_row % 2 != 0 || q_head % 2 != 0 || !aligned(out, 16) || !aligned(lse, 4) ||
        !aligned(seq_lens, 4) || !aligned(status, 4))
        return DCP_MLA_CACHE8_ERR_MISALIGNED;
    DecodeParams p;
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
    if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < ws.bytes)
        return DCP_MLA_CACHE8_ERR_WORKSPACE;
    if (T == 0) p.held = 0;  // nothing is cached: every row is empty
    for (int j = 0; j < kCpMax; ++j) {
        p.scales[j] = j < cp ? scale_ptrs[j] : nullptr;
        if (T > 0 && j < cp && kv_ptrs[j] != nullptr) {
            if (!encode_cache(&p.tm_latent[j], kv_ptrs[j], Dk, T, B, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
                (Dk > kDv && !encode_cache(&p.tm_rope[j], kv_ptrs[j], Dk, T, B, 64, CU_TENSOR_MAP_SWIZZLE_64B)))
                return DCP_MLA_CACHE8_ERR_TENSOR_MAP;
        }
    }
    uint8_t* const w = static_cast<uint8_t*>(workspace);
    p.q = static_cast<const uint8_t*>(q);
    p.q_row = q_row * 2;
    p.q_head = q_head * 2;
    p.seq_lens = seq_lens;
    p.part = reinterpret_cast<float*>(w + ws.part);
    p.part_lse = reinterpret_cast<float*>(w + ws.part_lse);
    p.row_info = reinterpret_cast<int*>(w + ws.row_info);
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
    p.min_tiles = 1;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.lse_scale = lse_base_e ? 0.6931471805599453f : 1.0f;
    p.wait_ns = kWaitLimitNs;
    // Rows of at most two tiles are not worth splitting: a join costs as much.
    const int64_t span = window > 0 && window < T ? window + kTile - 1 : T;
    const int64_t row_most = (int64_t)cp * ((span + kTile - 1) / kTile + (sinks > 0 ? (sinks + kTile - 1) / kTile : 0));
    p.row_mode = row_most <= 2 ? 1 : 0;
    if (p.row_mode && p.ranges > B) p.ranges = (int)B;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = Dk == 576 ? launch_decode_dk<576>(p, flags, st) : launch_decode_dk<512>(p, flags, st);
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        return (int)e;
    }
    return 0;
}
