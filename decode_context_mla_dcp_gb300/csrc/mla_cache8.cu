// The 8-bit latent cache's elementwise operators, sm_103a: rotary positions, the
// quantising append and the read-back. What they compute, and the cache's
// format, are stated in include/dcp_mla_cache8.h; the attention over the cache
// is in mla_cache8_decode.cu.
//
// All three move bytes and compute little: a few operations per element
// against 2 to 4 bytes. Their floors are DRAM time for large calls and one
// launch plus a few dependent memory round trips for small ones. So loads are
// 8 or 16 bytes a lane and issued before any is used, and everything that a
// token needs (its row, shard, place, angles) is found once and shared.
// Measured, against a copy's 6.79 TB/s: rotating 64 of 192 dims of 8,192 x 64
// heads 60.6 us (0.98), 128 x 128 heads x 64 into other rows 2.4 us; reading
// 262,144 tokens back from four shards 68.4 us (0.97), 2,047 tokens 3.0 us;
// appending 16,385 tokens in blocks of 64 9.2 us (0.45: two round trips before
// the tokens' own, and two barriers), 256 x 4 tokens over four shards 5.6 us, one
// token 1.9 to 2.1 us. Many tokens of one head stay far from the floor: 30,000 of
// 288 dims, 128 rotated, 15.3 us in halves and 12.7 interleaved against 5.1. A
// CTA's loads, its angles and its stores follow one another. Moving the data alone
// takes 9.2 and 6.7; the angles add 6 (without sine and cosine 4.6 and 3.4 of it
// stay: positions, 64-bit products, shared memory).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "dcp_lse_reduce.h"
#include "dcp_mla_cache8.h"
#include "dcp_mla_pages.h"

namespace {

constexpr int kLatent = 512;
constexpr int kCpMax = DCP_MLA_CACHE8_CP_MAX;
constexpr int kMinExp = -60;              // a scale is at least 2^-60
constexpr int64_t kMaxInterleave = 1 << 24;
constexpr int kSms = 152;  // GB300's multiprocessors, for the launch rules below: with another count they cost time only

// ---- element types -------------------------------------------------------------

struct Bf16 {
    // the larger magnitudes of two pairs; NaN loses to a number
    __device__ static uint32_t top2(uint32_t a, uint32_t b) {
        const __nv_bfloat162 m = __hmax2(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                         __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
    using T = uint16_t;
    __device__ static float get(T v) { return __uint_as_float((uint32_t)v << 16); }
    __device__ static T put(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
};
struct F16 {
    __device__ static uint32_t top2(uint32_t a, uint32_t b) {
        const __half2 m = __hmax2(__habs2(*reinterpret_cast<const __half2*>(&a)),
                                  __habs2(*reinterpret_cast<const __half2*>(&b)));
        return *reinterpret_cast<const uint32_t*>(&m);
    }
    using T = uint16_t;
    __device__ static float get(T v) { return __half2float(__ushort_as_half(v)); }
    __device__ static T put(float x) { return __half_as_ushort(__float2half_rn(x)); }
};
struct F32 {
    using T = float;
    __device__ static float get(T v) { return v; }
    __device__ static T put(float x) { return x; }
};

// The low and high 16-bit element of a 32-bit word.
template <class E>
__device__ __forceinline__ float get_lo(uint32_t w) { return E::get((uint16_t)(w & 0xffffu)); }
template <class E>
__device__ __forceinline__ float get_hi(uint32_t w) { return E::get((uint16_t)(w >> 16)); }

// ---- angles --------------------------------------------------------------------

// Turns per position as a 64-bit fraction of a turn: multiplying it by a
// position wraps at whole turns exactly, so a far position loses nothing but
// the fraction's last place. In integers, for 64-bit floating point is slow here
// (30,000 tokens of one head of 288 dims: 26.6 us with it, 19.6 without, 15.3 with
// each CTA's frequencies taken into turns once): the double is m 2^(e - 1075), and
// 1 / (2 pi) is kTurn 2^-66. A frequency that is not finite gives kNoTurns, whose
// cosine and sine are NaN (a finite one that has these low bits is the last place off).
constexpr uint32_t kNoTurns = 0x80000001u;
constexpr float kNaN = __builtin_nanf("");
__device__ __forceinline__ uint64_t turns_of(double inv_freq) {
    constexpr uint64_t kTurn = 0xa2f9836e4e44152aull;
    const int64_t bits = __double_as_longlong(inv_freq);
    const int s = 1077 - ((int)(bits >> 52) & 0x7ff);  // what the 117-bit product has to be shifted right by
    const uint64_t m = ((uint64_t)bits & 0xfffffffffffffull) | (1ull << 52);
    const uint64_t lo = m * kTurn, hi = __umul64hi(m, kTurn);
    const uint64_t u = s >= 128  ? 0
                       : s >= 64 ? hi >> (s - 64)
                       : s > 0   ? (lo >> s) | (hi << (64 - s))
                       : s > -64 ? lo << -s
                                 : 0;
    const uint64_t turns = bits < 0 ? 0 - u : u;
    if (s == 1077 - 0x7ff) return kNoTurns;
    return (uint32_t)turns == kNoTurns ? turns - 1 : turns;
}

// cos and sin of position * frequency, from the top 32 bits of the wrapped
// product read as half turns in [-1, 1).
__device__ __forceinline__ void angle_of(int64_t pos, uint64_t turns, float* c, float* s) {
    const uint64_t phase = (uint64_t)pos * turns;
    const float unit = (uint32_t)turns == kNoTurns ? kNaN : 4.656612873077393e-10f;  // 2^-31
    sincospif((float)(int32_t)(uint32_t)(phase >> 32) * unit, s, c);
}

// The same to fp32's last places, for values that are then rounded to a coarse grid, where a small error moves the few
// that lie beside a boundary a whole step: the quarter of a turn is taken out of the integer first, so that its
// conversion keeps 2^-27 of a half turn. (Keys on another code than in 64 bits: 1 to 4 in 260,000 to 1,050,000, the plain
// form in 32 bits 0 to 8; 1 to 12 with the form above, 6 to 29 with the hardware's sine and cosine, which saved 4% of a
// prompt's append in blocks of 64, 7% with a scale each.)
__device__ __forceinline__ void fine_angle_of(int64_t pos, uint64_t turns, float* c, float* s) {
    const uint32_t phase = (uint32_t)(((uint64_t)pos * turns) >> 32);
    const float unit = (uint32_t)turns == kNoTurns ? kNaN : 4.656612873077393e-10f;  // 2^-31
    const uint32_t quarter = (phase + 0x20000000u) >> 30;
    float x, y;
    sincospif((float)(int32_t)(phase - (quarter << 30)) * unit, &y, &x);
    const float u = quarter & 1 ? y : x, v = quarter & 1 ? x : y;
    *c = (quarter + 1) & 2 ? -u : u;
    *s = quarter & 2 ? -v : v;
}

// ---- rotary positions ------------------------------------------------------------

struct RopeParams {
    const void* x;
    void* out;
    const void* positions;
    const double* inv_freq;
    int64_t x_row, x_head, out_row, out_head;  // elements
    int64_t N;
    int H, start, half;      // half = rot / 2
    int interleaved, pos64, copy;
    float mscale;
    int tokens;              // tokens of a CTA
    int heads;               // heads of a CTA
    int slots;               // rows that the CTA's threads cover side by side
    int rot_units, units;    // work units of a head: rotating ones first, then copied ones
    int copy_lead;           // copied units before the rotated dims
};

constexpr int kRopeThreads = 256;
constexpr int kRopeAngles = 2048;  // cos/sin pairs a CTA holds
constexpr int kRopeHalf = 128;     // pairs of a head, at most
constexpr int kRopeBatch = 4;      // 16-byte vectors a thread has in flight

// A unit is kV elements (16 bytes) of a head, or with halves two of them (kV
// pairs); kV = 1 is the form for sizes or strides that are not multiples of 16
// bytes: a unit is one pair or one copied element.
template <class E, int kV, bool kInter>
struct RopeUnit {
    using T = typename E::T;
    static constexpr int kE = kInter && kV == 1 ? 2 : kV;  // elements of a vector
    static constexpr int kA = kInter ? kE / 2 : kE;        // angles
    struct alignas(kV * sizeof(T)) Vec { T e[kE]; };
    Vec v, w;
    // Each byte is used once: 16-byte accesses stream (evict first), which a large call gains 15% by.
    __device__ __forceinline__ static Vec get(const T* src) {
        if constexpr (sizeof(Vec) == 16) {
            const uint4 q = __ldcs(reinterpret_cast<const uint4*>(src));
            return *reinterpret_cast<const Vec*>(&q);
        } else {
            return *reinterpret_cast<const Vec*>(src);
        }
    }
    __device__ __forceinline__ static void put(T* dst, const Vec& x) {
        if constexpr (sizeof(Vec) == 16) __stcs(reinterpret_cast<uint4*>(dst), *reinterpret_cast<const uint4*>(&x));
        else *reinterpret_cast<Vec*>(dst) = x;
    }
    __device__ __forceinline__ void load(const T* src, int half, bool turn) {
        if (kE == kV) {
            v = get(src);
        } else {
            v.e[0] = src[0];
            if (turn) v.e[kE - 1] = src[1];
        }
        if (!kInter && turn) w = get(src + half);
    }
    __device__ __forceinline__ void turn_by(const float2* a) {
#pragma unroll
        for (int j = 0; j < kA; ++j) {
            T& p = v.e[kInter ? 2 * j : j];
            T& q = kInter ? v.e[kInter ? 2 * j + 1 : 0] : w.e[j];
            const float f = E::get(p), g = E::get(q);
            p = E::put(f * a[j].x - g * a[j].y);
            q = E::put(g * a[j].x + f * a[j].y);
        }
    }
    __device__ __forceinline__ void store(T* dst, int half, bool turn) const {
        if (kE == kV) {
            put(dst, v);
        } else {
            dst[0] = v.e[0];
            if (turn) dst[1] = v.e[kE - 1];
        }
        if (!kInter && turn) put(dst + half, w);
    }
};

// One CTA: `tokens` tokens x `heads` heads, the rows. A thread keeps one unit of
// the row and walks the rows in steps of `slots` (the rows that the CTA's threads
// cover side by side), so that its place in the row, its kind, its step and (with
// one token a CTA, !kMany) its angles are found once. It loads its first rows,
// then the CTA computes its tokens' angles (64-bit multiply, sincos) once into
// shared memory, then the rows are turned and stored: the angles cost their
// latency beside the loads'.
template <class E, int kV, bool kInter, bool kMany>
__global__ void __launch_bounds__(kRopeThreads, kMany ? 5 : 4)
rope_kernel(const __grid_constant__ RopeParams p) {
    using Unit = RopeUnit<E, kV, kInter>;
    using T = typename E::T;
    constexpr int kB = kInter ? kRopeBatch : kRopeBatch / 2;
    // (five CTAs a multiprocessor where a CTA has many tokens: 8,192 x 16 heads x 64 9.1 -> 8.1 us; four elsewhere: with
    // five the prompt's rotation spills, 60.5 -> 67.9 us, with its registers not limited it has fewer CTAs, 63.6)
    __shared__ alignas(16) float2 cs[kRopeAngles];
    __shared__ uint64_t turn_s[kMany ? kRopeHalf : 1];
    const int64_t n0 = (int64_t)blockIdx.x * p.tokens;
    const int ntok = kMany ? (int)(p.N - n0 < p.tokens ? p.N - n0 : p.tokens) : 1;
    const int h0 = blockIdx.y * p.heads;
    const int nh = p.H - h0 < p.heads ? p.H - h0 : p.heads;
    const int rows = ntok * nh;
    const int slots = p.slots, threads = (int)blockDim.x;
    const int slot = slots > 1 ? (int)threadIdx.x / p.units : 0;
    // the place of row `slot`, and a step of `slots` rows: tokens, heads, and on to the next token past the last head
    const int tok0 = kMany ? slot / nh : 0, head0 = slot - tok0 * nh;
    const int toks = kMany ? slots / nh : 0, hs = slots - toks * nh;
    const int64_t x_step = toks * p.x_row + hs * p.x_head, out_step = toks * p.out_row + hs * p.out_head;
    const int64_t x_wrap = p.x_row - nh * p.x_head, out_wrap = p.out_row - nh * p.out_head;
    bool angles = false;
    for (int u = (int)threadIdx.x - slot * p.units;; u += threads) {
        const bool turn = u < p.rot_units;
        const int c = u - p.rot_units;  // a copied unit lies before or behind the rotated dims
        const int d = turn ? p.start + u * Unit::kE
                           : (c < p.copy_lead ? c * kV : p.start + 2 * p.half + (c - p.copy_lead) * kV);
        const T* src = static_cast<const T*>(p.x) + ((n0 + tok0) * p.x_row + (h0 + head0) * p.x_head + d);
        T* dst = static_cast<T*>(p.out) + ((n0 + tok0) * p.out_row + (h0 + head0) * p.out_head + d);
        const float2* at = cs + tok0 * p.half + u * Unit::kA;
        int r = slot < slots && u < p.units ? slot : rows, h = head0, ht = head0;
        float2 mine[Unit::kA];
        do {
            Unit v[kB];
#pragma unroll
            for (int k = 0; k < kB; ++k) {
                if (r + k * slots < rows) {
                    v[k].load(src, p.half, turn);
                    src += x_step;
                    h += hs;
                    if (kMany && h >= nh) {
                        h -= nh;
                        src += x_wrap;
                    }
                }
            }
            if (!angles) {
                // (with many tokens the frequencies are taken into turns once, and no angle costs a division)
                if (kMany) {
                    for (int f = threadIdx.x; f < p.half; f += threads) turn_s[f] = turns_of(p.inv_freq[f]);
                    __syncthreads();
                }
                int tok = kMany ? (int)threadIdx.x / p.half : 0, f = (int)threadIdx.x - tok * p.half;
                const int dtok = kMany ? threads / p.half : 0, df = threads - dtok * p.half;
                for (int i = threadIdx.x; i < ntok * p.half; i += threads) {
                    const int64_t pos = p.pos64 ? static_cast<const int64_t*>(p.positions)[n0 + tok]
                                                : (int64_t) static_cast<const int32_t*>(p.positions)[n0 + tok];
                    float co, si;
                    angle_of(pos, kMany ? turn_s[f] : turns_of(p.inv_freq[f]), &co, &si);
                    cs[i] = make_float2(co * p.mscale, si * p.mscale);
                    tok += dtok;
                    f += df;
                    if (kMany && f >= p.half) {
                        f -= p.half;
                        ++tok;
                    }
                }
                __syncthreads();  // (every thread comes here once, with its first rows)
                angles = true;
            }
            if (!kMany && turn) {
#pragma unroll
                for (int j = 0; j < Unit::kA; ++j) mine[j] = at[j];
            }
#pragma unroll
            for (int k = 0; k < kB; ++k) {
                if (r + k * slots < rows) {
                    if (turn) v[k].turn_by(kMany ? at : mine);
                    v[k].store(dst, p.half, turn);
                    dst += out_step;
                    at += toks * p.half;
                    ht += hs;
                    if (kMany && ht >= nh) {
                        ht -= nh;
                        dst += out_wrap;
                        at += p.half;
                    }
                }
            }
            r += kB * slots;
        } while (r < rows);
        if (slots > 1 || u + threads >= p.units) break;
    }
}

// ---- rows of packed tokens ----------------------------------------------------------

// Row of packed token n: a b with cu[b] <= n < cu[b + 1], whatever cu holds; -1
// before cu[0] or past cu[B].
__device__ __forceinline__ int row_of(const int32_t* cu, int B, int64_t n) {
    if (n < cu[0] || n >= cu[B]) return -1;
    int lo = 0, hi = B;  // cu[lo] <= n < cu[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu[mid] <= n) lo = mid; else hi = mid;
    }
    return lo;
}

// Shard j's share of the first L positions of a row.
__device__ __forceinline__ uint32_t held_tokens(uint32_t L, int j, uint32_t cp, uint32_t interleave) {
    if (cp == 1) return L;
    const uint32_t round = cp * interleave, q = L / round, r = L - q * round, lo = (uint32_t)j * interleave;
    const uint32_t part = r > lo ? r - lo : 0;
    return q * interleave + (part < interleave ? part : interleave);
}

// ---- quantising ----------------------------------------------------------------------

// Exponent k of the smallest power of two with a <= 448 * 2^k, at least -60.
// 448 = 1.75 * 2^8: a = m * 2^e with 1 <= m < 2 needs k = e - 8, or e - 7 above 1.75.
__device__ __forceinline__ int scale_exp(float a) {
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 127;
    const int k = e - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return k < kMinExp ? kMinExp : k;  // (a subnormal or zero a has e = -127)
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }
// |x| of a finite x, 0 of a NaN or an infinity
__device__ __forceinline__ float mag(float x) { return finite(x) ? fabsf(x) : 0.f; }
// Two e4m3 codes (first in the low byte), round to nearest even. kOdd: NaN for an infinity too (the conversion gives
// the largest number).
template <bool kOdd>
__device__ __forceinline__ uint32_t codes2(float x, float y, float inv) {
    const float a = !kOdd || finite(x) ? x * inv : __uint_as_float(0x7fffffffu);
    const float b = !kOdd || finite(y) ? y * inv : __uint_as_float(0x7fffffffu);
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 values2(uint32_t codes) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3);
    return __half22float2(__half2(h));
}

struct AppendParams {
    const uint8_t* latent;
    const uint8_t* k_rope;
    int64_t latent_row, rope_row;  // bytes
    const int32_t* cu;             // or NULL: `even` tokens a row
    const int32_t* seq_lens;
    const double* inv_freq;
    uint8_t* kv[kCpMax];
    float* scales[kCpMax];
    int64_t N, T, blocks;          // blocks: scales of a row
    int B, Dk, even;
    uint32_t cp, interleave;
    int block_log2, interleaved;
    float mscale;
};

// A cache in pages: tables, and the pool's sizes. T is what a row's table has room for.
struct Tables {
    const int32_t* of[kCpMax];
    int64_t M;
    int P, page_log2;
};
struct PagedAppendParams : AppendParams {
    Tables tables;
};

// The place of token `loc` of a row in shard j's cache, in tokens; negative: it has none.
template <class P>
__device__ __forceinline__ int64_t row_place(const P& p, int, int row, uint32_t loc) {
    return (int64_t)row * p.T + loc;
}
__device__ __forceinline__ int64_t table_place(const Tables& t, int j, int row, uint32_t loc) {
    const int e = t.of[j][row * t.M + (loc >> t.page_log2)];
    return e >= 0 && e < t.P ? ((int64_t)e << t.page_log2) + (loc & ((1u << t.page_log2) - 1)) : -1;
}
__device__ __forceinline__ int64_t token_place(const AppendParams& p, int j, int row, uint32_t loc) {
    return row_place(p, j, row, loc);
}
__device__ __forceinline__ int64_t token_place(const PagedAppendParams& p, int j, int row, uint32_t loc) {
    return table_place(p.tables, j, row, loc);
}
// That of its block's scale (a page is whole blocks; a row's last block may be a part of one).
template <class P>
__device__ __forceinline__ int64_t row_scale(const P& p, int row, int64_t, uint32_t loc) {
    return (int64_t)row * p.blocks + (loc >> p.block_log2);
}
__device__ __forceinline__ int64_t scale_place(const AppendParams& p, int row, int64_t at, uint32_t loc) {
    return row_scale(p, row, at, loc);
}
__device__ __forceinline__ int64_t scale_place(const PagedAppendParams& p, int, int64_t at, uint32_t) {
    return at >> p.block_log2;
}

// A token in a warp's registers: lane l holds latent dims 8l .. 8l+7 and
// 256 + 8l .. 256 + 8l + 7 as they are, and the rotated rotary pair l.
struct Token {
    uint4 v[2];
    float r0, r1;
};

template <class E>
__device__ __forceinline__ void load_token(const AppendParams& p, int64_t src, int lane, Token* t, uint32_t* rope) {
    const uint4* const row = reinterpret_cast<const uint4*>(p.latent + src * p.latent_row);
    t->v[0] = __ldg(row + lane);
    t->v[1] = __ldg(row + 32 + lane);
    if (p.Dk > kLatent) {
        const uint8_t* const r = p.k_rope + src * p.rope_row;
        if (p.interleaved) {
            *rope = __ldg(reinterpret_cast<const uint32_t*>(r) + lane);
        } else {
            const uint16_t* const e = reinterpret_cast<const uint16_t*>(r);
            *rope = (uint32_t)__ldg(e + lane) | ((uint32_t)__ldg(e + 32 + lane) << 16);
        }
    }
}

template <class E>
__device__ __forceinline__ void turn_token(const AppendParams& p, uint32_t rope, bool rotate, uint64_t turns,
                                           int64_t pos, Token* t) {
    t->r0 = t->r1 = 0.f;
    if (p.Dk > kLatent) {
        t->r0 = get_lo<E>(rope);
        t->r1 = get_hi<E>(rope);
        if (rotate) {
            float c, s;
            fine_angle_of(pos, turns, &c, &s);
            c *= p.mscale;
            s *= p.mscale;
            const float a = t->r0, b = t->r1;
            t->r0 = a * c - b * s;
            t->r1 = b * c + a * s;
        }
    }
}

// A lane's largest magnitude of a token, cheaply: packed maxima, in which a NaN
// loses to a number. Where that or a rotated value is no finite number (`odd`) the
// warp looks at its tokens again one value at a time.
template <class E>
__device__ __forceinline__ float lane_top(const Token& t, bool* odd) {
    const uint32_t w[8] = {t.v[0].x, t.v[0].y, t.v[0].z, t.v[0].w, t.v[1].x, t.v[1].y, t.v[1].z, t.v[1].w};
    uint32_t m = E::top2(w[0], w[1]);
#pragma unroll
    for (int i = 2; i < 8; ++i) m = E::top2(m, w[i]);
    const float a = fmaxf(fmaxf(get_lo<E>(m), get_hi<E>(m)), fmaxf(fabsf(t.r0), fabsf(t.r1)));
    *odd |= !finite(a) || !finite(t.r0 + t.r1);
    return a;
}
template <class E>
__device__ __forceinline__ float lane_finite_top(const Token& t) {
    const uint32_t w[8] = {t.v[0].x, t.v[0].y, t.v[0].z, t.v[0].w, t.v[1].x, t.v[1].y, t.v[1].z, t.v[1].w};
    float a = fmaxf(mag(t.r0), mag(t.r1));
#pragma unroll
    for (int i = 0; i < 8; ++i) a = fmaxf(a, fmaxf(mag(get_lo<E>(w[i])), mag(get_hi<E>(w[i]))));
    return a;
}
// (magnitudes: their bits order like integers)
__device__ __forceinline__ float warp_top(float a) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(a)));
}

template <class E, bool kOdd>
__device__ __forceinline__ void store_codes(const AppendParams& p, const Token& t, uint8_t* dst, int lane, float inv) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t w[4] = {t.v[k].x, t.v[k].y, t.v[k].z, t.v[k].w};
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = codes2<kOdd>(get_lo<E>(w[i]), get_hi<E>(w[i]), inv);
        *reinterpret_cast<uint2*>(dst + 256 * k + 8 * lane) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
    }
    if (p.Dk > kLatent) {
        const uint32_t c = codes2<kOdd>(t.r0, t.r1, inv);
        if (p.interleaved) {
            *reinterpret_cast<uint16_t*>(dst + kLatent + 2 * lane) = (uint16_t)c;
        } else {
            dst[kLatent + lane] = (uint8_t)c;
            dst[kLatent + 32 + lane] = (uint8_t)(c >> 8);
        }
    }
}
template <class E>
__device__ __forceinline__ void store_token(const AppendParams& p, const Token& t, bool odd, uint8_t* dst, int lane,
                                            float inv) {
    if (odd) store_codes<E, true>(p, t, dst, lane, inv);
    else store_codes<E, false>(p, t, dst, lane, inv);
}

// Where packed token n goes. False: nowhere.
struct Place {
    int row, shard;
    uint32_t first, count, len;  // the row's first packed token, its new tokens, its length before
    uint32_t pos, loc, end;      // its position; its token of the shard; the shard's tokens after the call
};
__device__ __forceinline__ bool place_of(const AppendParams& p, const int32_t* cu, int64_t n, Place* w) {
    if (p.cu != nullptr) {
        w->row = row_of(cu, p.B, n);
        if (w->row < 0) return false;
        const int64_t first = cu[w->row], last = cu[w->row + 1] < p.N ? cu[w->row + 1] : p.N;
        if (first < 0) return false;
        w->first = (uint32_t)first;
        w->count = (uint32_t)(last - first);
    } else {
        w->row = (int)((uint32_t)n / (uint32_t)p.even);
        w->first = (uint32_t)w->row * (uint32_t)p.even;
        w->count = (uint32_t)p.even;
    }
    const int32_t len = p.seq_lens[w->row];
    w->len = len < 0 ? 0u : (uint32_t)len;
    w->pos = w->len + ((uint32_t)n - w->first);
    if (p.cp == 1) {
        w->shard = 0;
        w->loc = w->pos;
    } else {
        const uint32_t turn = w->pos / p.interleave, q = turn / p.cp;
        w->shard = (int)(turn - q * p.cp);
        w->loc = q * p.interleave + (w->pos - turn * p.interleave);
    }
    return true;
}

// Each token its own scale: a warp takes a token, one round trip for its data. (One token 1.9 us, 256 x 4 tokens over
// four shards 3.7, 16,385 tokens 7.5; the kernel of blocks took 3.0, 5.0 and 59 for them.)
template <class E, class Q>
__global__ void __launch_bounds__(128) append_token_kernel(const __grid_constant__ Q p) {
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (n >= p.N) return;
    Token t;
    uint32_t rope = 0;
    load_token<E>(p, n, lane, &t, &rope);  // the packed inputs have N rows, whether the token has a place or not
    const bool rotate = p.inv_freq != nullptr;
    const double f = rotate ? p.inv_freq[lane] : 0.0;
    Place w;
    if (!place_of(p, p.cu, n, &w) || (int64_t)w.loc >= p.T) return;
    uint8_t* const kv = p.kv[w.shard];
    if (kv == nullptr) return;
    const int64_t at = token_place(p, w.shard, w.row, w.loc);
    if (at < 0) return;
    turn_token<E>(p, rope, rotate, turns_of(f), (int64_t)w.pos, &t);
    bool odd = false;
    float top = lane_top<E>(t, &odd);
    odd = __any_sync(0xffffffffu, odd);
    if (odd) top = lane_finite_top<E>(t);
    const int k = scale_exp(warp_top(top));
    store_token<E>(p, t, odd, kv + at * p.Dk, lane, pow2(-k));
    if (lane == 0) p.scales[w.shard][at] = pow2(k);
}

// Blocks of tokens. A CTA writes whole blocks: a block's new tokens in registers
// (kTok a warp, every load in flight at once), their peak, the scale, the tokens
// that the block held before if the scale grows, and the new codes. A CTA has as
// many warps as a block needs, so that small blocks take small CTAs and all CTAs
// of a call are resident at once.
//
// Which blocks. kCounted: the CTA's warps count the blocks of all rows, 32 rows
// each in turn, once; then CTA c takes blocks c, c + G, ... of all rows' and
// shards' blocks in order, and every warp looks through the 32 rows that hold one.
// That spreads any mix of rows evenly and costs two round trips, but goes over all
// rows. Otherwise the first new token of a block (of a row, on a shard) stands for
// it: CTA c looks at tokens c, c + G, c + 2G, ... (a binary search each) with G odd,
// so that first tokens, which stand a power of two apart, spread over the CTAs; yet
// some CTAs find several. Counting is for up to kCountedRows rows and calls of more
// tokens than CTAs are resident. (16,385 tokens of 5 rows in blocks of 64: 9.2 us
// counted, 15.5 by first tokens; of 256 rows over four shards in blocks of 16 16.5
// and 23.5; of 1,024 rows over two shards in blocks of 64 50.2 and 26.5; 256 x 4
// tokens over four shards 6.1 and 5.6; 300 tokens of 256 rows 4.6 and 4.4.)
constexpr int kTok = 4;
constexpr int kCuShared = 1024;
constexpr int kCountedRows = 512;

// A row's new tokens, and how many blocks of all its held shards get some. The first L positions lie in q whole
// rounds over the shards and r positions of another, which cp shards ask for one division each.
struct NewTokens {
    uint32_t first, len, count;
    int blocks;
};
struct Part {
    uint32_t before, after;  // the shard's tokens
    int blocks;
};
__device__ __forceinline__ uint32_t part_of(const AppendParams& p, uint32_t L, uint32_t q, uint32_t j) {
    const uint32_t r = L - q * p.cp * p.interleave, lo = j * p.interleave, n = r > lo ? r - lo : 0;
    return q * p.interleave + (n < p.interleave ? n : p.interleave);
}
__device__ __forceinline__ Part shard_part(const AppendParams& p, uint32_t L0, uint32_t q0, uint32_t L1, uint32_t q1,
                                           int j) {
    Part s;
    s.before = p.cp == 1 ? L0 : part_of(p, L0, q0, (uint32_t)j);
    s.after = p.cp == 1 ? L1 : part_of(p, L1, q1, (uint32_t)j);
    if ((int64_t)s.after > p.T) s.after = (uint32_t)p.T;
    s.blocks = s.after > s.before && p.kv[j] != nullptr
                   ? (int)(((s.after - 1) >> p.block_log2) - (s.before >> p.block_log2)) + 1
                   : 0;
    return s;
}
__device__ __forceinline__ NewTokens new_tokens(const AppendParams& p, int b) {
    NewTokens r = {0u, 0u, 0u, 0};
    if (b >= p.B) return r;
    int64_t first = (int64_t)b * p.even, last = first + p.even;
    if (p.cu != nullptr) {
        first = p.cu[b];
        last = p.cu[b + 1];
    }
    const int32_t len = p.seq_lens[b];
    if (last > p.N) last = p.N;
    if (first < 0 || last <= first) return r;
    r.first = (uint32_t)first;
    r.count = (uint32_t)(last - first);
    r.len = len < 0 ? 0u : (uint32_t)len;
    const uint32_t round = p.cp * p.interleave, end = r.len + r.count;
    const uint32_t q0 = p.cp == 1 ? 0u : r.len / round, q1 = p.cp == 1 ? 0u : end / round;
    for (int j = 0; j < (int)p.cp; ++j) r.blocks += shard_part(p, r.len, q0, end, q1, j).blocks;
    return r;
}
// Inclusive sum over the warp's lanes.
__device__ __forceinline__ int lane_sums(int x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

template <class E, int kWarps, bool kCounted, class Q>
__global__ void __launch_bounds__(32 * kWarps, 32 / kWarps)
append_block_kernel(const __grid_constant__ Q p) {
    __shared__ int32_t cu_s[kCounted ? kCountedRows / 32 : kCuShared + 1];
    __shared__ Place list[kCounted ? 1 : 32 * kWarps];
    __shared__ int64_t at_s[kCounted ? 1 : 32 * kWarps];  // the listed blocks' places
    __shared__ int found;
    __shared__ float peak_s[kWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool rotate = p.inv_freq != nullptr;
    const double freq = rotate ? p.inv_freq[lane] : 0.0;
    const uint32_t block = 1u << p.block_log2;
    const int32_t* cu = p.cu;
    if constexpr (!kCounted) {
        if (tid == 0) found = 0;
        if (cu != nullptr && p.B <= kCuShared) {
            for (int i = tid; i <= p.B; i += 32 * kWarps) cu_s[i] = cu[i];
            cu = cu_s;
        }
    }
    const int chunks = (p.B + 31) / 32;  // of rows (counted: fewer than 32)
    if constexpr (kCounted) {
        for (int c = warp; c < chunks; c += kWarps) {
            const int n = __reduce_add_sync(0xffffffffu, new_tokens(p, c * 32 + lane).blocks);
            if (lane == 0) cu_s[c] = n;
        }
        __syncthreads();
    }
    for (int64_t base = blockIdx.x; base < p.N; base += (int64_t)gridDim.x * (kCounted ? 1 : 32 * kWarps)) {
        Place w;
        int nfound = 1;
        if constexpr (kCounted) {
            int u = (int)base;
            const int n = lane < chunks ? cu_s[lane] : 0;
            int sum = lane_sums(n, lane);
            uint32_t past = __ballot_sync(0xffffffffu, sum > u);
            if (!past) return;
            const int chunk = __ffs(past) - 1;
            u -= __shfl_sync(0xffffffffu, sum - n, chunk);
            const NewTokens r = new_tokens(p, chunk * 32 + lane);
            sum = lane_sums(r.blocks, lane);
            past = __ballot_sync(0xffffffffu, sum > u);
            if (!past) return;
            int l = __ffs(past) - 1;
            u -= __shfl_sync(0xffffffffu, sum - r.blocks, l);
            w.row = chunk * 32 + l;
            w.first = __shfl_sync(0xffffffffu, r.first, l);
            w.len = __shfl_sync(0xffffffffu, r.len, l);
            const uint32_t end = w.len + __shfl_sync(0xffffffffu, r.count, l);
            Part s = {0u, 0u, 0};  // a lane a shard
            if (lane < (int)p.cp) {
                const uint32_t round = p.cp * p.interleave;
                s = shard_part(p, w.len, p.cp == 1 ? 0u : w.len / round, end, p.cp == 1 ? 0u : end / round, lane);
            }
            sum = lane_sums(s.blocks, lane);
            past = __ballot_sync(0xffffffffu, sum > u);
            if (!past) return;
            l = __ffs(past) - 1;
            u -= __shfl_sync(0xffffffffu, sum - s.blocks, l);
            w.shard = l;
            w.end = __shfl_sync(0xffffffffu, s.after, l);
            const uint32_t before = __shfl_sync(0xffffffffu, s.before, l);
            w.loc = ((before >> p.block_log2) + (uint32_t)u) << p.block_log2;
            if (w.loc < before) w.loc = before;
            if (u < 0 || w.loc >= w.end) return;  // (only with offsets that are not in order)
        } else {
            __syncthreads();
            const int64_t n = base + (int64_t)tid * gridDim.x;
            if (n < p.N && place_of(p, cu, n, &w) && (int64_t)w.loc < p.T && p.kv[w.shard] != nullptr) {
                const uint32_t held = held_tokens(w.len, w.shard, p.cp, p.interleave);
                if (w.loc == held || (w.loc & (block - 1)) == 0) {
                    w.end = held_tokens(w.len + w.count, w.shard, p.cp, p.interleave);
                    if ((int64_t)w.end > p.T) w.end = (uint32_t)p.T;
                    // (only what has a place is listed: for each of those the CTA meets, before `found` begins again)
                    const int64_t at = token_place(p, w.shard, w.row, w.loc & ~(block - 1));
                    if (at >= 0) {
                        const int k = atomicAdd(&found, 1);
                        list[k] = w;
                        at_s[k] = at;
                    }
                }
            }
            __syncthreads();
            nfound = found;
        }
        for (int i = 0; i < nfound; ++i) {  // (in any order: blocks are independent of each other)
            if constexpr (!kCounted) w = list[i];
            const uint32_t b0 = w.loc & ~(block - 1);
            int64_t at;
            if constexpr (kCounted) {
                at = token_place(p, w.shard, w.row, b0);
                if (at < 0) continue;  // (the same in every thread, and nothing else is shared between turns)
            } else {
                at = at_s[i];
            }
            uint8_t* const kv = p.kv[w.shard] + (at - b0) * p.Dk;  // as if of token 0
            float* const scale = p.scales[w.shard] + scale_place(p, w.row, at, b0);
            const uint32_t end = w.end < b0 + block ? w.end : b0 + block;
            Token t[kTok];
            uint32_t rope[kTok], pos[kTok];
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                const uint32_t loc = w.loc + warp + k * kWarps;
                if (loc < end) {
                    pos[k] = p.cp == 1 ? loc
                                       : (loc / p.interleave * p.cp + w.shard) * p.interleave + loc % p.interleave;
                    load_token<E>(p, (int64_t)w.first + (pos[k] - w.len), lane, &t[k], &rope[k]);
                }
            }
            const float old = b0 < w.loc ? *scale : 0.f;  // the present scale counts where the block holds tokens
            const uint64_t turns = turns_of(freq);
            float peak = 0.f;
            bool odd = false;
#pragma unroll
            for (int k = 0; k < kTok; ++k)
                if (w.loc + warp + k * kWarps < end) {
                    turn_token<E>(p, rope[k], rotate, turns, (int64_t)pos[k], &t[k]);
                    peak = fmaxf(peak, lane_top<E>(t[k], &odd));
                }
            odd = __any_sync(0xffffffffu, odd);
            if (odd) {
                peak = 0.f;
#pragma unroll
                for (int k = 0; k < kTok; ++k)
                    if (w.loc + warp + k * kWarps < end) peak = fmaxf(peak, lane_finite_top<E>(t[k]));
            }
            peak = warp_top(peak);
            if (lane == 0) peak_s[warp] = peak;
            __syncthreads();
            peak = warp_top(peak_s[lane & (kWarps - 1)]);
            const int e = scale_exp(peak);
            float s = pow2(e);
            if (old > s) s = old;
            const float inv = 1.0f / s;
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                const uint32_t loc = w.loc + warp + k * kWarps;
                if (loc < end) store_token<E>(p, t[k], odd, kv + (int64_t)loc * p.Dk, lane, inv);
            }
            if (b0 < w.loc && s > old) {  // requantise what the block held
                const float ratio = old / s;
                for (uint32_t loc = b0 + warp; loc < w.loc; loc += kWarps) {
                    uint32_t* const row = reinterpret_cast<uint32_t*>(kv + (int64_t)loc * p.Dk);
                    for (int c = lane; c < p.Dk / 4; c += 32) {
                        const uint32_t u = row[c];
                        const float2 a = values2(u), b = values2(u >> 16);
                        row[c] = codes2<false>(a.x, a.y, ratio) | (codes2<false>(b.x, b.y, ratio) << 16);
                    }
                }
            }
            if (tid == 0) *scale = s;
            __syncthreads();  // peak_s is used again
        }
        if (!kCounted && tid == 0) found = 0;
    }
}

// ---- read-back -------------------------------------------------------------------------

struct ReadParams {
    const uint8_t* kv[kCpMax];
    const float* scales[kCpMax];
    const int32_t* starts;
    const int32_t* cu;
    uint8_t* out;
    int64_t out_row;  // bytes
    int64_t N, T, blocks;
    int B, even, block_log2;
    uint32_t cp, interleave;
    int tokens;       // tokens of a CTA
};
struct PagedReadParams : ReadParams {
    Tables tables;
};
__device__ __forceinline__ int64_t token_place(const ReadParams& p, int j, int row, uint32_t loc) {
    return row_place(p, j, row, loc);
}
__device__ __forceinline__ int64_t token_place(const PagedReadParams& p, int j, int row, uint32_t loc) {
    return table_place(p.tables, j, row, loc);
}
__device__ __forceinline__ int64_t scale_place(const ReadParams& p, int row, int64_t at, uint32_t loc) {
    return row_scale(p, row, at, loc);
}
__device__ __forceinline__ int64_t scale_place(const PagedReadParams& p, int, int64_t at, uint32_t) {
    return at >> p.block_log2;
}

constexpr int kReadThreads = 256;
constexpr int kReadTokens = 32;

__device__ __forceinline__ uint2 load_once(const uint8_t* src) {
    uint2 v;
    asm("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(src));
    return v;
}

// A CTA finds its tokens' places once, then moves 8 codes a thread: 8-byte
// loads, 16-byte stores of 16-bit values, both contiguous over the token.
template <class E, int kDk, class Q>
__global__ void __launch_bounds__(kReadThreads) read_kernel(const __grid_constant__ Q p) {
    using T = typename E::T;
    constexpr int kUnits = kDk / 8;  // 8 codes: 72 or 64 a token, a whole number of sweeps for 32 tokens
    __shared__ const uint8_t* src_s[kReadTokens];
    __shared__ float scale_s[kReadTokens];
    const int64_t n0 = (int64_t)blockIdx.x * p.tokens;
    const int ntok = (int)(p.N - n0 < p.tokens ? p.N - n0 : p.tokens);
    if ((int)threadIdx.x < ntok) {
        const int64_t n = n0 + threadIdx.x;
        const uint8_t* src = nullptr;
        float s = 0.f;
        int row = -1;
        uint32_t i = 0;
        if (p.cu != nullptr) {
            row = row_of(p.cu, p.B, n);
            if (row >= 0) i = (uint32_t)(n - p.cu[row]);
        } else {
            row = (int)((uint32_t)n / (uint32_t)p.even);
            i = (uint32_t)n - (uint32_t)row * (uint32_t)p.even;
        }
        if (row >= 0) {
            const int32_t start = p.starts != nullptr ? p.starts[row] : 0;
            const int64_t pos64 = (int64_t)start + i;
            if (pos64 >= 0) {
                const uint32_t pos = (uint32_t)pos64;
                int shard = 0;
                uint32_t loc = pos;
                if (p.cp > 1) {
                    const uint32_t turn = pos / p.interleave, q = turn / p.cp;
                    shard = (int)(turn - q * p.cp);
                    loc = q * p.interleave + (pos - turn * p.interleave);
                }
                if ((int64_t)loc < p.T && p.kv[shard] != nullptr) {
                    const int64_t at = token_place(p, shard, row, loc);
                    if (at >= 0) {
                        src = p.kv[shard] + at * kDk;
                        s = p.scales[shard][scale_place(p, row, at, loc)];
                    }
                }
            }
        }
        src_s[threadIdx.x] = src;
        scale_s[threadIdx.x] = s;
    }
    __syncthreads();
    // all loads of a thread in flight (a CTA's 32 tokens: nine, or eight of a 512-wide cache)
    constexpr int kBatch = kReadTokens * kUnits / kReadThreads;
    const int total = ntok * kUnits;
    uint2 c[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int i = k * kReadThreads + (int)threadIdx.x, t = i / kUnits, u = i - t * kUnits;
        c[k] = make_uint2(0u, 0u);
        if (i < total && src_s[t] != nullptr) c[k] = load_once(src_s[t] + 8 * u);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
        const int i = k * kReadThreads + (int)threadIdx.x, t = i / kUnits, u = i - t * kUnits;
        if (i < total && src_s[t] != nullptr) {
            const float s = scale_s[t];
            const float2 a = values2(c[k].x), b = values2(c[k].x >> 16), d = values2(c[k].y), e = values2(c[k].y >> 16);
            struct alignas(16) Vec { T e[8]; } v = {{E::put(a.x * s), E::put(a.y * s), E::put(b.x * s),
                                                     E::put(b.y * s), E::put(d.x * s), E::put(d.y * s),
                                                     E::put(e.x * s), E::put(e.y * s)}};
            uint4* const to = reinterpret_cast<uint4*>(p.out + (n0 + t) * p.out_row + (int64_t)u * sizeof(Vec));
#pragma unroll
            for (int j = 0; j < (int)(sizeof(Vec) / 16); ++j) __stcs(to + j, reinterpret_cast<const uint4*>(&v)[j]);
        }
    }
}

// ---- host side ---------------------------------------------------------------------------

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int launched() {
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? 0 : (int)e;
}

int log2_of(int block) {
    for (int k = 0; (1 << k) <= DCP_MLA_CACHE8_BLOCK_MAX; ++k)
        if (block == 1 << k) return k;
    return -1;
}

int check_shards(const void* const* kv, const float* const* scales, int cp, int64_t interleave) {
    if (cp < 1 || cp > kCpMax || interleave < 1 || interleave > kMaxInterleave) return DCP_MLA_CACHE8_ERR_BAD_CP;
    if (kv == nullptr || scales == nullptr) return DCP_MLA_CACHE8_ERR_NULL_POINTER;
    bool any = false;
    for (int j = 0; j < cp; ++j) {
        if ((kv[j] == nullptr) != (scales[j] == nullptr)) return DCP_MLA_CACHE8_ERR_NULL_POINTER;
        if (!aligned(kv[j], 16) || !aligned(scales[j], 4)) return DCP_MLA_CACHE8_ERR_MISALIGNED;
        any |= kv[j] != nullptr;
    }
    return any ? 0 : DCP_MLA_CACHE8_ERR_NULL_POINTER;
}

template <class E>
int launch_rope(RopeParams& p, int D, int64_t esize, cudaStream_t st) {
    // 16-byte units where every address that a unit can take allows it
    const int v = (int)(16 / esize);
    const bool al = (reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.out)) % 16 == 0 &&
                    (p.x_row | p.x_head | p.out_row | p.out_head) % v == 0 && p.start % v == 0 &&
                    (p.interleaved ? 2 * p.half : p.half) % v == 0 && (!p.copy || D % v == 0);
    const int kv = al ? v : 1;
    p.rot_units = p.interleaved ? (kv > 1 ? 2 * p.half / kv : p.half) : p.half / kv;
    p.copy_lead = p.copy ? p.start / kv : 0;
    p.units = p.rot_units + (p.copy ? (D - 2 * p.half) / kv : 0);
    // Rows side by side: a power of two, as counts of heads mostly are, so that no slot idles in the last step.
    // Tokens and heads of a CTA: at most about two batches of rows a thread, fewer where the call is small, so that
    // it still spreads over the GPU. More than one token only with all their heads.
    int64_t want = p.N * p.H / (kSms * 4);  // rows
    int slots = 1;
    while (2 * slots * p.units <= kRopeThreads && (slots < want || slots * p.units < 32)) slots *= 2;
    p.slots = slots;
    const int threads = slots * p.units < kRopeThreads ? (slots * p.units + 31) / 32 * 32 : kRopeThreads;
    const int64_t batch = (int64_t)slots * (p.interleaved ? kRopeBatch : kRopeBatch / 2);
    want = want < slots ? slots : (want > 2 * batch ? 2 * batch : want);
    const int64_t parts = (p.H + want - 1) / want, heads = (p.H + parts - 1) / parts;
    int64_t tokens = heads < p.H ? 1 : want / heads;
    if (tokens > kRopeAngles / p.half) tokens = kRopeAngles / p.half;
    tokens = tokens < 1 ? 1 : (tokens > p.N ? p.N : tokens);
    p.heads = (int)heads;
    p.tokens = (int)tokens;
    const int64_t gx = (p.N + tokens - 1) / tokens, gy = (p.H + heads - 1) / heads;
    if (gx > 0x7fffffff || gy > 65535) return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    const dim3 grid((unsigned)gx, (unsigned)gy);
    constexpr int kWide = 16 / sizeof(typename E::T);
    void (*kernel)(const RopeParams);
    if (tokens > 1) {
        if (p.interleaved) kernel = kv > 1 ? rope_kernel<E, kWide, true, true> : rope_kernel<E, 1, true, true>;
        else kernel = kv > 1 ? rope_kernel<E, kWide, false, true> : rope_kernel<E, 1, false, true>;
    } else {
        if (p.interleaved) kernel = kv > 1 ? rope_kernel<E, kWide, true, false> : rope_kernel<E, 1, true, false>;
        else kernel = kv > 1 ? rope_kernel<E, kWide, false, false> : rope_kernel<E, 1, false, false>;
    }
    kernel<<<grid, threads, 0, st>>>(p);
    return launched();
}

template <class E, class Q>
int launch_append(const Q& p, int block, cudaStream_t st) {
    if (block == 1) {
        append_token_kernel<E, Q><<<(unsigned)((p.N + 3) / 4), 128, 0, st>>>(p);
        return launched();
    }
    // about as many CTAs as are resident at once (32 warps a multiprocessor), an odd number
    const int warps = block <= 16 ? 4 : block / 4, resident = kSms * (32 / warps) + 1;
    const unsigned grid = (unsigned)(p.N < resident ? p.N : resident);
    if (p.N > resident && p.B <= kCountedRows) {
        if (warps == 4) append_block_kernel<E, 4, true, Q><<<grid, 128, 0, st>>>(p);
        else if (warps == 8) append_block_kernel<E, 8, true, Q><<<grid, 256, 0, st>>>(p);
        else if (warps == 16) append_block_kernel<E, 16, true, Q><<<grid, 512, 0, st>>>(p);
        else append_block_kernel<E, 32, true, Q><<<grid, 1024, 0, st>>>(p);
    } else {
        if (warps == 4) append_block_kernel<E, 4, false, Q><<<grid, 128, 0, st>>>(p);
        else if (warps == 8) append_block_kernel<E, 8, false, Q><<<grid, 256, 0, st>>>(p);
        else if (warps == 16) append_block_kernel<E, 16, false, Q><<<grid, 512, 0, st>>>(p);
        else append_block_kernel<E, 32, false, Q><<<grid, 1024, 0, st>>>(p);
    }
    return launched();
}

template <class E, class Q>
int launch_read(const Q& p, int Dk, cudaStream_t st) {
    const unsigned grid = (unsigned)((p.N + p.tokens - 1) / p.tokens);
    if (Dk == 576) read_kernel<E, 576, Q><<<grid, kReadThreads, 0, st>>>(p);
    else read_kernel<E, 512, Q><<<grid, kReadThreads, 0, st>>>(p);
    return launched();
}

// The checks and parameters that both forms of the append share; `room` tokens of a row on a shard, `blocks` scales.
int append_params(const void* latent, int64_t latent_row, const void* k_rope, int64_t rope_row, int dtype, int64_t N,
                  int64_t B, int Dk, const int32_t* cu_new, const int32_t* seq_lens, void* const* kv_ptrs,
                  float* const* scale_ptrs, int cp, int64_t T, int block, int interleave, const double* inv_freq,
                  int interleaved, float mscale, bool empty, AppendParams* p, bool* nothing) {
    *nothing = false;
    if (N < 0 || N > 0x7fffffff || B < 0 || B > 65535 || T < 0 || T > 0x7fffffff || (Dk != 512 && Dk != 576) ||
        (cu_new == nullptr && B > 0 && N % B != 0) || (B == 0 && N > 0))
        return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    if (dtype != DCP_DTYPE_BF16 && dtype != DCP_DTYPE_F16) return DCP_MLA_CACHE8_ERR_BAD_DTYPE;
    const int lg = log2_of(block);
    if (lg < 0) return DCP_MLA_CACHE8_ERR_BAD_BLOCK;
    if (const int rc = check_shards(kv_ptrs, scale_ptrs, cp, interleave)) return rc;
    // (a cache that stands for two shards would be written by both at once)
    for (int j = 0; j < cp; ++j)
        for (int k = 0; k < j; ++k)
            if (!empty && kv_ptrs[j] != nullptr && (kv_ptrs[j] == kv_ptrs[k] || scale_ptrs[j] == scale_ptrs[k]))
                return DCP_MLA_CACHE8_ERR_BAD_CP;
    if (N == 0 || empty) {
        *nothing = true;
        return 0;
    }
    if (latent == nullptr || seq_lens == nullptr || (Dk == 576 && k_rope == nullptr))
        return DCP_MLA_CACHE8_ERR_NULL_POINTER;
    if (!aligned(latent, 16) || !aligned(k_rope, 16) || latent_row % 8 != 0 || (Dk == 576 && rope_row % 8 != 0) ||
        !aligned(seq_lens, 4) || !aligned(cu_new, 4) || !aligned(inv_freq, 8))
        return DCP_MLA_CACHE8_ERR_MISALIGNED;
    p->latent = static_cast<const uint8_t*>(latent);
    p->k_rope = static_cast<const uint8_t*>(k_rope);
    p->latent_row = latent_row * 2;
    p->rope_row = rope_row * 2;
    p->cu = cu_new;
    p->seq_lens = seq_lens;
    p->inv_freq = Dk == 576 ? inv_freq : nullptr;
    for (int j = 0; j < cp; ++j) {
        p->kv[j] = static_cast<uint8_t*>(kv_ptrs[j]);
        p->scales[j] = scale_ptrs[j];
    }
    p->N = N;
    p->T = T;
    p->blocks = (T + block - 1) / block;
    p->B = (int)B;
    p->Dk = Dk;
    p->even = cu_new == nullptr ? (int)(N / B) : 0;
    p->cp = (uint32_t)cp;
    p->interleave = (uint32_t)interleave;
    p->block_log2 = lg;
    p->interleaved = interleaved != 0;
    p->mscale = mscale;
    return 0;
}

// The same for the read-back.
int read_params(const void* const* kv_ptrs, const float* const* scale_ptrs, int cp, int64_t B, int64_t T, int Dk,
                int block, int interleave, const int32_t* starts, const int32_t* cu, int64_t N, void* out,
                int64_t out_row, int dtype, bool empty, ReadParams* p, bool* nothing) {
    *nothing = false;
    if (N < 0 || N > 0x7fffffff || B < 0 || B > 65535 || T < 0 || T > 0x7fffffff || (Dk != 512 && Dk != 576) ||
        (cu == nullptr && B > 0 && N % B != 0) || (B == 0 && N > 0))
        return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    if (dtype != DCP_DTYPE_BF16 && dtype != DCP_DTYPE_F16 && dtype != DCP_DTYPE_F32)
        return DCP_MLA_CACHE8_ERR_BAD_DTYPE;
    const int lg = log2_of(block);
    if (lg < 0) return DCP_MLA_CACHE8_ERR_BAD_BLOCK;
    if (const int rc = check_shards(kv_ptrs, scale_ptrs, cp, interleave)) return rc;
    if (N == 0 || empty) {
        *nothing = true;
        return 0;
    }
    if (out == nullptr) return DCP_MLA_CACHE8_ERR_NULL_POINTER;
    const int64_t esize = dtype == DCP_DTYPE_F32 ? 4 : 2;
    if (!aligned(out, 16) || (out_row * esize) % 16 != 0 || !aligned(starts, 4) || !aligned(cu, 4))
        return DCP_MLA_CACHE8_ERR_MISALIGNED;
    for (int j = 0; j < cp; ++j) {
        p->kv[j] = static_cast<const uint8_t*>(kv_ptrs[j]);
        p->scales[j] = scale_ptrs[j];
    }
    p->starts = starts;
    p->cu = cu;
    p->out = static_cast<uint8_t*>(out);
    p->out_row = out_row * esize;
    p->N = N;
    p->T = T;
    p->blocks = (T + block - 1) / block;
    p->B = (int)B;
    p->even = cu == nullptr ? (int)(N / B) : 0;
    p->block_log2 = lg;
    p->cp = (uint32_t)cp;
    p->interleave = (uint32_t)interleave;
    // 32 tokens a CTA, 8 where that would leave multiprocessors idle (2,047 tokens: 3.0 us with 8, 3.6 with 32; 8,192
    // tokens: 5.3 and 4.5; 262,144: 99 and 69)
    p->tokens = N >= kSms * kReadTokens ? kReadTokens : 8;
    return 0;
}

template <class Q>
int run_append(const Q& p, int dtype, int block, cudaStream_t st) {
    return dtype == DCP_DTYPE_BF16 ? launch_append<Bf16>(p, block, st) : launch_append<F16>(p, block, st);
}
template <class Q>
int run_read(const Q& p, int dtype, int Dk, cudaStream_t st) {
    if (dtype == DCP_DTYPE_BF16) return launch_read<Bf16>(p, Dk, st);
    if (dtype == DCP_DTYPE_F16) return launch_read<F16>(p, Dk, st);
    return launch_read<F32>(p, Dk, st);
}

// The tables of the shards that are held.
int tables_of(const void* const* kv_ptrs, const int32_t* const* table_ptrs, int cp, int64_t B, int64_t M, int64_t P,
              int page, int block, Tables* t) {
    if (M < 1 || P < 0 || P > 0x7fffffff || M > 0x7fffffff || B < 0 || B > 65535 || B * M > 0x7fffffff)
        return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    t->page_log2 = -1;
    for (int k = 0; (1 << k) <= DCP_MLA_PAGE_MAX; ++k)
        if (page == 1 << k) t->page_log2 = k;
    if (log2_of(block) < 0) return DCP_MLA_CACHE8_ERR_BAD_BLOCK;
    if (page < DCP_MLA_PAGE_MIN || t->page_log2 < 0 || page % block != 0) return DCP_MLA_CACHE8_ERR_BAD_PAGE;
    if (M * page > 0x7fffffff) return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    if (cp < 1 || cp > kCpMax) return DCP_MLA_CACHE8_ERR_BAD_CP;
    if (kv_ptrs == nullptr || table_ptrs == nullptr) return DCP_MLA_CACHE8_ERR_NULL_POINTER;
    for (int j = 0; j < cp; ++j) {
        if (kv_ptrs[j] != nullptr && table_ptrs[j] == nullptr && B > 0) return DCP_MLA_CACHE8_ERR_NULL_POINTER;
        if (!aligned(table_ptrs[j], 4)) return DCP_MLA_CACHE8_ERR_MISALIGNED;
        t->of[j] = table_ptrs[j];
    }
    t->M = M;
    t->P = (int)P;
    return 0;
}

}  // namespace

extern "C" const char* dcp_mla_cache8_strerror(int status) {
    switch (status) {
        case DCP_MLA_CACHE8_ERR_NULL_POINTER: return "a required pointer is NULL, or every shard's";
        case DCP_MLA_CACHE8_ERR_BAD_SHAPE: return "a size is out of range";
        case DCP_MLA_CACHE8_ERR_BAD_BLOCK: return "block must be a power of two in [1, 128]";
        case DCP_MLA_CACHE8_ERR_BAD_CP:
            return "cp must be in [1, 16] and interleave in [1, 2^24], and two shards must not share what is written";
        case DCP_MLA_CACHE8_ERR_MISALIGNED: return "a pointer or a stride is not aligned as the call asks";
        case DCP_MLA_CACHE8_ERR_BAD_DTYPE: return "a dtype that the call does not take";
        case DCP_MLA_CACHE8_ERR_BAD_FLAGS: return "unknown flag bits";
        case DCP_MLA_CACHE8_ERR_WORKSPACE:
            return "the workspace is NULL, not 256-byte aligned, or smaller than the call's workspace_bytes";
        case DCP_MLA_CACHE8_ERR_BAD_WINDOW: return "window and sinks must not be negative, and sinks need a window";
        case DCP_MLA_CACHE8_ERR_TENSOR_MAP: return "a TMA tensor map of a cache could not be encoded";
        case DCP_MLA_CACHE8_ERR_BAD_PAGE: return "page must be a power of two in [32, 4096] and a multiple of block";
        case DCP_MLA_CACHE8_ERR_ALIAS:
            return "outputs overlap inputs other than in place, or two pools overlap";
        case DCP_MLA_CACHE8_ERR_CLUSTER:
            return "the device or context cannot hold a cluster of 16 blocks, a multiprocessor each";
        default: return dcp_lse_reduce_strerror(status);
    }
}

extern "C" int dcp_mla_rope(const void* x, int64_t x_row, int64_t x_head, const void* positions, int pos64,
                            const double* inv_freq, int64_t N, int H, int D, int start, int rot, int interleaved,
                            float mscale, int dtype, void* out, int64_t out_row, int64_t out_head, void* stream) {
    if (N < 0 || N > 0x7fffffff || H < 1 || H > 65535 || D < 1 || D > 65536 || rot < 2 || rot > 256 || rot % 2 != 0 ||
        start < 0 || start > D - rot)
        return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    if (dtype != DCP_DTYPE_BF16 && dtype != DCP_DTYPE_F16 && dtype != DCP_DTYPE_F32)
        return DCP_MLA_CACHE8_ERR_BAD_DTYPE;
    if (N == 0) return 0;
    if (x == nullptr || out == nullptr || positions == nullptr || inv_freq == nullptr)
        return DCP_MLA_CACHE8_ERR_NULL_POINTER;
    const int64_t esize = dtype == DCP_DTYPE_F32 ? 4 : 2;
    if (!aligned(x, esize) || !aligned(out, esize) || !aligned(positions, pos64 ? 8 : 4) || !aligned(inv_freq, 8))
        return DCP_MLA_CACHE8_ERR_MISALIGNED;
    if (x == out && (x_row != out_row || x_head != out_head)) return DCP_MLA_CACHE8_ERR_BAD_SHAPE;
    RopeParams p = {};
    p.x = x;
    p.out = out;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.x_row = x_row;
    p.x_head = x_head;
    p.out_row = out_row;
    p.out_head = out_head;
    p.N = N;
    p.H = H;
    p.start = start;
    p.half = rot / 2;
    p.interleaved = interleaved != 0;
    p.pos64 = pos64 != 0;
    p.copy = x != out && D > rot;
    p.mscale = mscale;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dtype == DCP_DTYPE_BF16) return launch_rope<Bf16>(p, D, esize, st);
    if (dtype == DCP_DTYPE_F16) return launch_rope<F16>(p, D, esize, st);
    return launch_rope<F32>(p, D, esize, st);
}

extern "C" int dcp_mla_cache8_append(const void* latent, int64_t latent_row, const void* k_rope, int64_t rope_row,
                                     int dtype, int64_t N, int64_t B, int Dk, const int32_t* cu_new,
                                     const int32_t* seq_lens, void* const* kv_ptrs, float* const* scale_ptrs, int cp,
                                     int64_t T, int block, int interleave, const double* inv_freq, int interleaved,
                                     float mscale, void* stream) {
    AppendParams p = {};
    bool nothing;
    const int rc = append_params(latent, latent_row, k_rope, rope_row, dtype, N, B, Dk, cu_new, seq_lens, kv_ptrs,
                                 scale_ptrs, cp, T, block, interleave, inv_freq, interleaved, mscale, T == 0, &p,
                                 &nothing);
    return rc != 0 || nothing ? rc : run_append(p, dtype, block, static_cast<cudaStream_t>(stream));
}

extern "C" int dcp_mla_cache8_append_paged(const void* latent, int64_t latent_row, const void* k_rope,
                                           int64_t rope_row, int dtype, int64_t N, int64_t B, int Dk,
                                           const int32_t* cu_new, const int32_t* seq_lens, void* const* kv_ptrs,
                                           float* const* scale_ptrs, const int32_t* const* table_ptrs, int cp,
                                           int64_t P, int page, int64_t M, int block, int interleave,
                                           const double* inv_freq, int interleaved, float mscale, void* stream) {
    PagedAppendParams p = {};
    bool nothing;
    int rc = tables_of(kv_ptrs, table_ptrs, cp, B, M, P, page, block, &p.tables);
    if (rc == 0)
        rc = append_params(latent, latent_row, k_rope, rope_row, dtype, N, B, Dk, cu_new, seq_lens, kv_ptrs,
                           scale_ptrs, cp, M * page, block, interleave, inv_freq, interleaved, mscale, P == 0, &p,
                           &nothing);
    return rc != 0 || nothing ? rc : run_append(p, dtype, block, static_cast<cudaStream_t>(stream));
}

extern "C" int dcp_mla_cache8_read(const void* const* kv_ptrs, const float* const* scale_ptrs, int cp, int64_t B,
                                   int64_t T, int Dk, int block, int interleave, const int32_t* starts,
                                   const int32_t* cu, int64_t N, void* out, int64_t out_row, int dtype,
                                   void* stream) {
    ReadParams p = {};
    bool nothing;
    const int rc = read_params(kv_ptrs, scale_ptrs, cp, B, T, Dk, block, interleave, starts, cu, N, out, out_row,
                               dtype, T == 0, &p, &nothing);
    return rc != 0 || nothing ? rc : run_read(p, dtype, Dk, static_cast<cudaStream_t>(stream));
}

extern "C" int dcp_mla_cache8_read_paged(const void* const* kv_ptrs, const float* const* scale_ptrs,
                                         const int32_t* const* table_ptrs, int cp, int64_t B, int64_t P, int page,
                                         int64_t M, int Dk, int block, int interleave, const int32_t* starts,
                                         const int32_t* cu, int64_t N, void* out, int64_t out_row, int dtype,
                                         void* stream) {
    PagedReadParams p = {};
    bool nothing;
    int rc = tables_of(kv_ptrs, table_ptrs, cp, B, M, P, page, block, &p.tables);
    if (rc == 0)
        rc = read_params(kv_ptrs, scale_ptrs, cp, B, M * page, Dk, block, interleave, starts, cu, N, out, out_row,
                         dtype, P == 0, &p, &nothing);
    return rc != 0 || nothing ? rc : run_read(p, dtype, Dk, static_cast<cudaStream_t>(stream));
}
