// kv4.cu -- a paged key/value cache held in 4 bits, and alpha-entmax attention of the
// newest tokens against it (layout and visibility: kv4_index.h).
//
//   kv4_write_kernel    new keys and values quantised as they are written;
//   kv4_read_kernel     a stretch of every sequence as values again;
//   kv4_scores_kernel   x = (alpha-1) q.k / sqrt(d) of a run of keys against the rows of one
//                       key head, and the keys with x > (the maximum so far) - 1;
//   kv4_solve_kernel    per query row: tau over all runs' keys, then O = sum p_j v_j over the
//                       support alone.
// tau >= m - 1 (m the row maximum) and the maximum over some keys is at most m, so a key at or
// below such a maximum - 1 has p = 0: the scores never leave the chip but for the few that
// can weigh, and value rows without a weight are never read.
//
// 16 sequences of 16k to 32k tokens, 32 query and 8 key heads of 128 (B200): 99 us a call for
// 253 MB of keys and weighed values, 39 at the copy rate; the scores kernel takes 78 of them,
// bound by its instructions (half of the issue slots at four warps a scheduler; matrix pipe
// 22 %, 3.2 TB/s), the solver the rest after it.
#include "kernels.h"
#include "tc_common.cuh"

#include <cuda_fp16.h>

namespace ent {

namespace {

constexpr int kKvThreads = 256;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// the larger, or NaN where either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ Kv4Seq seq_of(const Kv4Args& a, int b) {
    return kv4_seq(a.g, a.start[b], a.new_lens ? a.new_lens[b] : a.g.L);
}

// 8 consecutive values of a row
__device__ __forceinline__ void load8(const float* p, float* x) {
    const float4 u = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + 4);
    x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w; x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[2 * i] = bf16_lo(w[i]); x[2 * i + 1] = bf16_hi(w[i]); }
}
__device__ __forceinline__ void store8(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// What the copying kernels share: blockIdx.y is the sequence and head, z 0 for keys, 1 for
// values; a CTA takes kCopyRows * (256 / (D/8)) consecutive rows of the L, a thread the same
// 8-value part of kCopyRows of them, so that their loads are in flight together (one row a
// thread keeps 20 KB of reads in flight on an SM, a third of what the memory's latency asks).
constexpr int kCopyRows = 4;
template <int D>
struct RowParts {
    static constexpr int kParts = D / 8, kStep = kKvThreads / kParts, kRows = kCopyRows * kStep;
    int b, h, l0, grp, c;   // sequence, head, first row; the part's group of 32 dimensions and quarter
    int page[kCopyRows];    // of each row; -1: the row is padding, -2: its page is not in the pool
    Kv4Seq s;
    size_t at0;             // element offset of the part of row l0 in [B][Hkv][L][D]
    __device__ __forceinline__ explicit RowParts(const Kv4Args& a) {
        const int bh = blockIdx.y, t = threadIdx.x % kParts;
        b = bh / a.Hkv;
        h = bh - b * a.Hkv;
        l0 = blockIdx.x * kRows + threadIdx.x / kParts;
        grp = t >> 2;
        c = t & 3;
        at0 = ((size_t)bh * a.g.L + l0) * D + t * 8;
        s = seq_of(a, b);
        if (s.bad && a.bad && l0 == 0 && t == 0) atomicOr(a.bad, s.bad);
        const int* table = a.table + (size_t)b * a.g.max_pages;
#pragma unroll
        for (int u = 0; u < kCopyRows; ++u) {
            page[u] = -1;
            if (l(u) < s.rows) {
                page[u] = kv4_page(a.g, table, s.start + l(u));
                if (page[u] < 0) {
                    page[u] = -2;
                    if (a.bad && t == 0) atomicOr(a.bad, kKvBadPage);
                }
            }
        }
    }
    __device__ __forceinline__ int l(int u) const { return l0 + u * kStep; }
    __device__ __forceinline__ size_t at(int u) const { return at0 + (size_t)u * kStep * D; }
};

// ------------------------------------------------------------------ write
// Four threads per group of 32 dimensions, 8 each.
//     zero = bf16(min),  scale = bf16((max - zero) / 15),  code = rint((x - zero) / scale)
// as they are in 64-bit arithmetic, so that the codes do not depend on who computes them.
// Float gets there but for values next to a border: its scale is within 2^-21 of the exact
// one, so only a quotient that near to the middle of two bf16 numbers can round otherwise;
// and its quotient of an element is off by at most 4e-6 (2^-22 of at most 15.1).  Where the
// scale lies within 8 float steps (2^-20) of a middle it is computed in double.  An element
// within 1e-4 of a half-integer h -- exact ties are common, 0.2 % of bf16 elements -- is
// decided by the sign of (x - z) - scale h: the difference is carried exactly as t + e (the
// error-free sum), scale h has 13 bits, and t - scale h is exact that near to zero.
// A group with a NaN, an infinity, or a minimum that rounds to one is stored as (0, NaN):
// it reads back as NaN.
// 4 x 4096 rows of 8 heads of 128 (bf16, three quarters real): 42 us, 1.6 TB/s; bound by its
// instructions, since two warps of five hold an exact tie.
template <typename T, int D>
__global__ void __launch_bounds__(kKvThreads) kv4_write_kernel(const Kv4Args a) {
    constexpr int G = D / kKvGroup;
    const RowParts<D> p(a);
    const unsigned quad = 0xfu << (threadIdx.x & 28);   // (rows are whole quads)
    const T* src = static_cast<const T*>(blockIdx.z ? a.v : a.k);
    float xs[kCopyRows][8];
#pragma unroll
    for (int u = 0; u < kCopyRows; ++u)
        if (p.l(u) < p.s.rows) load8(src + p.at(u), xs[u]);
#pragma unroll
    for (int u = 0; u < kCopyRows; ++u) {
    if (p.page[u] < 0) continue;
    const float (&x)[8] = xs[u];
    // (a NaN passes through max_nan; lo is only used where hi, and so every value, is fine)
    float lo = x[0], hi = x[0], big = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        big = max_nan(big, fabsf(x[i]));
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(quad, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(quad, hi, o));
        big = max_nan(big, __shfl_xor_sync(quad, big, o));
    }
    const __nv_bfloat16 zb = __float2bfloat16_rn(lo);
    const float z = __bfloat162float(zb);
    const bool fine = big < INFINITY && fabsf(z) < INFINITY;
    float sq = (hi - z) * (1.f / 15.f);
    const int low = (int)(__float_as_uint(sq) & 0xffffu) - 0x8000;
    if (!(sq > 1e-30f && sq < 1e30f) || (low > -8 && low < 8)) {
        const double range = (double)hi - (double)z;
        sq = range > 0. ? (float)(range / 15.) : 0.f;
    }
    const __nv_bfloat16 sb = __float2bfloat16_rn(fine ? sq : 0.f);
    const float sc = __bfloat162float(sb);
    uint32_t w = 0;
    if (sc > 0.f) {
        const float inv = 1.f / sc;
        constexpr float kRound = 12582912.f;   // 1.5 * 2^23: adding it rounds to an integer
        float near = 0.f;                      // largest distance from the integer taken
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = fminf(fmaxf((x[i] - z) * inv, 0.f), 15.f);
            const float y = q + kRound;
            near = max_nan(near, fabsf(q - (y - kRound)));
            w += (__float_as_uint(y) & 15u) << (4 * i);
        }
        if (!(inv >= 1e-30f && inv <= 1e30f)) {
            w = 0;
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                float xi = x[0];
#pragma unroll
                for (int k = 1; k < 8; ++k) xi = k == i ? x[k] : xi;
                const double q = rint(((double)xi - (double)z) / (double)sc);
                w |= (uint32_t)(int)fmin(fmax(q, 0.), 15.) << (4 * i);
            }
        } else if (near >= 0.4999f) {
            w = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float t = x[i] - z, bb = t - x[i], e = (x[i] - (t - bb)) - (z + bb);
                const float q = fminf(fmaxf(t * inv, 0.f), 15.f);
                const float n = truncf(q), h = n + 0.5f;
                uint32_t code = (uint32_t)(int)rintf(q);
                if (fabsf(q - h) < 2e-4f) {
                    const float d = (t - sc * h) + e;
                    const uint32_t down = (uint32_t)(int)n;
                    code = d > 0.f ? down + 1 : d < 0.f ? down : down + (down & 1u);
                }
                w |= code << (4 * i);
            }
        }
    }
    const size_t at = kv4_row(a.g, a.Hkv, p.page[u], p.h, p.s.start + p.l(u));
    reinterpret_cast<uint32_t*>(blockIdx.z ? a.v_codes : a.k_codes)[at * (D / 8) + p.c * G + p.grp] = w;
    if (p.c == 0) {
        const uint32_t zw = fine ? (uint32_t)__bfloat16_as_ushort(zb) : 0x7fffu;
        reinterpret_cast<uint32_t*>(blockIdx.z ? a.v_meta : a.k_meta)[at * G + p.grp] =
            (uint32_t)__bfloat16_as_ushort(sb) | zw << 16;
    }
    }   // rows
}

// ------------------------------------------------------------------ read
// A thread per word of codes: 8 values zero + scale * code (one fused multiply-add each:
// exact but for the last rounding).  A nibble under the bits of 2^23 is the float 2^23 +
// 16^i code: the first five need no shift, and the scale carries the 16^-i.
// Rows past new_lens, and rows of a page outside the pool, are zeros.
// 8 x 8192 rows of 8 heads of 128 to bf16: 68 us, 3.9 TB/s; the loads wait for the page table.
template <typename T, int D>
__global__ void __launch_bounds__(kKvThreads) kv4_read_kernel(const Kv4Args a) {
    constexpr int G = D / kKvGroup;
    const RowParts<D> p(a);
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(blockIdx.z ? a.v_codes : a.k_codes);
    const uint32_t* meta = reinterpret_cast<const uint32_t*>(blockIdx.z ? a.v_meta : a.k_meta);
    T* dst = static_cast<T*>(blockIdx.z ? a.v_out : a.k_out);
    uint32_t w[kCopyRows], m[kCopyRows];
#pragma unroll
    for (int u = 0; u < kCopyRows; ++u) {
        w[u] = m[u] = 0u;   // zeros
        if (p.page[u] >= 0) {
            const size_t at = kv4_row(a.g, a.Hkv, p.page[u], p.h, p.s.start + p.l(u));
            w[u] = __ldg(codes + at * (D / 8) + p.c * G + p.grp);
            m[u] = __ldg(meta + at * G + p.grp);
        }
    }
#pragma unroll
    for (int u = 0; u < kCopyRows; ++u) {
        if (p.l(u) >= a.g.L) break;
        const float sc = bf16_lo(m[u]), z = bf16_hi(m[u]);
        float x[8];
        // (a scale below 2^-106 would lose bits to the 16^-4: it takes the codes themselves)
        if (sc > 1e-31f) {
            float f = sc;
#pragma unroll
            for (int i = 0; i < 5; ++i) {
                x[i] = fmaf(f, __uint_as_float((w[u] & (15u << (4 * i))) | 0x4b000000u) - 8388608.f, z);
                f *= 0.0625f;
            }
            f = sc;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                x[5 + i] = fmaf(f, __uint_as_float((w[u] >> 20 & (15u << (4 * i))) | 0x4b000000u) - 8388608.f, z);
                f *= 0.0625f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf(sc, (float)((w[u] >> (4 * i)) & 15u), z);
        }
        store8(dst + p.at(u), x);
    }
}

// ------------------------------------------------------------------ scores
// A warp per (run of chunks of C keys, block of R rows, sequence and key head); the four warps
// of a CTA share nothing but the rows' maxima so far.  The rows are the new tokens' queries of all heads that share the
// key head, row = l * group + head of the group.  Keys are the M = 16 rows of an m16n8k16
// product and the queries its 8 columns; the contraction index is permuted so that a lane's
// four A registers are its own words of two keys, masked: a nibble at bits 0-3 of a half is
// code * 2^-24 (a subnormal, which the product takes exactly), one at bits 4-7 is 16 times
// that, and the queries' other operand carries the 1/16.  So 8 codes cost four ANDs and a
// shift, and the product is exact in the codes.  The pair (scale, zero) of each group comes
// in afterwards:
//     q.k = sum_groups scale * (codes . q) + zero * sum q,
// the second sum as a product too: a lane's pair of group c is two elements of an A operand,
// met by (0, sum q of group c) in three bf16 parts (24 bits).
// The queries are fp16, scaled per row by a power of two so that the largest lies in
// [2^14, 2^15): exact for bf16 values down to 2^-27 of the largest (2^-31 in the dimensions
// without the 1/16), below which the rounding is 2^-35 (2^-39) of it.  The products' sums lose
// what lies under 2^-24 of their largest term, and the pair's terms largely cancel (codes lie
// about 8, zero about -8 scale): bf16 results do not see it, float32 ones would.
// A float32 row is hi + mid: hi a multiple of 16, so that every partial sum of codes . hi is a
// multiple of 16 below 2^24 and the product exact, mid the rest rounded to fp16 (2^-23 of the
// row's largest value at most).  The sums begin at -8 sum hi, which centres the codes, and are
// joined in float:
//     q.k = sum_groups scale * (((codes - 8) . hi) + codes . mid) + (zero + 8 scale) sum hi + zero sum mid.
// O then lies 0.3e-6 to 0.6e-6 from the 64-bit result, where plain float products of the same keys
// leave 0.4e-6 to 1.6e-6; with one chain of truncated sums, queries of two times 11 bits and the
// zeros' term as a product it was 1.2e-6 to 2.9e-6, and calls were 2 to 7 % shorter (16 x 8192 of
// 32 heads of 128: 50 us instead of 51; eight rows of 4 x 8192: 79 instead of 85).
// The scores of a chunk pass through the warp's shared memory (queries by keys), where 32/R
// lanes a row take their maximum and the candidates above the CTA's maximum so far - 1 (which
// of the warps got how far does not matter: the solver drops what the final maximum rules out).
// c = A B (+ c); the first form takes no accumulator, so that none has to be cleared
__device__ __forceinline__ void mma_16816_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_16816_bf_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_1688_bf(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(b0));
}

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// x rounded to bf16, in the upper half of a word; what is left stays in x
__device__ __forceinline__ uint32_t bf16_part(float& x) {
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    x -= __bfloat162float(h);
    return (uint32_t)__bfloat16_as_ushort(h) << 16;
}

// G consecutive 4-byte words of shared memory (one load)
template <int G>
__device__ __forceinline__ void load_words(const char* p, uint32_t (&w)[G]) {
    if constexpr (G == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (G == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// `bytes` (a multiple of 16, as both addresses) from this GPU's memory into shared memory,
// counted at `bar`; first to leave the L2 cache: the keys pass through once, and the candidates
// that the solver reads next are to stay.
__device__ __forceinline__ uint64_t evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}
__device__ __forceinline__ void bulk_copy(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            tc::smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(tc::smem_u32(bar)), "l"(policy)
        : "memory");
}

// Waits for a phase, 2 s at most.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity) {
    if (tc::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = tc::globaltimer_ns();
    while (!tc::mbar_try_wait(bar, parity))
        if (tc::globaltimer_ns() - t0 > tc::kWaitLimitNs) return false;
    return true;
}

constexpr int kScoreWarps = 4;
constexpr int kScoreThreads = kScoreWarps * 32;
constexpr int kStages = 2;   // chunks of a warp in shared memory: one on its way while one is worked on

template <int D, int R>
struct ScoreSmem {   // of one warp
    static constexpr int C = kv4_chunk_keys(R), kCodes = C * (D / 2), kMeta = C * (D / kKvGroup) * 4;
    static constexpr int kStage = kCodes + kMeta;
    static constexpr int kStride = C + 4;   // floats a row of scores: spreads a product's 8 keys x 4 row pairs over the banks
    static constexpr int kBytes = kStages * kStage + (R <= 8 ? 8 : R) * kStride * 4;
};

// R: rows of a block (4, 8, 16 or 32), in NT products of 8 columns.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kScoreThreads, R == 4 ? 4 : R == 8 ? 3 : 2) kv4_scores_kernel(const Kv4Args a) {
    constexpr int G = D / kKvGroup, NT = R <= 8 ? 1 : R / 8, C = kv4_chunk_keys(R), U = C / kKvTile;
    constexpr int LPR = 32 / R, KPL = C / LPR;   // lanes a row, keys a lane
    using L = ScoreSmem<D, R>;
    constexpr int kStride = L::kStride;
    constexpr bool F32 = sizeof(T) == 4;
    extern __shared__ __align__(128) char score_smem[];
    __shared__ uint64_t bars_all[kScoreWarps][kStages];
    // With four rows the product's 8 columns hold two groups of dimensions, h and h + G/2, each
    // MMA half of its contraction over either: columns 0-3 are the rows with the first group,
    // 4-7 with the second.  As many products, but half the scale multiplications.
    constexpr bool PAIR = R == 4 && G >= 2;
    constexpr int GS = PAIR ? G / 2 : G;         // groups that a lane scales
    __shared__ float row_max[R];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    char* ring = score_smem + warp * L::kBytes;                       // [kStages][codes, meta]
    float* xs = reinterpret_cast<float*>(ring + kStages * L::kStage);
    uint64_t* bars = bars_all[warp];
    const int bk = blockIdx.z, b = bk / a.Hkv, hk = bk - b * a.Hkv;
    const Kv4Seq s = seq_of(a, b);
    if (s.bad && a.bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.bad, s.bad);
    const int row0 = blockIdx.y * R, nrows = s.rows * a.group;   // real rows of this key head
    const int nch = kv4_seq_chunks(a.g, s, C), run = kv4_run(nch, a.nrun);
    const int slot = blockIdx.x * kScoreWarps + warp;
    const int ch0 = slot * run, ch1 = kv4_min(ch0 + run, nch);
    if (threadIdx.x < R) row_max[threadIdx.x] = -INFINITY;
    __syncthreads();
    if (row0 >= nrows || ch0 >= ch1) return;   // (the solver takes no more runs than hold a chunk)

    const int c = lane & 3, key = lane >> 2;   // the lane's keys of a tile: key and key + 8
    const int lrow = lane / LPR, sub = lane % LPR;   // the row that it looks through, and its part of it
    constexpr int kTokenB = D / 2, kMetaB = 4 * G;   // bytes of a token
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) tc::mbar_init(&bars[i], 1);
        tc::fence_barrier_init();
        tc::fence_proxy_async_smem();
    }
    __syncwarp();

    const int* table = a.table + (size_t)b * a.g.max_pages;
    const Kv4Chunks chunks(a.g, s, C);
    // page of tile `lane` of a chunk (lanes below U)
    auto page_of = [&](int ch) {
        int p = -1;
        if (ch < ch1 && lane < U) {
            const int kb = chunks.first(ch) + lane * kKvTile;
            if (kb < chunks.end(ch)) {
                p = kv4_page(a.g, table, kb);
                if (p < 0 && a.bad) atomicOr(a.bad, kKvBadPage);
            }
        }
        return p;
    };
    // Starts the copies of a chunk into its stage, a tile a lane; what is not there is not
    // copied, and no row sees it.  `has`: four bits a stage, the tiles that are there.
    unsigned has = 0;
    const uint64_t policy = evict_first();
    int next_stage = 0, pages = page_of(ch0);
    auto issue = [&](int ch) {
        const unsigned there = __ballot_sync(kFull, pages >= 0);
        uint64_t* bar = &bars[next_stage];
        if (lane == 0) tc::mbar_arrive_expect_tx(bar, __popc(there) * (kKvTile * (kTokenB + kMetaB)));
        __syncwarp();
        if (pages >= 0) {
            char* dst = ring + next_stage * L::kStage;
            const size_t row = kv4_row(a.g, a.Hkv, pages, hk, chunks.first(ch) + lane * kKvTile);
            bulk_copy(dst + lane * kKvTile * kTokenB, reinterpret_cast<const char*>(a.k_codes) + row * kTokenB,
                      kKvTile * kTokenB, bar, policy);
            bulk_copy(dst + L::kCodes + lane * kKvTile * kMetaB, reinterpret_cast<const char*>(a.k_meta) + row * kMetaB,
                      kKvTile * kMetaB, bar, policy);
        }
        has = (has & ~(15u << (4 * next_stage))) | there << (4 * next_stage);
        next_stage = next_stage + 1 == kStages ? 0 : next_stage + 1;
        pages = page_of(ch + 1);
    };
    for (int i = 0; i < kStages - 1 && ch0 + i < ch1; ++i) issue(ch0 + i);

    // ---- queries: lane (n = lane / 4, c = lane % 4) holds dimensions 32 w + 8 c + i of row n
    // (PAIR: row n % 4, and of its two groups the one that columns 0-3 or 4-7 take)
    constexpr int QG = PAIR ? GS : G;
    uint32_t qf[NT][QG][4], ql[F32 ? NT : 1][QG][4];   // B operands; float32 rows: hi and mid
    uint32_t qz[F32 ? 1 : NT][3];                    // sum q of group c in three parts
    float sh[F32 ? NT : 1][QG][2], sm[F32 ? NT : 1][QG][2];   // float32: sum hi, sum mid of columns 2c, 2c + 1
    uint32_t qb[PAIR ? QG : 1][4][2], qbl[PAIR && F32 ? QG : 1][4][2];   // PAIR: the two halves of the operand
    float mul = 0.f, mul2 = 1.f;                     // of row lrow: x = mul mul2 acc
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int col = PAIR ? key & 3 : key, r = row0 + nt * 8 + col;
        const bool real = r < nrows && nt * 8 + col < R;
        const int l = real ? r / a.group : 0, gi = real ? r - l * a.group : 0;
        const T* q = static_cast<const T*>(a.q) + (((size_t)b * a.Hkv * a.group + hk * a.group + gi) * a.g.L + l) * D;
        float x[G][8];
        float top = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            if (real) load8(q + 32 * g + 8 * c, x[g]);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (!real) x[g][k] = 0.f;
                top = max_nan(top, fabsf(x[g][k]));
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) top = max_nan(top, __shfl_xor_sync(kFull, top, o));
        const bool fine = top < INFINITY;
        int e = 0;
        // (2^126 at most: a row below 2^-111 is held to 2^-150)
        if (top > 0.f && fine) { frexpf(top, &e); e = min(15 - e, 126); }
        const float fe = __int_as_float((e + 127) << 23);
        float zsum = 0.f;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x[g][k] *= fe;
                sum += x[g][k];
            }
            sum += __shfl_xor_sync(kFull, sum, 1);
            sum += __shfl_xor_sync(kFull, sum, 2);
            if (PAIR && G == 2 ? 2 * g == c : g == c) zsum = sum * 5.9604644775390625e-08f;   // 2^-24, the codes' unit
        }
        if (PAIR && key >= 4) zsum = 0.f;   // (the zero terms go to columns 0-3)
#pragma unroll
        for (int g = 0; g < QG; ++g) {
            float y[8], lo[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = PAIR && key >= 4 ? x[(g + GS) % G][k] : x[g][k];
            if constexpr (F32) {
                float hs = 0.f, ms = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float hi = rintf(y[k] * 0.0625f) * 16.f;
                    lo[k] = y[k] - hi;
                    y[k] = hi;
                    hs += hi;
                    ms += lo[k];
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    hs += __shfl_xor_sync(kFull, hs, o);
                    ms += __shfl_xor_sync(kFull, ms, o);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    sh[nt][g][k] = __shfl_sync(kFull, hs, 4 * (2 * c + k)) * 5.9604644775390625e-08f;
                    sm[nt][g][k] = __shfl_sync(kFull, ms, 4 * (2 * c + k)) * 5.9604644775390625e-08f;
                }
            }
            const float f = 0.0625f;
            qf[nt][g][0] = pack_half(y[0], y[4]);
            qf[nt][g][1] = pack_half(y[1] * f, y[5] * f);
            qf[nt][g][2] = pack_half(y[2], y[6]);
            qf[nt][g][3] = pack_half(y[3] * f, y[7] * f);
            if constexpr (F32) {
                ql[nt][g][0] = pack_half(lo[0], lo[4]);
                ql[nt][g][1] = pack_half(lo[1] * f, lo[5] * f);
                ql[nt][g][2] = pack_half(lo[2], lo[6]);
                ql[nt][g][3] = pack_half(lo[3] * f, lo[7] * f);
            }
        }
        if constexpr (!F32) {
#pragma unroll
            for (int t = 0; t < 3; ++t) qz[nt][t] = bf16_part(zsum);
        }
        // x = cx 2^(24 - e) s, in two factors where one would overflow (24 - e <= 137);
        // a row with a NaN or an infinity has NaN scores
        const int e1 = min(24 - e, 100);
        const float f1 = fine ? a.cx * __int_as_float((e1 + 127) << 23) : nanf("");
        const float f2 = __int_as_float((24 - e - e1 + 127) << 23);
        const float g1 = __shfl_sync(kFull, f1, 4 * (lrow & 7)), g2 = __shfl_sync(kFull, f2, 4 * (lrow & 7));
        if (lrow >> 3 == nt) { mul = g1; mul2 = g2; }
    }
    if constexpr (PAIR) {
#pragma unroll
        for (int g = 0; g < QG; ++g)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                qb[g][t][0] = key < 4 ? qf[0][g][t] : 0u;
                qb[g][t][1] = key < 4 ? 0u : qf[0][g][t];
                if constexpr (F32) {
                    qbl[g][t][0] = key < 4 ? ql[0][g][t] : 0u;
                    qbl[g][t][1] = key < 4 ? 0u : ql[0][g][t];
                }
            }
    }

    const bool lreal = row0 + lrow < nrows;
    const int lpos = lreal ? s.start + (row0 + lrow) / a.group : -1;
    const size_t grow = ((size_t)b * a.Hkv + hk) * a.g.L * a.group + row0 + lrow;   // the lane's row
    int2* out = a.cand + (grow * a.nchunk + ch0) * C;
    const int pos_first = s.start + row0 / a.group;
    const int pos_last = s.start + (kv4_min(row0 + R, nrows) - 1) / a.group;
    float m = -INFINITY;    // of the row, over the run so far (and what other warps told)
    int n = 0;              // candidates of the row so far

    // ---- keys, a chunk of U tiles at a time
    const char* lane_codes = ring + key * kTokenB + c * 4 * G;
    const char* lane_meta = ring + L::kCodes + key * kMetaB + (PAIR ? (c >> 1) * 4 * GS : 0);
    int stage = 0, phase = 0;
    bool ok = true;
#pragma unroll 1
    for (int ch = ch0; ch < ch1; ++ch) {
        // (the stage of the chunk before this one, which every lane has read)
        if (ch + kStages - 1 < ch1) issue(ch + kStages - 1);
        const int k0 = chunks.first(ch), k1 = chunks.end(ch);
        const unsigned there = has >> (4 * stage) & 15u;
        ok = wait_phase(&bars[stage], phase);
        if (!__all_sync(kFull, ok)) { ok = false; break; }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            uint32_t w[2][G], mt[2][GS];   // codes, and the pairs of the groups that the lane scales
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                load_words<G>(lane_codes + stage * L::kStage + (u * kKvTile + 8 * h) * kTokenB, w[h]);
                load_words<GS>(lane_meta + stage * L::kStage + (u * kKvTile + 8 * h) * kMetaB, mt[h]);
            }
            float acc[NT][4];
            if constexpr (F32) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
            } else {
                uint32_t mz[2];   // the pair of group c (PAIR with two groups: of group c/2; else zeros)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if constexpr (PAIR && G == 4) mz[h] = c & 1 ? mt[h][GS - 1] : mt[h][0];
                    else if constexpr (PAIR) mz[h] = c & 1 ? 0u : mt[h][0];
                    else {
                        mz[h] = c == 0 ? mt[h][0] : 0u;
#pragma unroll
                        for (int g = 1; g < G; ++g) mz[h] = c == g ? mt[h][g] : mz[h];
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    mma_16816_bf_0(acc[nt], mz[0], mz[1], mz[0], mz[1], qz[nt][0], qz[nt][1]);
                    mma_1688_bf(acc[nt], mz[0], mz[1], qz[nt][2]);
                }
            }
            // a word's codes as four pairs of halves
            auto halves = [](uint32_t x, uint32_t (&h)[4]) {
                h[0] = x & 0x000f000fu;
                h[1] = x & 0x00f000f0u;
                x >>= 8;
                h[2] = x & 0x000f000fu;
                h[3] = x & 0x00f000f0u;
            };
#pragma unroll
            for (int g = 0; g < GS; ++g) {
                const float sc[2] = {bf16_lo(mt[0][g]), bf16_lo(mt[1][g])};
                uint32_t k0h[4], k1h[4];
                halves(w[0][g], k0h);
                halves(w[1][g], k1h);
                // float32: acc of keys h, columns k from its two sums
                auto join = [&](float (&r)[4], int nt, const float (&dh)[4], const float (&dm)[4]) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float z = bf16_hi(mt[h][g]), zc = fmaf(8.f, sc[h], z);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float t = fmaf(z, sm[nt][g][k], r[2 * h + k]);
                            t = fmaf(zc, sh[nt][g][k], t);
                            r[2 * h + k] = fmaf(sc[h], dh[2 * h + k] + dm[2 * h + k], t);
                        }
                    }
                };
                if constexpr (PAIR) {
                    uint32_t o0[4], o1[4];   // the second group's
                    halves(w[0][g + GS], o0);
                    halves(w[1][g + GS], o1);
                    float d[4];
                    if constexpr (F32) {
                        float dm[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) d[k] = -8.f * sh[0][g][k & 1];
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            mma_16816(d, k0h[t], k1h[t], o0[t], o1[t], qb[g][t][0], qb[g][t][1]);
                            if (t == 0) mma_16816_0(dm, k0h[t], k1h[t], o0[t], o1[t], qbl[g][t][0], qbl[g][t][1]);
                            else mma_16816(dm, k0h[t], k1h[t], o0[t], o1[t], qbl[g][t][0], qbl[g][t][1]);
                        }
                        join(acc[0], 0, d, dm);
                    } else {
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            if (t == 0) mma_16816_0(d, k0h[t], k1h[t], o0[t], o1[t], qb[g][t][0], qb[g][t][1]);
                            else mma_16816(d, k0h[t], k1h[t], o0[t], o1[t], qb[g][t][0], qb[g][t][1]);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[0][k] = fmaf(sc[k >> 1], d[k], acc[0][k]);
                    }
                } else {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float d[4];
                        if constexpr (F32) {
                            float dm[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) d[k] = -8.f * sh[nt][g][k & 1];
                            mma_16816(d, k0h[0], k1h[0], k0h[1], k1h[1], qf[nt][g][0], qf[nt][g][1]);
                            mma_16816(d, k0h[2], k1h[2], k0h[3], k1h[3], qf[nt][g][2], qf[nt][g][3]);
                            mma_16816_0(dm, k0h[0], k1h[0], k0h[1], k1h[1], ql[nt][g][0], ql[nt][g][1]);
                            mma_16816(dm, k0h[2], k1h[2], k0h[3], k1h[3], ql[nt][g][2], ql[nt][g][3]);
                            join(acc[nt], nt, d, dm);
                        } else {
                            mma_16816_0(d, k0h[0], k1h[0], k0h[1], k1h[1], qf[nt][g][0], qf[nt][g][1]);
                            mma_16816(d, k0h[2], k1h[2], k0h[3], k1h[3], qf[nt][g][2], qf[nt][g][3]);
#pragma unroll
                            for (int k = 0; k < 4; ++k) acc[nt][k] = fmaf(sc[k >> 1], d[k], acc[nt][k]);
                        }
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        xs[(nt * 8 + 2 * c + k) * kStride + u * kKvTile + key + 8 * h] = acc[nt][2 * h + k];
        }
        __syncwarp();
        // not every row sees every key of the chunk: those it does not see leave as -inf
        const bool whole = there == (1u << U) - 1u && k1 - k0 == C && k1 - 1 <= pos_first &&
                           (!a.g.window || k1 <= a.g.sinks || k0 > pos_last - a.g.window);
        // ---- the row's part of the chunk: keys (i * LPR + sub) * 4 + e
        float v[KPL];
#pragma unroll
        for (int k = 0; k < KPL / 4; ++k) {
            float4 f = *reinterpret_cast<const float4*>(xs + lrow * kStride + (k * LPR + sub) * 4);
            if constexpr (PAIR) {   // the second groups' share
                const float4 h = *reinterpret_cast<const float4*>(xs + (lrow + 4) * kStride + (k * LPR + sub) * 4);
                f = make_float4(f.x + h.x, f.y + h.y, f.z + h.z, f.w + h.w);
            }
            v[4 * k] = f.x * mul; v[4 * k + 1] = f.y * mul; v[4 * k + 2] = f.z * mul; v[4 * k + 3] = f.w * mul;
        }
        if (mul2 != 1.f) {
#pragma unroll
            for (int k = 0; k < KPL; ++k) v[k] *= mul2;
        }
        if (!whole) {
#pragma unroll
            for (int k = 0; k < KPL; ++k) {
                const int kk = ((k >> 2) * LPR + sub) * 4 + (k & 3);
                const bool see = k0 + kk < k1 && (there >> (kk / kKvTile) & 1u) && kv4_sees(a.g, lpos, k0 + kk);
                v[k] = see ? v[k] : -INFINITY;
            }
        }
        // a NaN passes through every maximum; +inf is caught at the end.  (A store of row_max that
        // loses to another warp's costs a weaker filter, no more.)
        m = max_nan(m, *const_cast<volatile float*>(&row_max[lrow]));
#pragma unroll
        for (int k = 0; k < KPL; ++k) m = max_nan(m, v[k]);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, o));
        if (sub == 0) *const_cast<volatile float*>(&row_max[lrow]) = m;
        // above m - 1, and the maximum itself: where |m| >= 2^24 makes them equal, the limit is
        // the next float below m (m = -inf: the step gives NaN; m = NaN: m - 1 is; nothing is above
        // either).  (A higher bound of tau, proved by the run's own keys, halves the candidates of a
        // run of 20 chunks and costs as much as they do.)
        float lim = m - 1.f;
        if (lim >= m) lim = __int_as_float(__float_as_int(m) + (m > 0.f ? -1 : 1));
        unsigned take = 0;
#pragma unroll
        for (int k = 0; k < KPL; ++k) take |= (v[k] > lim ? 1u : 0u) << k;
        if (!lreal) take = 0;
        const int cnt = __popc(take);
        int incl = cnt;
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, o, LPR);
            if (sub >= o) incl += y;
        }
        int put = n + incl - cnt;
        n += __shfl_sync(kFull, incl, LPR - 1, LPR);
        // (few lanes have more than one or two: read again what is taken, rather than hold every
        // value against its bit)
        while (take) {
            const int k = __ffs(take) - 1;
            take &= take - 1u;
            const int kk = ((k >> 2) * LPR + sub) * 4 + (k & 3);
            float x = xs[lrow * kStride + kk];
            if constexpr (PAIR) x += xs[(lrow + 4) * kStride + kk];
            out[put++] = make_int2(__float_as_int(x * mul * mul2), k0 + kk);
        }
        __syncwarp();
        if (++stage == kStages) { stage = 0; phase ^= 1; }
    }
    if (!ok) {
        // a copy that never came: report it, let the others land (2 s each at most), no scores
        if (a.bad && lane == 0) atomicOr(a.bad, kKvBadWait);
        for (int i = 0; i < kStages; ++i) wait_phase(&bars[i], i >= stage ? phase : phase ^ 1);
        m = nanf("");
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (lreal && sub == 0) {
        a.run_max[grow * a.nrun + slot] = m < INFINITY ? m : nanf("");
        a.run_n[grow * a.nrun + slot] = n;
    }
}

// ------------------------------------------------------------------ solve and P.V
// One CTA per query row.  The runs' candidates are gathered in key order into shared memory,
// those above m - 1 (m the maximum over the runs) kept, tau - m is found by Halley-bisection
// from the bracket [-1, -n^(1-alpha)] (n the candidates' count: f <= 0 there since at most n
// keys weigh), and O accumulates over the support, D/8 lanes per value row.  Scores are held
// relative to m, so tau keeps its precision for scores of any size.  Every sum has a fixed
// order: the result does not change from run to run.  A row with more than kCap candidates
// above what is known to lie below tau goes over the runs' lists again in every pass.
constexpr int kSolveThreads = 256;
constexpr int kSolveWarps = kSolveThreads / 32;
constexpr int kCap = 4096;
static_assert((2 * kCap + kKvMaxRuns + 1) * 4 <= 40 * 1024, "beside 5 KB of static shared memory, within 48");
constexpr float kKvFtol = 2e-7f, kKvStol = 6e-8f;   // to the rounding of the sums

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
    return x;
}

// Exclusive prefix over the CTA's warps of one count each; total in *all.  Two barriers.
__device__ __forceinline__ int warps_before(int n, int* box, int* all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) box[warp] = n;
    __syncthreads();
    int before = 0, sum = 0;
#pragma unroll
    for (int w = 0; w < kSolveWarps; ++w) {
        if (w < warp) before += box[w];
        sum += box[w];
    }
    *all = sum;
    return before;
}

template <typename T, int D, int GM>
__global__ void __launch_bounds__(kSolveThreads, 4) kv4_solve_kernel(const Kv4Args a) {
    constexpr int G = D / kKvGroup, LPK = D / 8, KPW = 32 / LPK;
    extern __shared__ int solve_smem[];
    float* ys = reinterpret_cast<float*>(solve_smem);   // [kCap] x - m of the candidates, then their weights
    int* js = solve_smem + kCap;                        // [kCap] their keys
    int* off = js + kCap;               // [nrun + 1] the runs' candidates before each run
    __shared__ float red[3][kSolveWarps];
    __shared__ int box[kSolveWarps], box2[kSolveWarps], found;
    __shared__ float bc[2];
    __shared__ float halves[kSolveWarps][D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = a.g.L * a.group;    // rows of one key head
    const int bk = blockIdx.x / per, r = blockIdx.x - bk * per;
    const int b = bk / a.Hkv, hk = bk - b * a.Hkv;
    const int l = r / a.group, gi = r - l * a.group;
    const Kv4Seq s = seq_of(a, b);
    const size_t orow = ((size_t)b * a.Hkv * a.group + hk * a.group + gi) * a.g.L + l;
    T* o = static_cast<T*>(a.o) + orow * D;
    const size_t at = ((size_t)bk * per + r) * a.nrun;
    const float* cm = a.run_max + at;
    int* cn = a.run_n + at;
    int2* cand = a.cand + ((size_t)bk * per + r) * a.nchunk * a.chunk;
    int nrun = 0, stride = 0;   // the sequence's runs, entries from one's list to the next's
    if (l < s.rows) {
        const int nch = kv4_seq_chunks(a.g, s, a.chunk), run = kv4_run(nch, a.nrun);
        stride = run * a.chunk;   // (a row's part holds at most 2^30 entries)
        nrun = (nch + run - 1) / run;
    }
    auto list_of = [&](int i) { return cand + (size_t)i * stride; };
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // (a call that covers no token has no scores kernel to report its lengths)
    if (a.nchunk == 0 && s.bad && a.bad && hk == 0 && r == 0 && tid == 0) atomicOr(a.bad, s.bad);

    // ---- row maximum (every warp for itself), then the runs' offsets, a share each warp
    float m = -INFINITY;
    bool nan = false;
    for (int i = lane; i < nrun; i += 32) {
        const float x = cm[i];
        nan |= x != x;
        m = fmaxf(m, x);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
    nan = __any_sync(kFull, nan);
    if (nan || m == -INFINITY) {   // no key is seen: zeros
        const float v = nan ? nanf("") : 0.f;
        for (int i = tid; i < D; i += kSolveThreads) store_f(o, i, v);
        if (tid == 0 && a.tau) a.tau[orow] = v;
        return;
    }
    // (warps share the runs out here, and again when there are more candidates than fit)
    const int c0 = (int)((long long)nrun * warp / kSolveWarps), c1 = (int)((long long)nrun * (warp + 1) / kSolveWarps);
    int sum = 0;
    for (int i0 = c0; i0 < c1; i0 += 32) {
        const int i = i0 + lane;
        const int n = i < c1 && cm[i] - m > -1.f ? cn[i] : 0;
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int y = __shfl_up_sync(kFull, incl, d);
            if (lane >= d) incl += y;
        }
        if (i < c1) off[i] = sum + incl - n;
        sum += __shfl_sync(kFull, incl, 31);
    }
    int raw;
    const int before = warps_before(sum, box, &raw);
    for (int i = c0 + lane; i < c1; i += 32) off[i] += before;
    if (tid == 0) off[nrun] = raw;
    __syncthreads();

    // ---- tau - m over what `each_y` goes through, n keys at most
    const float gamma = a.gamma;
    RowSolver sv;
    auto solve = [&](int n, float lo, auto each_y) {
        sv.done = 0;
        sv.iters = 0;
        sv.lo = lo;
        sv.hi = fmaxf(lo, -exp2f((1.f - a.alpha) * __log2f((float)n)) + 1e-6f);
        sv.tau = 0.5f * (sv.lo + sv.hi);
        for (int pass = 1;; ++pass) {
            float F0 = 0.f, F1 = 0.f, F2 = 0.f;
            each_y([&](float y) {
                float t0, t1, t2;
                entmax_terms_bf<GM>(y - sv.tau, gamma, t0, t1, t2);
                F0 += t0; F1 += t1; F2 += t2;
            });
            F0 = warp_sum(F0); F1 = warp_sum(F1); F2 = warp_sum(F2);
            if (lane == 0) { red[0][warp] = F0; red[1][warp] = F1; red[2][warp] = F2; }
            __syncthreads();
            if (tid == 0) {
                F0 = F1 = F2 = 0.f;
                for (int w = 0; w < kSolveWarps; ++w) { F0 += red[0][w]; F1 += red[1][w]; F2 += red[2][w]; }
                solver_update(sv, F0, F1, F2, gamma, gamma == 1.f, pass, kKvFtol, kKvStol);
                bc[0] = sv.tau;
                bc[1] = sv.done ? 1.f : 0.f;
            }
            __syncthreads();
            sv.tau = bc[0];
            if (bc[1] != 0.f) break;
        }
    };

    // ---- candidates above a bound of tau, in order, into shared memory.  All runs' entries are
    // one sequence, of which each warp takes an equal part.
    // calls f(y, key, is there) for 32 of the entries [from, to) at a time, and after 128 of them
    // stops where `enough` says so
    auto each = [&](int from, int to, auto f, auto enough) {
        int i = 0;   // the run that holds the first entry (by halving), then forward
#pragma unroll 1
        for (int step = kKvMaxRuns / 2; step > 0; step >>= 1)
            if (i + step < nrun && off[i + step] <= from) i += step;
        constexpr int U = 4;
#pragma unroll 1
        for (int base = from; base < to; base += 32 * U) {
            int2 c[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = base + u * 32 + lane;
                c[u] = make_int2(0, -1);
                if (e < to) {
                    while (off[i + 1] <= e) ++i;
                    c[u] = list_of(i)[e - off[i]];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) f(__int_as_float(c[u].x) - m, c[u].y, c[u].y >= 0);
            if (enough()) break;
        }
    };
    auto part = [&](int n, int w) { return (int)((long long)n * w / kSolveWarps); };
    // Kept entries lie in each warp's own part of the arrays, from e0 on.  Entry i of all parts in
    // order: which part it lies in depends on the raw counts, but not the sequence of entries, so
    // sums over i are the same from call to call.
    int e0 = 0, mine = 0;
    int ends[kSolveWarps], from[kSolveWarps];
    auto close_up = [&](int n) {
        __syncthreads();
        if (lane == 0) { box[warp] = n; box2[warp] = e0; }
        __syncthreads();
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kSolveWarps; ++w) {
            from[w] = box2[w] - sum;
            sum += box[w];
            ends[w] = sum;
        }
        return sum;
    };
    auto where = [&](int i) {
        int f = from[0];
#pragma unroll
        for (int k = 0; k + 1 < kSolveWarps; ++k)
            if (i >= ends[k]) f = from[k + 1];
        return f + i;
    };
    // the entries of the first n that lie above `bound`; false where they are more than fit, which
    // the warps' common count tells before all are looked through
    auto gather = [&](int n, float bound, int* total) {
        const int p0 = part(n, warp), p1 = part(n, warp + 1);
        auto place = [&](int room) {
            int told = mine = 0;
            each(p0, p1, [&](float y, int j, bool there) {
                const bool take = there && y > bound;
                const unsigned mask = __ballot_sync(kFull, take);
                const int p = mine + __popc(mask & ((1u << lane) - 1u));
                if (take && p < room) {
                    ys[e0 + p] = y;
                    js[e0 + p] = j;
                }
                mine += __popc(mask);
            }, [&] {
                // (one lane reads: the warp must go on or stop as one)
                int all = 0;
                if (lane == 0) {
                    if (mine > told) atomicAdd(&found, mine - told);
                    all = *const_cast<volatile int*>(&found);
                }
                told = mine;
                return __shfl_sync(kFull, all, 0) > kCap;
            });
        };
        __syncthreads();
        if (tid == 0) found = 0;
        __syncthreads();
        // where all would fit, each warp has the room; else an equal share, and if that was too
        // little for one of them, what they counted
        const int room = n <= kCap ? p1 - p0 : kCap / kSolveWarps;
        e0 = n <= kCap ? p0 : warp * room;
        place(room);
        const bool again = __syncthreads_or(mine > room);
        if (found > kCap) return false;
        if (again) {
            e0 = warps_before(mine, box, total);   // (its barriers: `found` was read by all)
            if (tid == 0) found = 0;
            __syncthreads();
            place(mine);
        }
        *total = close_up(mine);
        return true;
    };
    // tau > m - 1.  Where more entries lie above that than fit, tau also lies above the tau of
    // fewer keys: of the first runs that surely fit, then of eight times as many above that, and
    // so on (with the dense weights of alpha 1.25 the first drops nine candidates of ten).  What
    // decides is the count above m - 1, which the keys alone determine; how many entries the lists
    // hold besides is a matter of timing, and deciding by that number, though it spares a row of
    // many entries the first look (sixteen sequences of 32768 at alpha 1.25 take 366 us, not 354;
    // of 16384 with 4300 a row above m - 1 116, not 158), changed last bits from call to call.
    float bound = -1.f;
    int total = 0;
    bool fits;
    for (int runs = nrun, first = 1;; first = 0) {
        fits = gather(off[min(runs, nrun)], bound, &total);
        if (first) {
            if (fits) break;
            runs = max(1, kCap / stride);
            continue;
        }
        if (runs >= nrun) break;
        if (fits && total > 0) {   // (no key of the first runs may be near m)
            solve(total, -1.f, [&](auto add) {
                for (int i = tid; i < total; i += kSolveThreads) add(ys[where(i)]);
            });
            bound = fmaxf(bound, sv.tau - 2e-6f);   // (it stops within 2e-7 of the sum, a step of it at most)
            __syncthreads();
        }
        runs = runs > nrun / 8 ? nrun : runs * 8;
    }
    if (!fits) {
        // scores too equal: the lists stay in the workspace, closed up so that what follows does
        // not depend on what else the scores kernel left in them
        mine = 0;
        for (int i = c0; i < c1; ++i) {
            int2* list = list_of(i);
            const int n = off[i + 1] - off[i];
            int kept = 0;
            for (int b0 = 0; b0 < n; b0 += 32) {
                const int e = b0 + lane;
                const int2 c = e < n ? list[e] : make_int2(0, -1);
                const bool take = c.y >= 0 && __int_as_float(c.x) - m > bound;
                const unsigned mask = __ballot_sync(kFull, take);
                if (take) list[kept + __popc(mask & ((1u << lane) - 1u))] = c;
                kept += __popc(mask);
                __syncwarp();
            }
            __syncwarp();
            if (lane == 0) cn[i] = kept;
            __syncwarp();
            mine += kept;
        }
        total = close_up(mine);
    }

    solve(total, -1.f, [&](auto add) {
        if (fits) {
            for (int i = tid; i < total; i += kSolveThreads) add(ys[where(i)]);
        } else {
            for (int i = c0; i < c1; ++i) {
                const int n = cn[i];
                const int2* list = list_of(i);
                for (int e = lane; e < n; e += 32) add(__int_as_float(list[e].x) - m);
            }
        }
    });
    if (tid == 0 && a.tau) a.tau[orow] = sv.tau + m;

    // ---- O over the support
    const int slot = lane / LPK, t = lane - slot * LPK;   // key slot of the warp, word of the row
    const int grp = t % G;
    const int* table = a.table + (size_t)b * a.g.max_pages;
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.v_codes);
    const uint32_t* meta = reinterpret_cast<const uint32_t*>(a.v_meta);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    auto fetch = [&](int j, uint32_t& w, uint32_t& mt) {
        const int page = kv4_page(a.g, table, j);
        w = mt = 0u;
        if (page >= 0) {
            const size_t row = kv4_row(a.g, a.Hkv, page, hk, j);
            w = __ldg(codes + row * (D / 8) + t);
            mt = __ldg(meta + row * G + grp);
        }
    };
    auto weigh = [&](float p, uint32_t w, uint32_t mt) {   // (values first: the pair's terms cancel)
        const float sc = bf16_lo(mt), z = bf16_hi(mt);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(p, fmaf(sc, (float)((w >> (4 * i)) & 15u), z), acc[i]);
    };
    if (fits) {
        // the support in key order, over the same arrays: each warp compacts its own run
        int n = 0;
        for (int base = 0; base < mine; base += 32) {
            const int e = base + lane;
            const float p = e < mine ? entmax_p<GM>(ys[e0 + e] - sv.tau, gamma) : 0.f;
            const int j = e < mine ? js[e0 + e] : 0;
            const unsigned mask = __ballot_sync(kFull, p > 0.f);
            __syncwarp();
            if (p > 0.f) {
                const int q = e0 + n + __popc(mask & ((1u << lane) - 1u));
                ys[q] = p;
                js[q] = j;
            }
            n += __popc(mask);
            __syncwarp();
        }
        const int sup = close_up(n);
        constexpr int U = 8, STEP = kSolveWarps * KPW;
        for (int i0 = warp * KPW + slot; i0 < sup; i0 += U * STEP) {
            float p[U];
            uint32_t w[U], mt[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * STEP;
                p[u] = 0.f;
                w[u] = mt[u] = 0u;
                if (i < sup) {
                    const int q = where(i);
                    p[u] = ys[q];
                    fetch(js[q], w[u], mt[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) weigh(p[u], w[u], mt[u]);
        }
    } else {
        // 32 candidates at a time: each lane its weight, then the warp's key slots take those that
        // have one, four rounds of loads in flight
        for (int i = c0; i < c1; ++i) {
            const int n = cn[i];
            const int2* list = list_of(i);
            for (int b0 = 0; b0 < n; b0 += 32) {
                const int2 c = b0 + lane < n ? list[b0 + lane] : make_int2(0, 0);
                const float pl = b0 + lane < n ? entmax_p<GM>(__int_as_float(c.x) - m - sv.tau, gamma) : 0.f;
                unsigned left = __ballot_sync(kFull, pl > 0.f);
                while (left) {
                    constexpr int U = 4;
                    float p[U];
                    uint32_t w[U], mt[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int from = __fns(left, 0, slot + 1);   // the slot's bit of what is left (-1: none)
                        const float pu = __shfl_sync(kFull, pl, from & 31);
                        const int ju = __shfl_sync(kFull, c.y, from & 31);
                        p[u] = 0.f;
                        w[u] = mt[u] = 0u;
                        if (from >= 0 && from < 32) {
                            p[u] = pu;
                            fetch(ju, w[u], mt[u]);
                        }
#pragma unroll
                        for (int k = 0; k < KPW; ++k) left &= left - 1u;
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) weigh(p[u], w[u], mt[u]);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
        for (int d = LPK; d < 32; d <<= 1) acc[i] += __shfl_xor_sync(kFull, acc[i], d);
    }
    if (slot == 0) {
        // word t = c G + w holds dimensions 32 w + 8 c ..
#pragma unroll
        for (int i = 0; i < 8; ++i) halves[warp][32 * (t % G) + 8 * (t / G) + i] = acc[i];
    }
    __syncthreads();
    for (int i = tid; i < D; i += kSolveThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kSolveWarps; ++w) v += halves[w][i];
        store_f(o, i, v);
    }
}

// ------------------------------------------------------------------ launches
template <typename T, int D>
cudaError_t write_or_read(const Kv4Args& a, bool write, cudaStream_t s) {
    constexpr int rows = RowParts<D>::kRows;
    const dim3 grid((a.g.L + rows - 1) / rows, a.g.B * a.Hkv, 2);
    if (write) kv4_write_kernel<T, D><<<grid, kKvThreads, 0, s>>>(a);
    else kv4_read_kernel<T, D><<<grid, kKvThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int D, int R>
cudaError_t launch_scores(const Kv4Args& a, cudaStream_t s) {
    const dim3 grid((a.nrun + kScoreWarps - 1) / kScoreWarps, a.blocks, a.g.B * a.Hkv);
    constexpr int sm = kScoreWarps * ScoreSmem<D, R>::kBytes;
    if (sm > 47 * 1024) {   // (beside the static part)
        cudaError_t e = cudaFuncSetAttribute(kv4_scores_kernel<T, D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, sm);
        if (e != cudaSuccess) return e;
    }
    kv4_scores_kernel<T, D, R><<<grid, kScoreThreads, sm, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t attn(const Kv4Args& a, int gm, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (a.nchunk > 0) switch (a.block) {   // (a call that covers no token: zeros only)
        case 4: e = launch_scores<T, D, 4>(a, s); break;
        case 8: e = launch_scores<T, D, 8>(a, s); break;
        case 16: e = launch_scores<T, D, 16>(a, s); break;
        default:   // (float32 rows of 128 stay at 16)
            if constexpr (!(sizeof(T) == 4 && D == 128)) e = launch_scores<T, D, 32>(a, s);
            break;
    }
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.g.B * a.Hkv * a.g.L * a.group));
    cfg.blockDim = dim3(kSolveThreads);
    cfg.dynamicSmemBytes = (size_t)(2 * kCap + a.nrun + 1) * 4;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = a.nchunk > 0 ? 1 : 0;   // (behind a kernel that is not ours it starts in order: it reads the lengths first)
    auto kern = gm == 1 ? kv4_solve_kernel<T, D, 1> : gm == 2 ? kv4_solve_kernel<T, D, 2>
              : gm == 3 ? kv4_solve_kernel<T, D, 3> : gm == 4 ? kv4_solve_kernel<T, D, 4> : kv4_solve_kernel<T, D, 0>;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t kv4_write(const Kv4Args& a, int d, bool bf16, cudaStream_t s) {
    if (bf16) return d == 128 ? write_or_read<__nv_bfloat16, 128>(a, true, s)
                   : d == 64 ? write_or_read<__nv_bfloat16, 64>(a, true, s)
                             : write_or_read<__nv_bfloat16, 32>(a, true, s);
    return d == 128 ? write_or_read<float, 128>(a, true, s)
         : d == 64 ? write_or_read<float, 64>(a, true, s) : write_or_read<float, 32>(a, true, s);
}

cudaError_t kv4_read(const Kv4Args& a, int d, bool bf16, cudaStream_t s) {
    if (bf16) return d == 128 ? write_or_read<__nv_bfloat16, 128>(a, false, s)
                   : d == 64 ? write_or_read<__nv_bfloat16, 64>(a, false, s)
                             : write_or_read<__nv_bfloat16, 32>(a, false, s);
    return d == 128 ? write_or_read<float, 128>(a, false, s)
         : d == 64 ? write_or_read<float, 64>(a, false, s) : write_or_read<float, 32>(a, false, s);
}

cudaError_t kv4_attn(const Kv4Args& a, int d, bool bf16, int gm, cudaStream_t s) {
    if (bf16) return d == 128 ? attn<__nv_bfloat16, 128>(a, gm, s)
                   : d == 64 ? attn<__nv_bfloat16, 64>(a, gm, s) : attn<__nv_bfloat16, 32>(a, gm, s);
    return d == 128 ? attn<float, 128>(a, gm, s) : d == 64 ? attn<float, 64>(a, gm, s) : attn<float, 32>(a, gm, s);
}

}  // namespace ent
