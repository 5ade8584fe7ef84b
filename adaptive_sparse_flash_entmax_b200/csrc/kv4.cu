// kv4.cu -- a paged key/value cache held in 4 bits, and alpha-entmax attention of the
// newest tokens against it (layout and visibility: kv4_index.h).
//
//   kv4_write_kernel    new keys and values quantised as they are written;
//   kv4_read_kernel     a stretch of every sequence as values again;
//   kv4_scores_kernel   x = (alpha-1) q.k / sqrt(d) of a chunk of keys against the rows of
//                       one key head, and the keys with x > (the chunk's maximum) - 1;
//   kv4_solve_kernel    per query row: tau over all chunks' keys, then O = sum p_j v_j over
//                       the support alone.
// tau >= m - 1 (m the row maximum) and a chunk's maximum is at most m, so a key at or below
// its chunk's maximum - 1 has p = 0: the scores never leave the chip but for the few that
// can weigh, and value rows without a weight are never read.
#include "kernels.h"

#include <cuda_fp16.h>

namespace ent {

namespace {

constexpr int kKvThreads = 256;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

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

// ------------------------------------------------------------------ write
// Four threads per group of 32 dimensions, 8 each; blockIdx.y: 0 keys, 1 values.
//     zero = bf16(min),  scale = bf16((max - zero) / 15),  code = rint((x - zero) / scale)
// as they are in 64-bit arithmetic, so that the codes do not depend on who computes them:
// the pair is computed in double by the group's threads, and an element's code in float
// where its quotient is clear of a half-integer, in double where it is not (float's
// quotient is within 2^-22 of it relative, at most 4e-6 for one up to 15.1; the few
// elements nearer than 1e-4 to a tie, exact ties among them, take the division again).
// A group with a NaN, an infinity, or a minimum that rounds to one is stored as (0, NaN):
// it reads back as NaN.
template <typename T, int D>
__global__ void __launch_bounds__(kKvThreads) kv4_write_kernel(const Kv4Args a) {
    constexpr int TPR = D / 8, G = D / kKvGroup;
    const T* src = static_cast<const T*>(blockIdx.y ? a.v : a.k);
    uint32_t* codes = reinterpret_cast<uint32_t*>(blockIdx.y ? a.v_codes : a.k_codes);
    uint32_t* meta = reinterpret_cast<uint32_t*>(blockIdx.y ? a.v_meta : a.k_meta);
    const long long item = (long long)blockIdx.x * kKvThreads + threadIdx.x;
    const long long row = item / TPR;   // (b * Hkv + h) * L + l
    const int t = (int)(item % TPR);
    if (row >= (long long)a.g.B * a.Hkv * a.g.L) return;   // whole quads leave together
    const int l = (int)(row % a.g.L);
    const int bh = (int)(row / a.g.L), b = bh / a.Hkv, h = bh - b * a.Hkv;
    const Kv4Seq s = seq_of(a, b);
    if (s.bad && a.bad && l == 0 && t == 0) atomicOr(a.bad, s.bad);
    if (l >= s.rows) return;
    const int pos = s.start + l;
    const int page = kv4_page(a.g, a.table + (size_t)b * a.g.max_pages, pos);
    if (page < 0) {
        if (a.bad && t == 0) atomicOr(a.bad, kKvBadPage);
        return;
    }
    const unsigned quad = 0xfu << (threadIdx.x & 28);
    float x[8];
    load8(src + row * D + t * 8, x);
    float lo = x[0], hi = x[0];
    bool fine = isfinite(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        fine &= isfinite(x[i]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(quad, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(quad, hi, o));
        fine &= __shfl_xor_sync(quad, (int)fine, o) != 0;
    }
    const __nv_bfloat16 zb = __float2bfloat16_rn(lo);
    const float z = __bfloat162float(zb);
    fine &= isfinite(z);
    const double range = (double)hi - (double)z;
    const __nv_bfloat16 sb = __float2bfloat16_rn(fine && range > 0. ? (float)(range / 15.) : 0.f);
    const float sc = __bfloat162float(sb);
    uint32_t w = 0;
    if (sc > 0.f) {
        const float inv = 1.f / sc;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float qv = (x[i] - z) * inv;   // (an underflowing or overflowing inverse is caught below)
            float r = rintf(qv);
            if (!(fabsf(fabsf(qv - r) - 0.5f) > 1e-4f) || !(inv >= 1e-30f && inv <= 1e30f)) {
                const double qd = ((double)x[i] - (double)z) / (double)sc;
                r = (float)rint(qd);
            }
            w |= (uint32_t)fminf(fmaxf(r, 0.f), 15.f) << (4 * i);
        }
    }
    const size_t at = kv4_row(a.g, a.Hkv, page, h, pos);
    const int grp = t >> 2, c = t & 3;
    codes[at * (D / 8) + c * G + grp] = w;
    if (c == 0) {
        const uint32_t zw = fine ? (uint32_t)__bfloat16_as_ushort(zb) : 0x7fffu;
        meta[at * G + grp] = (uint32_t)__bfloat16_as_ushort(sb) | zw << 16;
    }
}

// ------------------------------------------------------------------ read
// A thread per word of codes: 8 values zero + scale * code (one fused multiply-add each:
// exact but for the last rounding).  Rows past new_lens, and rows of a page outside the
// pool, are zeros.
template <typename T, int D>
__global__ void __launch_bounds__(kKvThreads) kv4_read_kernel(const Kv4Args a) {
    constexpr int TPR = D / 8, G = D / kKvGroup;
    T* dst = static_cast<T*>(blockIdx.y ? a.v_out : a.k_out);
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(blockIdx.y ? a.v_codes : a.k_codes);
    const uint32_t* meta = reinterpret_cast<const uint32_t*>(blockIdx.y ? a.v_meta : a.k_meta);
    const long long item = (long long)blockIdx.x * kKvThreads + threadIdx.x;
    const long long row = item / TPR;
    const int t = (int)(item % TPR);
    if (row >= (long long)a.g.B * a.Hkv * a.g.L) return;
    const int l = (int)(row % a.g.L);
    const int bh = (int)(row / a.g.L), b = bh / a.Hkv, h = bh - b * a.Hkv;
    const Kv4Seq s = seq_of(a, b);
    if (s.bad && a.bad && l == 0 && t == 0) atomicOr(a.bad, s.bad);
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int grp = t >> 2, c = t & 3;
    if (l < s.rows) {
        const int pos = s.start + l;
        const int page = kv4_page(a.g, a.table + (size_t)b * a.g.max_pages, pos);
        if (page >= 0) {
            const size_t at = kv4_row(a.g, a.Hkv, page, h, pos);
            const uint32_t w = codes[at * (D / 8) + c * G + grp];
            const uint32_t m = meta[at * G + grp];
            const float sc = bf16_lo(m), z = bf16_hi(m);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf(sc, (float)((w >> (4 * i)) & 15u), z);
        } else if (a.bad && t == 0) {
            atomicOr(a.bad, kKvBadPage);
        }
    }
    store8(dst + row * D + t * 8, x);
}

// ------------------------------------------------------------------ scores
// A warp per (run of chunks of C keys, block of R rows, sequence and key head); the eight warps
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
// [2^14, 2^15): exact for bf16 values down to 2^-31 of the largest, below which the
// rounding is 2^-39 of it; a float32 row is the sum of two such halves (22 bits).
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
// the larger, or NaN where either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// x rounded to bf16, in the upper half of a word; what is left stays in x
__device__ __forceinline__ uint32_t bf16_part(float& x) {
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    x -= __bfloat162float(h);
    return (uint32_t)__bfloat16_as_ushort(h) << 16;
}

// G consecutive 4-byte words (one load)
template <int G>
__device__ __forceinline__ void load_words(const uint32_t* p, uint32_t (&w)[G]) {
    if constexpr (G == 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
    } else if constexpr (G == 2) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
        w[0] = v.x; w[1] = v.y;
    } else {
        w[0] = __ldg(p);
    }
}

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;

// R: rows of a block (4, 8, 16 or 32), in NT products of 8 columns.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kScoreThreads, R <= 8 ? 2 : 1) kv4_scores_kernel(const Kv4Args a) {
    constexpr int G = D / kKvGroup, NT = R <= 8 ? 1 : R / 8, C = kv4_chunk_keys(R), U = C / kKvTile;
    constexpr int LPR = 32 / R, KPL = C / LPR;   // lanes a row, keys a lane
    constexpr int kStride = C + 4;   // spreads a product's 8 keys x 4 row pairs over the banks
    constexpr bool F32 = sizeof(T) == 4;
    __shared__ __align__(16) float xs_all[kScoreWarps][8 * NT * kStride];
    __shared__ float row_max[R];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* xs = xs_all[warp];
    const int bk = blockIdx.z, b = bk / a.Hkv, hk = bk - b * a.Hkv;
    const Kv4Seq s = seq_of(a, b);
    if (s.bad && a.bad && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.bad, s.bad);
    const int row0 = blockIdx.y * R, nrows = s.rows * a.group;   // real rows of this key head
    const int nch = kv4_seq_chunks(a.g, s, C), run = kv4_run(nch, a.nsplit);
    const int split = blockIdx.x * kScoreWarps + warp;
    const int ch0 = split * run, ch1 = kv4_min(ch0 + run, nch);
    if (threadIdx.x < R) row_max[threadIdx.x] = -INFINITY;
    __syncthreads();
    if (row0 >= nrows || ch0 >= ch1) return;   // (the solver takes no more runs than hold a chunk)

    // ---- queries: lane (n = lane / 4, c = lane % 4) holds dimensions 32 w + 8 c + i of row n
    const int c = lane & 3;
    uint32_t qf[NT][G][4], ql[F32 ? NT : 1][G][4];   // B operands; float32 rows: high and low parts
    uint32_t qz[NT][3];                              // sum q of group c in three parts
    // the row that this lane looks through, in its lanes' part `sub`, and its factors
    const int lrow = lane / LPR, sub = lane % LPR;
    float mul = 0.f, mul2 = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int r = row0 + nt * 8 + (lane >> 2);
        const bool real = r < nrows && nt * 8 + (lane >> 2) < R;
        const int l = real ? r / a.group : 0, gi = real ? r - l * a.group : 0;
        const T* q = static_cast<const T*>(a.q) + (((size_t)b * a.Hkv * a.group + hk * a.group + gi) * a.g.L + l) * D;
        float x[G][8];
        float top = 0.f;
        bool fine = true;
#pragma unroll
        for (int w = 0; w < G; ++w) {
            if (real) load8(q + 32 * w + 8 * c, x[w]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (!real) x[w][i] = 0.f;
                fine &= isfinite(x[w][i]);
                top = fmaxf(top, fabsf(x[w][i]));
            }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
            fine &= __shfl_xor_sync(kFull, (int)fine, o) != 0;
        }
        int e = 0;
        if (top > 0.f && fine) { frexpf(top, &e); e = 15 - e; }
        const float fe1 = ldexpf(1.f, e / 2), fe2 = ldexpf(1.f, e - e / 2);
        float zsum = 0.f;
#pragma unroll
        for (int w = 0; w < G; ++w) {
            float sum = 0.f, hi[8], lo[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float y = x[w][i] * fe1 * fe2;   // 2^e in two exact steps
                hi[i] = __half2float(__float2half_rn(y));
                lo[i] = y - hi[i];
                sum += y;
            }
            const float f = 0.0625f;
            qf[nt][w][0] = pack_half(hi[0], hi[4]);
            qf[nt][w][1] = pack_half(hi[1] * f, hi[5] * f);
            qf[nt][w][2] = pack_half(hi[2], hi[6]);
            qf[nt][w][3] = pack_half(hi[3] * f, hi[7] * f);
            if constexpr (F32) {
                ql[nt][w][0] = pack_half(lo[0], lo[4]);
                ql[nt][w][1] = pack_half(lo[1] * f, lo[5] * f);
                ql[nt][w][2] = pack_half(lo[2], lo[6]);
                ql[nt][w][3] = pack_half(lo[3] * f, lo[7] * f);
            }
            sum += __shfl_xor_sync(kFull, sum, 1);
            sum += __shfl_xor_sync(kFull, sum, 2);
            if (w == c) zsum = sum * 5.9604644775390625e-08f;   // 2^-24, the codes' unit
        }
        qz[nt][0] = bf16_part(zsum);
        qz[nt][1] = bf16_part(zsum);
        qz[nt][2] = bf16_part(zsum);
        // x = cx 2^(24 - e) s: in two factors, either of which is in range
        const int e1 = (24 - e) / 2;
        // a row with a NaN or an infinity has NaN scores
        const float f1 = fine ? a.cx * ldexpf(1.f, e1) : nanf(""), f2 = ldexpf(1.f, 24 - e - e1);
        const float g1 = __shfl_sync(kFull, f1, 4 * (lrow & 7)), g2 = __shfl_sync(kFull, f2, 4 * (lrow & 7));
        if (lrow >> 3 == nt) { mul = g1; mul2 = g2; }
    }

    // ---- keys, a chunk of U tiles at a time
    const int* table = a.table + (size_t)b * a.g.max_pages;
    const int key = lane >> 2;   // the lane's keys of a tile: key and key + 8
    const bool lreal = row0 + lrow < nrows;
    const int lpos = lreal ? s.start + (row0 + lrow) / a.group : -1;
    const size_t list = ((size_t)bk * a.g.L * a.group + row0 + lrow) * a.nsplit + split;
    int2* out = a.cand + list * a.cap;
    const int pos_first = s.start + row0 / a.group;
    const int pos_last = s.start + (kv4_min(row0 + R, nrows) - 1) / a.group;
    float m = -INFINITY;    // of the row, over the run so far
    int n = 0;              // candidates of the row so far
    // chunk ch holds keys k0 .. k1-1 (kv4_chunk, with what does not change taken out)
    const int ns = kv4_sink_chunks(a.g, C), sink_end = kv4_min(kv4_sink_end(a.g), s.end);
    const int base = kv4_base(a.g, s.start) - ns * C;
    auto first_key = [&](int ch) { return ch * C + (ch < ns ? 0 : base); };
    auto end_key = [&](int ch, int k0) { return kv4_min(k0 + C, ch < ns ? sink_end : s.end); };
    // page of tile `lane` of a chunk (lanes below U), one chunk ahead of its loads
    auto page_of = [&](int ch) {
        int p = -1;
        if (ch < ch1 && lane < U) {
            const int k0 = first_key(ch), kb = k0 + lane * kKvTile;
            if (kb < end_key(ch, k0)) {
                p = kv4_page(a.g, table, kb);
                if (p < 0 && a.bad) atomicOr(a.bad, kKvBadPage);
            }
        }
        return p;
    };
    // bytes: of a token, of a page of all heads, and the lane's place in this head's page
    constexpr int kTokenB = D / 2, kMetaB = 4 * G;
    const size_t page_b = (size_t)a.Hkv << a.g.page_shift;
    const int mask = (1 << a.g.page_shift) - 1;
    const char* lane_codes = reinterpret_cast<const char*>(a.k_codes) +
                             (((size_t)hk << a.g.page_shift) + key) * kTokenB + c * 4 * G;
    const char* lane_meta = reinterpret_cast<const char*>(a.k_meta) +
                            (((size_t)hk << a.g.page_shift) + key) * kMetaB;
    int pages = page_of(ch0);
#pragma unroll 1
    for (int ch = ch0; ch < ch1; ++ch) {
        const int k0 = first_key(ch), k1 = end_key(ch, k0);
        uint32_t w[U][2][G], mt[U][2][G];
        const unsigned has = __ballot_sync(kFull, pages >= 0);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            // a tile that is not there reads the pool's first page instead, and no row sees it
            const int page = max(__shfl_sync(kFull, pages, u), 0);
            const size_t row = page * page_b + ((k0 + u * kKvTile) & mask);
            const char* pc = lane_codes + row * kTokenB;
            const char* pm = lane_meta + row * kMetaB;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                load_words<G>(reinterpret_cast<const uint32_t*>(pc + 8 * h * kTokenB), w[u][h]);
                load_words<G>(reinterpret_cast<const uint32_t*>(pm + 8 * h * kMetaB), mt[u][h]);
            }
        }
        pages = page_of(ch + 1);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float acc[NT][4];
            uint32_t mz[2];   // the pair of group c (lanes past the groups: zeros)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                mz[h] = c == 0 ? mt[u][h][0] : 0u;
#pragma unroll
                for (int i = 1; i < G; ++i) mz[h] = c == i ? mt[u][h][i] : mz[h];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma_16816_bf_0(acc[nt], mz[0], mz[1], mz[0], mz[1], qz[nt][0], qz[nt][1]);
                mma_1688_bf(acc[nt], mz[0], mz[1], qz[nt][2]);
            }
#pragma unroll
            for (int i = 0; i < G; ++i) {
                uint32_t w0 = w[u][0][i], w1 = w[u][1][i];
                uint32_t av[8];
                av[0] = w0 & 0x000f000fu; av[1] = w1 & 0x000f000fu;
                av[2] = w0 & 0x00f000f0u; av[3] = w1 & 0x00f000f0u;
                w0 >>= 8; w1 >>= 8;
                av[4] = w0 & 0x000f000fu; av[5] = w1 & 0x000f000fu;
                av[6] = w0 & 0x00f000f0u; av[7] = w1 & 0x00f000f0u;
                const float s0 = bf16_lo(mt[u][0][i]), s1 = bf16_lo(mt[u][1][i]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float d[4];
                    mma_16816_0(d, av[0], av[1], av[2], av[3], qf[nt][i][0], qf[nt][i][1]);
                    mma_16816(d, av[4], av[5], av[6], av[7], qf[nt][i][2], qf[nt][i][3]);
                    if constexpr (F32) {
                        mma_16816(d, av[0], av[1], av[2], av[3], ql[nt][i][0], ql[nt][i][1]);
                        mma_16816(d, av[4], av[5], av[6], av[7], ql[nt][i][2], ql[nt][i][3]);
                    }
                    acc[nt][0] = fmaf(s0, d[0], acc[nt][0]);
                    acc[nt][1] = fmaf(s0, d[1], acc[nt][1]);
                    acc[nt][2] = fmaf(s1, d[2], acc[nt][2]);
                    acc[nt][3] = fmaf(s1, d[3], acc[nt][3]);
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
        // ---- the row's part of the chunk: keys (i * LPR + sub) * 4 + e
        float v[KPL];
#pragma unroll
        for (int i = 0; i < KPL / 4; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(xs + lrow * kStride + (i * LPR + sub) * 4);
            v[4 * i] = f.x * mul * mul2; v[4 * i + 1] = f.y * mul * mul2;
            v[4 * i + 2] = f.z * mul * mul2; v[4 * i + 3] = f.w * mul * mul2;
        }
        __syncwarp();
        // not every row sees every key of the chunk: those it does not see leave as -inf
        const bool whole = has == (1u << U) - 1u && k1 - k0 == C && k1 - 1 <= pos_first &&
                           (!a.g.window || k1 <= a.g.sinks || k0 > pos_last - a.g.window);
        if (!whole) {
#pragma unroll
            for (int i = 0; i < KPL; ++i) {
                const int kk = ((i >> 2) * LPR + sub) * 4 + (i & 3);
                const bool see = k0 + kk < k1 && (has >> (kk / kKvTile) & 1u) && kv4_sees(a.g, lpos, k0 + kk);
                v[i] = see ? v[i] : -INFINITY;
            }
        }
        // a NaN passes through every maximum; +inf is caught at the end.  (A store that loses to
        // another warp's costs a weaker filter, no more.)
        m = max_nan(m, *const_cast<volatile float*>(&row_max[lrow]));
#pragma unroll
        for (int i = 0; i < KPL; ++i) m = max_nan(m, v[i]);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, o));
        if (sub == 0) *const_cast<volatile float*>(&row_max[lrow]) = m;
        // above m - 1, and the maximum itself: where |m| >= 2^24 makes them equal, the limit is
        // the next float below m (m = -inf or NaN: it is NaN, and nothing is above)
        float lim = m - 1.f;
        if (!(lim < m)) lim = __int_as_float(__float_as_int(m) + (m > 0.f ? -1 : 1));
        unsigned take = 0;
#pragma unroll
        for (int i = 0; i < KPL; ++i) take |= (v[i] > lim ? 1u : 0u) << i;
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
#pragma unroll
        for (int i = 0; i < KPL; ++i)
            if (take >> i & 1u)
                out[put++] = make_int2(__float_as_int(v[i]), k0 + ((i >> 2) * LPR + sub) * 4 + (i & 3));
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (lreal && sub == 0) {
        a.split_max[list] = m < INFINITY ? m : nanf("");
        a.split_n[list] = n;
    }
}

// ------------------------------------------------------------------ solve and P.V
// One CTA per query row.  The runs' candidates are gathered in key order into shared memory,
// those above m - 1 (m the maximum over the runs) kept, tau - m is found by Halley-bisection
// from the bracket [-1, -n^(1-alpha)] (n the candidates' count: f <= 0 there since at most n
// keys weigh), and O accumulates over the support, D/8 lanes per value row.  Scores are held
// relative to m, so tau keeps its precision for scores of any size.  Every sum has a fixed
// order: the result does not change from run to run.  A row with more than kCap candidates
// even above m - 1 goes over the runs' lists again in every pass.
constexpr int kSolveThreads = 128;
constexpr int kSolveWarps = kSolveThreads / 32;
constexpr int kCap = 4096;
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
__global__ void __launch_bounds__(kSolveThreads) kv4_solve_kernel(const Kv4Args a) {
    constexpr int G = D / kKvGroup, LPK = D / 8, KPW = 32 / LPK;
    __shared__ float ys[kCap];          // x - m of the candidates, then their weights
    __shared__ int js[kCap];            // their keys
    __shared__ int off[kKvMaxSplit + 1];   // the runs' candidates before each run
    __shared__ float red[3][kSolveWarps];
    __shared__ int box[kSolveWarps], box2[kSolveWarps];
    __shared__ float bc[2];
    __shared__ float part[kSolveWarps][D];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = a.g.L * a.group;    // rows of one key head
    const int bk = blockIdx.x / per, r = blockIdx.x - bk * per;
    const int b = bk / a.Hkv, hk = bk - b * a.Hkv;
    const int l = r / a.group, gi = r - l * a.group;
    const Kv4Seq s = seq_of(a, b);
    const size_t orow = ((size_t)b * a.Hkv * a.group + hk * a.group + gi) * a.g.L + l;
    T* o = static_cast<T*>(a.o) + orow * D;
    int nrun = 0;
    if (l < s.rows) {
        const int nch = kv4_seq_chunks(a.g, s, a.chunk), run = kv4_run(nch, a.nsplit);
        nrun = run > 0 ? (nch + run - 1) / run : 0;
    }
    const size_t at = ((size_t)bk * per + r) * a.nsplit;
    const float* cm = a.split_max + at;
    const int* cn = a.split_n + at;
    const int2* cand = a.cand + at * a.cap;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // ---- row maximum (every warp for itself), then the runs' offsets, a quarter each warp
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

    // ---- candidates: each warp holds a run [e0, e0 + mine) of the arrays
    const bool direct = raw <= kCap;
    bool fits = true;
    int e0, mine = 0, total;
    if (direct) {
        e0 = (int)((long long)raw * warp / kSolveWarps);
        const int e1 = (int)((long long)raw * (warp + 1) / kSolveWarps);
        int i = 0;   // the run that holds entry e0 (by halving), then forward
        for (int step = kKvMaxSplit; step > 0; step >>= 1)
            if (i + step < nrun && off[i + step] <= e0) i += step;
        constexpr int U = 4;
        for (int base = e0; base < e1; base += 32 * U) {
            int2 c[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int e = base + u * 32 + lane;
                c[u] = make_int2(0, -1);
                if (e < e1) {
                    while (off[i + 1] <= e) ++i;
                    c[u] = cand[(size_t)i * a.cap + (e - off[i])];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float y = __int_as_float(c[u].x) - m;
                const bool take = c[u].y >= 0 && y > -1.f;
                const unsigned mask = __ballot_sync(kFull, take);
                if (take) {
                    const int p = e0 + mine + __popc(mask & ((1u << lane) - 1u));
                    ys[p] = y;
                    js[p] = c[u].y;
                }
                mine += __popc(mask);
            }
        }
    } else {
        // each warp closes up its own lists in the workspace, so that what follows does not
        // depend on what the scores kernel left in them
        for (int i = c0; i < c1; ++i) {
            int2* list = a.cand + (at + i) * a.cap;
            const int n = off[i + 1] - off[i];
            int kept = 0;
            for (int b0 = 0; b0 < n; b0 += 32) {
                const int e = b0 + lane;
                const int2 c = e < n ? list[e] : make_int2(0, -1);
                const bool take = c.y >= 0 && __int_as_float(c.x) - m > -1.f;
                const unsigned mask = __ballot_sync(kFull, take);
                if (take) list[kept + __popc(mask & ((1u << lane) - 1u))] = c;
                kept += __popc(mask);
                __syncwarp();
            }
            if (lane == 0) a.split_n[at + i] = kept;
            mine += kept;
        }
        __syncwarp();
        e0 = warps_before(mine, box, &total);
        fits = total <= kCap;
        int put = e0;
        for (int i = c0; fits && i < c1; ++i) {
            const int n = cn[i];
            for (int e = lane; e < n; e += 32) {
                const int2 c = cand[(size_t)i * a.cap + e];
                ys[put + e] = __int_as_float(c.x) - m;
                js[put + e] = c.y;
            }
            put += n;
        }
    }
    // entry i of all warps' runs in order: which of them lie where depends on the raw counts, but
    // not the sequence of entries, so sums over i are the same from call to call
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
    const int all = close_up(mine);
    if (direct) total = all;

    // ---- tau - m
    const float gamma = a.gamma;
    RowSolver sv;
    sv.done = 0;
    sv.iters = 0;
    sv.lo = -1.f;
    sv.hi = fmaxf(-1.f, -exp2f((1.f - a.alpha) * __log2f((float)total)) + 1e-6f);
    sv.tau = 0.5f * (sv.lo + sv.hi);
    for (int pass = 1;; ++pass) {
        float F0 = 0.f, F1 = 0.f, F2 = 0.f;
        auto add = [&](float y) {
            float t0, t1, t2;
            entmax_terms_bf<GM>(y - sv.tau, gamma, t0, t1, t2);
            F0 += t0; F1 += t1; F2 += t2;
        };
        if (fits) {
            for (int i = tid; i < total; i += kSolveThreads) add(ys[where(i)]);
        } else {
            for (int i = c0; i < c1; ++i) {
                const int n = cn[i];
                for (int e = lane; e < n; e += 32) add(__int_as_float(cand[(size_t)i * a.cap + e].x) - m);
            }
        }
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
    if (tid == 0 && a.tau) a.tau[orow] = sv.tau + m;

    // ---- O over the support
    const int slot = lane / LPK, t = lane - slot * LPK;   // key slot of the warp, word of the row
    const int grp = t % G;
    const int* table = a.table + (size_t)b * a.g.max_pages;
    const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.v_codes);
    const uint32_t* meta = reinterpret_cast<const uint32_t*>(a.v_meta);
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, accz = 0.f;
    auto fetch = [&](int j, uint32_t& w, uint32_t& mt) {
        const int page = kv4_page(a.g, table, j);
        w = mt = 0u;
        if (page >= 0) {
            const size_t row = kv4_row(a.g, a.Hkv, page, hk, j);
            w = __ldg(codes + row * (D / 8) + t);
            mt = __ldg(meta + row * G + grp);
        }
    };
    auto weigh = [&](float p, uint32_t w, uint32_t mt) {
        const float ps = p * bf16_lo(mt);
        accz = fmaf(p, bf16_hi(mt), accz);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(ps, (float)((w >> (4 * i)) & 15u), acc[i]);
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
        for (int i = c0; i < c1; ++i) {
            const int n = cn[i];
            for (int e = slot; e < n; e += KPW) {
                const int2 c = cand[(size_t)i * a.cap + e];
                const float p = entmax_p<GM>(__int_as_float(c.x) - m - sv.tau, gamma);
                if (!(p > 0.f)) continue;
                uint32_t w, mt;
                fetch(c.y, w, mt);
                weigh(p, w, mt);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        acc[i] += accz;
#pragma unroll
        for (int d = LPK; d < 32; d <<= 1) acc[i] += __shfl_xor_sync(kFull, acc[i], d);
    }
    if (slot == 0) {
        // word t = c G + w holds dimensions 32 w + 8 c ..
#pragma unroll
        for (int i = 0; i < 8; ++i) part[warp][32 * (t % G) + 8 * (t / G) + i] = acc[i];
    }
    __syncthreads();
    for (int i = tid; i < D; i += kSolveThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kSolveWarps; ++w) v += part[w][i];
        store_f(o, i, v);
    }
}

// ------------------------------------------------------------------ launches
template <typename T, int D>
cudaError_t write_or_read(const Kv4Args& a, bool write, cudaStream_t s) {
    const long long items = (long long)a.g.B * a.Hkv * a.g.L * (D / 8);
    const dim3 grid((unsigned)((items + kKvThreads - 1) / kKvThreads), 2);
    if (write) kv4_write_kernel<T, D><<<grid, kKvThreads, 0, s>>>(a);
    else kv4_read_kernel<T, D><<<grid, kKvThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int D, int R>
cudaError_t launch_scores(const Kv4Args& a, cudaStream_t s) {
    const int rows = a.g.L * a.group;
    const dim3 grid((a.nsplit + kScoreWarps - 1) / kScoreWarps, (rows + R - 1) / R, a.g.B * a.Hkv);
    kv4_scores_kernel<T, D, R><<<grid, kScoreThreads, 0, s>>>(a);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t attn(const Kv4Args& a, int gm, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (a.nchunk > 0) switch (a.block) {   // (a call that covers no token: zeros only)
        case 4: e = launch_scores<T, D, 4>(a, s); break;
        case 8: e = launch_scores<T, D, 8>(a, s); break;
        case 16: e = launch_scores<T, D, 16>(a, s); break;
        default: e = launch_scores<T, D, 32>(a, s); break;
    }
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.g.B * a.Hkv * a.g.L * a.group));
    cfg.blockDim = dim3(kSolveThreads);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    switch (gm) {
        case 1: return cudaLaunchKernelEx(&cfg, kv4_solve_kernel<T, D, 1>, a);
        case 2: return cudaLaunchKernelEx(&cfg, kv4_solve_kernel<T, D, 2>, a);
        case 3: return cudaLaunchKernelEx(&cfg, kv4_solve_kernel<T, D, 3>, a);
        case 4: return cudaLaunchKernelEx(&cfg, kv4_solve_kernel<T, D, 4>, a);
        default: return cudaLaunchKernelEx(&cfg, kv4_solve_kernel<T, D, 0>, a);
    }
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
