// win_f32.cu -- float32 attention under a sliding window, forward and backward, where the
// visible scores of 16 query rows fit in shared memory (window + sinks up to 1584 at d = 32,
// 1392 at 64, 1072 at 128).
//
//     s = Q K^T / sqrt(d),  x = (alpha-1) s,  u = (x - tau)_+,  p = u^gamma,  sum p = 1,  O = P V,
//     g = u^(gamma-1),  delta = sum g dP / sum g,  dS = g (dP - delta),  dP = dO V^T,
//     dQ = dS K / sqrt(d),  dK = dS^T Q / sqrt(d),  dV = P^T dO.
//
// The general float32 kernels (simt_impl.cuh) stream the keys again for every solver pass,
// one query row a thread; here a CTA of 256 threads takes 16 rows, computes their scores once
// into shared memory and solves there, two rows a warp with no barrier between passes, and the
// products with V, K, Q and dO skip the keys without weight.  At N = 257, d = 64, two heads,
// window 64 the forward takes 14 us instead of 300 and the backward 41 instead of 295: a
// training step this small is bound by the chain of latencies in one tile, and smaller tiles
// make the chain short and the grid eight times as wide.
#include "kernels.h"

namespace ent {

namespace {

constexpr int kWinThreads = 256, kWinRows = 16, kWinChunk = 64;
constexpr unsigned kAllLanes = 0xffffffffu;

// The keys that the rows i0 .. i0+15 see, numbered without gap: n < sinks_before is key n,
// the others follow from w0 on.
struct Seen {
    int sinks_before, w0, n;
    __device__ __forceinline__ Seen(int window, int sinks, int i0, int N) {
        const int last = min(i0 + kWinRows, N) - 1;
        w0 = max(0, i0 - window + 1);
        sinks_before = min(sinks, w0);
        n = sinks_before + last + 1 - w0;
    }
    __device__ __forceinline__ int key(int k) const { return k < sinks_before ? k : w0 + k - sinks_before; }
};

__host__ __device__ constexpr int win_cols(int window, int sinks) {   // row length of the score arrays
    return (window + sinks + kWinRows + kWinChunk - 1) / kWinChunk * kWinChunk + 4;
}
template <int D>
constexpr size_t win_smem(int cols, int arrays, int tiles) {
    return sizeof(float) * ((size_t)arrays * kWinRows * cols + (size_t)tiles * kWinRows * (D + 4) +
                            2 * kWinChunk * (D + 4));
}

__device__ __forceinline__ float warp_total(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kAllLanes, x, o);
    return x;
}

// rows src[row(k)], k < n, into dst[k][D + 4]
template <int D, typename F>
__device__ __forceinline__ void stage(float* dst, const float* src, int n, F row) {
    for (int i = threadIdx.x; i < n * (D / 4); i += kWinThreads) {
        const int k = i / (D / 4), c = i % (D / 4) * 4;
        *reinterpret_cast<float4*>(dst + k * (D + 4) + c) =
            __ldg(reinterpret_cast<const float4*>(src + (size_t)row(k) * D + c));
    }
}

// r[e] = a_{4 rg + e} . b_kk for the four rows of this thread (a staged rows, b one staged row)
template <int D>
__device__ __forceinline__ void dots(float (&r)[4], const float* a, const float* b) {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
        const float4 k = *reinterpret_cast<const float4*>(b + c);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float4 q = *reinterpret_cast<const float4*>(a + e * (D + 4) + c);
            r[e] = fmaf(q.x, k.x, r[e]);
            r[e] = fmaf(q.y, k.y, r[e]);
            r[e] = fmaf(q.z, k.z, r[e]);
            r[e] = fmaf(q.w, k.w, r[e]);
        }
    }
}

// acc += w * v over this thread's D/16 columns, from column c0 on
template <int D>
__device__ __forceinline__ void add_row(float (&acc)[D / 16], float w, const float* v) {
    if constexpr (D == 32) {
        const float2 f = *reinterpret_cast<const float2*>(v);
        acc[0] = fmaf(w, f.x, acc[0]); acc[1] = fmaf(w, f.y, acc[1]);
    } else {
#pragma unroll
        for (int c = 0; c < D / 16; c += 4) {
            const float4 f = *reinterpret_cast<const float4*>(v + c);
            acc[c] = fmaf(w, f.x, acc[c]); acc[c + 1] = fmaf(w, f.y, acc[c + 1]);
            acc[c + 2] = fmaf(w, f.z, acc[c + 2]); acc[c + 3] = fmaf(w, f.w, acc[c + 3]);
        }
    }
}
template <int D>
__device__ __forceinline__ void store_row(float* dst, const float (&acc)[D / 16], float sc) {
    if constexpr (D == 32) {
        *reinterpret_cast<float2*>(dst) = make_float2(acc[0] * sc, acc[1] * sc);
    } else {
#pragma unroll
        for (int c = 0; c < D / 16; c += 4)
            *reinterpret_cast<float4*>(dst + c) =
                make_float4(acc[c] * sc, acc[c + 1] * sc, acc[c + 2] * sc, acc[c + 3] * sc);
    }
}

template <int D, int GM>
__global__ void __launch_bounds__(kWinThreads) win_fwd_f32_kernel(const FwdArgs a, int cols) {
    extern __shared__ __align__(16) float win_mem[];
    float* xs = win_mem;                              // [16][cols] x, then u
    float* qs = xs + kWinRows * cols;                 // [16][D + 4]
    float* ks = qs + kWinRows * (D + 4);              // [64][D + 4]
    __shared__ float gsum[kWinRows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bh = blockIdx.y, i0 = blockIdx.x * kWinRows, N = a.N;
    const size_t head = (size_t)bh * N * D;
    const float* q = static_cast<const float*>(a.q) + head;
    const float* k = static_cast<const float*>(a.k) + head;
    const float* v = static_cast<const float*>(a.v) + head;
    const Seen seen(a.window, a.sinks, i0, N);
    const float gamma = a.gamma;

    stage<D>(qs, q, kWinRows, [&](int r) { return min(i0 + r, N - 1); });
    for (int n0 = 0; n0 < seen.n; n0 += kWinChunk) {
        __syncthreads();
        stage<D>(ks, k, min(kWinChunk, seen.n - n0), [&](int kk) { return seen.key(n0 + kk); });
        __syncthreads();
        const int kk = tid & 63, rg = tid >> 6, n = n0 + kk;
        float r[4];
        dots<D>(r, qs + 4 * rg * (D + 4), ks + kk * (D + 4));
        const int j = seen.key(n);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + 4 * rg + e;
            const bool in = n < seen.n && i < N && j <= i && (i - j < a.window || j < a.sinks);
            xs[(4 * rg + e) * cols + n] = in ? __fmul_rn(a.cx, r[e]) : -INFINITY;
        }
    }
    __syncthreads();

    // ---- tau: two rows a warp, each in its own time
    int passes = 0;
#pragma unroll 1
    for (int rr = 0; rr < 2; ++rr) {
        const int row = warp * 2 + rr, i = i0 + row;
        if (i >= N) break;
        float* x = xs + row * cols;
        float m = -INFINITY;
        for (int n = lane; n < seen.n; n += 32) m = fmaxf(m, x[n]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAllLanes, m, o));
        RowSolver sv;
        sv.done = 0;
        sv.iters = 0;
        sv.lo = m - 1.f;
        sv.hi = fmaxf(sv.lo, m - exp2f((1.f - a.alpha) * __log2f((float)win_keys(a.window, a.sinks, i))));
        sv.tau = 0.5f * (sv.lo + sv.hi);
        float F1 = 0.f;
        for (int pass = 1; !sv.done; ++pass) {
            float F0 = 0.f, F2 = 0.f;
            F1 = 0.f;
            for (int n = lane; n < seen.n; n += 32) {
                float t0, t1, t2;
                entmax_terms_bf<GM>(x[n] - sv.tau, gamma, t0, t1, t2);
                F0 += t0; F1 += t1; F2 += t2;
            }
            F0 = warp_total(F0); F1 = warp_total(F1); F2 = warp_total(F2);
            solver_update(sv, F0, F1, F2, gamma, gamma == 1.f, pass, a.ftol, a.stol);
        }
        passes = max(passes, sv.iters);
        // (a row stops at the tau it evaluated, so F1 = sum g is that tau's)
        uint8_t* mrow = a.mask + ((size_t)bh * a.T + i / kBlk) * a.T;
        for (int n = lane; n < seen.n; n += 32) {
            const float u = x[n] - sv.tau;
            x[n] = u;
            if (u > 0.f) mrow[seen.key(n) / kBlk] = 1;   // (zeroed before the launch; every writer writes 1)
        }
        if (lane == 0) {
            a.tau[(size_t)bh * N + i] = sv.tau;
            if (a.iters) a.iters[(size_t)bh * N + i] = (uint8_t)sv.iters;
            gsum[row] = F1;
        }
    }

    // ---- O (and otilde): 16 threads a row, D/16 columns each
    const int row = tid >> 4, c0 = (tid & 15) * (D / 16), i = i0 + row;
    float acc[D / 16], accg[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c) acc[c] = accg[c] = 0.f;
    for (int n0 = 0; n0 < seen.n; n0 += kWinChunk) {
        const int nn = min(kWinChunk, seen.n - n0);
        __syncthreads();
        stage<D>(ks, v, nn, [&](int kk) { return seen.key(n0 + kk); });
        __syncthreads();
        if (i >= N) continue;
        for (int kk = 0; kk < nn; ++kk) {
            const float u = xs[row * cols + n0 + kk];
            if (!(u > 0.f)) continue;
            add_row<D>(acc, entmax_p<GM>(u, gamma), ks + kk * (D + 4) + c0);
            if (a.otilde) add_row<D>(accg, entmax_g<GM>(u, gamma), ks + kk * (D + 4) + c0);
        }
    }
    if (i < N) {
        store_row<D>(static_cast<float*>(a.o) + head + (size_t)i * D + c0, acc, 1.f);
        if (a.otilde)   // (no weight at all, as of a query with a NaN: zeros)
            store_row<D>(a.otilde + head + (size_t)i * D + c0, accg, gsum[row] > 0.f ? 1.f / gsum[row] : 0.f);
    }
    if (tid == 0 && i0 % kBlk == 0) {   // counted once per 128-row tile, whose scores are computed once
        const WinBlocks wb(a.window, a.sinks, i0 / kBlk);
        atomicAdd(&a.hdr->counters[kCtrQkBlocks], (unsigned long long)wb.count(i0 / kBlk));
        atomicAdd(&a.hdr->counters[kCtrPvBlocks], (unsigned long long)wb.count(i0 / kBlk));
        atomicAdd(&a.hdr->counters[kCtrPasses], (unsigned long long)passes);
        atomicAdd(&a.hdr->counters[kCtrTiles], 1ull);
        if (a.otilde) atomicAdd(&a.hdr->counters[kCtrGvBlocks], (unsigned long long)wb.count(i0 / kBlk));
    }
}

// delta and dQ of 16 rows: g and g dP of every visible key in shared memory, then dS = g dP -
// delta g and dQ over the keys with g > 0.
template <int D, int GM>
__global__ void __launch_bounds__(kWinThreads) win_dq_f32_kernel(const BwdArgs a, int cols) {
    extern __shared__ __align__(16) float win_mem[];
    float* gs = win_mem;                              // [16][cols] g
    float* gp = gs + kWinRows * cols;                 // [16][cols] g dP, then dS
    float* qs = gp + kWinRows * cols;                 // [16][D + 4]
    float* dos = qs + kWinRows * (D + 4);             // [16][D + 4]
    float* ks = dos + kWinRows * (D + 4);             // [64][D + 4]
    float* vs = ks + kWinChunk * (D + 4);             // [64][D + 4]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int bh = blockIdx.y, i0 = blockIdx.x * kWinRows, N = a.N;
    const size_t head = (size_t)bh * N * D;
    const float* k = static_cast<const float*>(a.k) + head;
    const float* v = static_cast<const float*>(a.v) + head;
    const Seen seen(a.window, a.sinks, i0, N);

    stage<D>(qs, static_cast<const float*>(a.q) + head, kWinRows, [&](int r) { return min(i0 + r, N - 1); });
    stage<D>(dos, static_cast<const float*>(a.dout) + head, kWinRows, [&](int r) { return min(i0 + r, N - 1); });
    float tau[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) tau[e] = a.tau[(size_t)bh * N + min(i0 + 4 * (tid >> 6) + e, N - 1)];
    for (int n0 = 0; n0 < seen.n; n0 += kWinChunk) {
        const int nn = min(kWinChunk, seen.n - n0);
        __syncthreads();
        stage<D>(ks, k, nn, [&](int kk) { return seen.key(n0 + kk); });
        stage<D>(vs, v, nn, [&](int kk) { return seen.key(n0 + kk); });
        __syncthreads();
        const int kk = tid & 63, rg = tid >> 6, n = n0 + kk;
        float r[4], dp[4];
        dots<D>(r, qs + 4 * rg * (D + 4), ks + kk * (D + 4));
        dots<D>(dp, dos + 4 * rg * (D + 4), vs + kk * (D + 4));
        const int j = seen.key(n);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = i0 + 4 * rg + e;
            const bool in = n < seen.n && i < N && j <= i && (i - j < a.window || j < a.sinks);
            // the forward's u: the same product, rounded once, minus tau
            const float g = in ? entmax_g<GM>(__fmul_rn(a.cx, r[e]) - tau[e], a.gamma) : 0.f;
            gs[(4 * rg + e) * cols + n] = g;
            gp[(4 * rg + e) * cols + n] = g > 0.f ? g * dp[e] : 0.f;
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int rr = 0; rr < 2; ++rr) {
        const int row = warp * 2 + rr, i = i0 + row;
        if (i >= N) break;
        float delta = 0.f;
        if (a.otilde) {
            const float* ot = a.otilde + head + (size_t)i * D;
            for (int c = lane; c < D; c += 32) delta = fmaf(dos[row * (D + 4) + c], ot[c], delta);
            delta = warp_total(delta);
        } else {
            float sg = 0.f, sgp = 0.f;
            for (int n = lane; n < seen.n; n += 32) { sg += gs[row * cols + n]; sgp += gp[row * cols + n]; }
            sg = warp_total(sg);
            sgp = warp_total(sgp);
            delta = sg > 0.f ? sgp / sg : 0.f;
        }
        for (int n = lane; n < seen.n; n += 32)
            gp[row * cols + n] = fmaf(-delta, gs[row * cols + n], gp[row * cols + n]);
        if (lane == 0) a.delta[(size_t)bh * N + i] = delta;
    }
    const int row = tid >> 4, c0 = (tid & 15) * (D / 16), i = i0 + row;
    float acc[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c) acc[c] = 0.f;
    for (int n0 = 0; n0 < seen.n; n0 += kWinChunk) {
        const int nn = min(kWinChunk, seen.n - n0);
        __syncthreads();
        if (seen.n > kWinChunk) {   // (a single chunk of keys is still there)
            stage<D>(ks, k, nn, [&](int kk) { return seen.key(n0 + kk); });
            __syncthreads();
        }
        if (i >= N) continue;
        for (int kk = 0; kk < nn; ++kk) {
            const float ds = gp[row * cols + n0 + kk];
            if (ds != 0.f) add_row<D>(acc, ds, ks + kk * (D + 4) + c0);
        }
    }
    if (i < N) store_row<D>(static_cast<float*>(a.dq) + head + (size_t)i * D + c0, acc, a.scale);
    if (tid == 0 && i0 % kBlk == 0) {
        const WinBlocks wb(a.window, a.sinks, i0 / kBlk);
        atomicAdd(&a.hdr->counters[kCtrBwdBlocks], 3ull * wb.count(i0 / kBlk));
    }
}

// dK and dV of 16 keys, over chunks of 64 of the queries that see one of them.
template <int D, int GM>
__global__ void __launch_bounds__(kWinThreads) win_dkv_f32_kernel(const BwdArgs a) {
    extern __shared__ __align__(16) float win_mem[];
    constexpr int kCols = kWinChunk + 4;
    float* ps = win_mem;                              // [16][68] p
    float* ds = ps + kWinRows * kCols;                // [16][68] dS
    float* ks = ds + kWinRows * kCols;                // [16][D + 4]
    float* vs = ks + kWinRows * (D + 4);              // [16][D + 4]
    float* qs = vs + kWinRows * (D + 4);              // [64][D + 4]
    float* dos = qs + kWinChunk * (D + 4);            // [64][D + 4]
    const int tid = threadIdx.x;
    const int bh = blockIdx.y, j0 = blockIdx.x * kWinRows, N = a.N;
    const size_t head = (size_t)bh * N * D;
    const float* q = static_cast<const float*>(a.q) + head;
    const float* dout = static_cast<const float*>(a.dout) + head;
    const int jlast = min(j0 + kWinRows, N) - 1;
    // queries j0 .. i_end - 1: those of the last key's window, or all after a sink
    const int i_end = j0 < a.sinks || N - jlast <= a.window ? N : jlast + a.window;

    stage<D>(ks, static_cast<const float*>(a.k) + head, kWinRows, [&](int r) { return min(j0 + r, N - 1); });
    stage<D>(vs, static_cast<const float*>(a.v) + head, kWinRows, [&](int r) { return min(j0 + r, N - 1); });
    const int row = tid >> 4, c0 = (tid & 15) * (D / 16), j = j0 + row;
    float dk[D / 16], dv[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c) dk[c] = dv[c] = 0.f;
    for (int q0 = j0; q0 < i_end; q0 += kWinChunk) {
        const int nq = min(kWinChunk, i_end - q0);
        __syncthreads();
        stage<D>(qs, q, nq, [&](int r) { return q0 + r; });
        stage<D>(dos, dout, nq, [&](int r) { return q0 + r; });
        __syncthreads();
        const int qq = tid & 63, kg = tid >> 6, i = q0 + qq;
        float r[4], dp[4];
        dots<D>(r, ks + 4 * kg * (D + 4), qs + qq * (D + 4));
        dots<D>(dp, vs + 4 * kg * (D + 4), dos + qq * (D + 4));
        const float tau = a.tau[(size_t)bh * N + min(i, N - 1)], delta = a.delta[(size_t)bh * N + min(i, N - 1)];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int jj = j0 + 4 * kg + e;
            const bool in = i < i_end && jj < N && jj <= i && (i - jj < a.window || jj < a.sinks);
            const float u = in ? __fmul_rn(a.cx, r[e]) - tau : -1.f;
            const bool on = u > 0.f;
            ps[(4 * kg + e) * kCols + qq] = on ? entmax_p<GM>(u, a.gamma) : 0.f;
            ds[(4 * kg + e) * kCols + qq] = on ? entmax_g<GM>(u, a.gamma) * (dp[e] - delta) : 0.f;
        }
        __syncthreads();
        if (j >= N) continue;
        for (int r2 = 0; r2 < nq; ++r2) {
            const float p = ps[row * kCols + r2], s = ds[row * kCols + r2];
            if (p == 0.f && s == 0.f) continue;
            add_row<D>(dv, p, dos + r2 * (D + 4) + c0);
            add_row<D>(dk, s, qs + r2 * (D + 4) + c0);
        }
    }
    if (j < N) {
        store_row<D>(static_cast<float*>(a.dk) + head + (size_t)j * D + c0, dk, a.scale);
        store_row<D>(static_cast<float*>(a.dv) + head + (size_t)j * D + c0, dv, 1.f);
    }
    if (tid == 0 && j0 % kBlk == 0)   // S, dP, dV, dK of the blocks of a column, as many as of a row
        atomicAdd(&a.hdr->counters[kCtrBwdBlocks], 4ull * (unsigned long long)((i_end - j0 + kBlk - 1) / kBlk));
}

template <typename K>
cudaError_t grow_smem(K kern, size_t bytes) {
    return bytes > 48 * 1024 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes)
                             : cudaSuccess;
}

template <int D, int GM>
cudaError_t win_fwd(const FwdArgs& a, cudaStream_t s) {
    const int cols = win_cols(a.window, a.sinks);
    const size_t sm = win_smem<D>(cols, 1, 1);
    cudaError_t e = cudaMemsetAsync(a.mask, 0, (size_t)a.BH * a.T * a.T, s);
    if (e == cudaSuccess) e = grow_smem(win_fwd_f32_kernel<D, GM>, sm);
    if (e != cudaSuccess) return e;
    win_fwd_f32_kernel<D, GM><<<dim3((a.N + kWinRows - 1) / kWinRows, a.BH), kWinThreads, sm, s>>>(a, cols);
    return cudaGetLastError();
}

template <int D, int GM>
cudaError_t win_bwd(const BwdArgs& a, cudaStream_t s) {
    const int cols = win_cols(a.window, a.sinks);
    const dim3 grid((a.N + kWinRows - 1) / kWinRows, a.BH);
    size_t sm = win_smem<D>(cols, 2, 2);
    cudaError_t e = grow_smem(win_dq_f32_kernel<D, GM>, sm);
    if (e != cudaSuccess) return e;
    win_dq_f32_kernel<D, GM><<<grid, kWinThreads, sm, s>>>(a, cols);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    sm = win_smem<D>(kWinChunk + 4, 2, 2);
    if ((e = grow_smem(win_dkv_f32_kernel<D, GM>, sm)) != cudaSuccess) return e;
    win_dkv_f32_kernel<D, GM><<<grid, kWinThreads, sm, s>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t win_fwd_d(const FwdArgs& a, int gm, cudaStream_t s) {
    return gm == 1 ? win_fwd<D, 1>(a, s) : gm == 2 ? win_fwd<D, 2>(a, s) : gm == 4 ? win_fwd<D, 4>(a, s) : win_fwd<D, 0>(a, s);
}
template <int D>
cudaError_t win_bwd_d(const BwdArgs& a, int gm, cudaStream_t s) {
    return gm == 1 ? win_bwd<D, 1>(a, s) : gm == 2 ? win_bwd<D, 2>(a, s) : gm == 4 ? win_bwd<D, 4>(a, s) : win_bwd<D, 0>(a, s);
}

}  // namespace

// The backward's two score arrays are the larger need: both directions take this path, or
// neither (they share tau to the last bit of the scores).  On either side of the border, 8 heads
// of 2048, forward and backward: d = 64, 1392 keys 531 and 936 us, the general kernels at 1400
// keys 1891 and 1577; d = 128, 1072 keys 624 and 1474, 1080 keys 2815 and 2832; d = 32, 1584 keys
// 377 and 655, 1585 keys 1283 and 1403.  Smaller windows: d = 64, 1000 keys 307 and 840, 512 keys
// 177 and 593, 256 keys 111 and 386.
bool win_f32_fits(int window, int sinks, int d) {
    const int cols = win_cols(window, sinks);
    const size_t sm = d == 128 ? win_smem<128>(cols, 2, 2) : d == 64 ? win_smem<64>(cols, 2, 2) : win_smem<32>(cols, 2, 2);
    return sm <= 227 * 1024 - 1024;
}

cudaError_t win_fwd_f32(const FwdArgs& a, int d, int gm, cudaStream_t s) {
    return d == 128 ? win_fwd_d<128>(a, gm, s) : d == 64 ? win_fwd_d<64>(a, gm, s) : win_fwd_d<32>(a, gm, s);
}
cudaError_t win_bwd_f32(const BwdArgs& a, int d, int gm, cudaStream_t s) {
    return d == 128 ? win_bwd_d<128>(a, gm, s) : d == 64 ? win_bwd_d<64>(a, gm, s) : win_bwd_d<32>(a, gm, s);
}

}  // namespace ent
