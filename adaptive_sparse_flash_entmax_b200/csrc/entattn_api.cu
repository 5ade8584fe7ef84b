// entattn_api.cu -- the C ABI (include/entattn.h): argument validation,
// workspace layout, and dispatch to the kernels.  No exception crosses it.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <string>

#include "../../include/entattn.h"
#include "kernels.h"

namespace ent {

// A non-blocking stream per device for work forked from the caller's stream (created on
// first use, kept for the life of the process); null if it cannot be created.
cudaStream_t side_stream() {
    static cudaStream_t streams[64] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!streams[dev] && cudaStreamCreateWithFlags(&streams[dev], cudaStreamNonBlocking) != cudaSuccess)
        streams[dev] = nullptr;
    return streams[dev];
}

}  // namespace ent

namespace {

thread_local std::string g_err;

ent_status fail(ent_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    g_err = buf;
    return st;
}

ent_status cuda_fail(cudaError_t e, const char* where) {
    return fail(ENT_ECUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

constexpr size_t kHdr = sizeof(ent::WsHeader);

size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int n_tiles(int N) { return (N + ent::kBlk - 1) / ent::kBlk; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Exact integer gamma = 1/(alpha-1) in {1,2,3,4} gets a specialised kernel
// (alpha = 2, 1.5, 4/3, 1.25); any other alpha in (1, 2] uses exp2/log2.
int gamma_mode(float alpha, float* gamma_out) {
    const float gamma = 1.f / (alpha - 1.f);
    const float r = nearbyintf(gamma);
    if (r >= 1.f && r <= 4.f && fabsf(gamma - r) <= 1e-5f * r) {
        *gamma_out = r;
        return (int)r;
    }
    *gamma_out = gamma;
    return 0;
}

// Histogram insert budget of a bf16 forward tile (after its first block).  The
// default 0 starts every row from the plain bracket [m-1, m - n^(1-alpha)]: on B200
// the histogram's inserts and per-row bracket cost more than the ~2 solver passes
// they save, on every workload measured (the tiles then run ~4 cheap passes).
// ENTATTN_HIST_BUDGET selects the histogram start instead: a positive budget builds
// it until the tile has made that many inserts, a negative one always.
int hist_budget() {
    const char* v = getenv("ENTATTN_HIST_BUDGET");
    if (v && *v) return atoi(v);
    return 0;
}

// Forward workspace layout: the 256-byte header, then (bf16 path) the key-block bounds
// of the statistics pass: per head max |c| and min R (float bits), per 64-key
// half-block {R, L} and the bf16 centroid.
struct FwdLayout {
    size_t maxc, minr, stats, cent, fix, gap, calib, total;
};

FwdLayout fwd_layout(int B, int H, int N, int d) {
    const size_t BH = (size_t)B * H, T2 = 2 * (size_t)n_tiles(N);
    FwdLayout L;
    L.fix = kHdr;                        // failure list, one int per tile (zeroed with the header)
    L.maxc = L.fix + round_up(BH * T2 / 2 * 4, 256);   // [BH] words, then min R [BH]
    L.minr = L.maxc + BH * 4;
    L.stats = L.maxc + round_up(BH * 8, 256);
    L.cent = L.stats + round_up(BH * T2 * 8, 256);
    L.gap = L.cent + round_up(BH * T2 * (size_t)d * 2, 256);
    // calibrated start (sequences of >= kBoundMinBlocks query tiles): the sampled rows'
    // gaps and scores
    const bool cal = n_tiles(N) >= ent::kBoundMinBlocks;
    L.calib = L.gap + (cal ? round_up(BH * ent::kCalRows * 4, 256) : 0);
    L.total = L.calib + (cal ? round_up(BH * ent::kCalRows * (size_t)N * 4, 256) : 0);
    return L;
}

// Calibrated solver start (bf16 path, sequences of >= kBoundMinBlocks query tiles), on by
// default.  ENTATTN_CALIB=0 (environment, read per call) starts every row at the plain
// bracket's midpoint instead, for ablations; the outputs meet the same stop rule either way.
bool calib_enabled() {
    const char* v = getenv("ENTATTN_CALIB");
    return !(v && *v && atoi(v) == 0);
}

// Statistics-pass skipping by key-block bounds (bf16 path), on by default.
// ENTATTN_BOUND=0 (environment, read per call) turns it off, for ablations; the
// outputs are the same either way (a block it rules out holds no u > 0 and no row
// maximum, so every later pass sees the same blocks and sums).
bool bound_enabled() {
    const char* v = getenv("ENTATTN_BOUND");
    return !(v && *v && atoi(v) == 0);
}

// Unverified Halley steps of the bf16 forward (each checked in the P.V pass, see
// solver_update): steps up to 1e-2 either way whose boundary crossings can change f by
// at most 5e-5 upward (a bound on all leaving elements together, from the sums: half
// the check's 1e-4) or 3e-5 per entering element downward (at least four would have to
// enter within the step to miss the check).  ENTATTN_ACCEPT=0
// (environment, read per call) stops every row at an evaluated tau instead, for
// ablations.  ENTATTN_VERIFY_TOL sets the check's tolerance on |sum_j p - 1| (default
// 1e-4; a negative value makes every tile with such a row be solved again, which
// tests that path).
ent::AcceptRule accept_rule() {
    ent::AcceptRule r;
    const char* v = getenv("ENTATTN_ACCEPT");
    if (v && *v && atoi(v) == 0) return r;
    r.step = 1e-2f;
    r.cert_up = 5e-5f;
    r.cert_down = 3e-5f;
    return r;
}

// Speculative first job of each score pass in the bf16 forward (on by default);
// ENTATTN_SPEC=0 (environment, read per call) waits for each decision instead, for ablations.
int spec_enabled() {
    const char* v = getenv("ENTATTN_SPEC");
    return (v && *v && atoi(v) == 0) ? 0 : 1;
}

float verify_tol() {
    const char* v = getenv("ENTATTN_VERIFY_TOL");
    return (v && *v) ? (float)atof(v) : 1e-4f;
}

// Backward workspace layout: the 256-byte header, then delta (one float per query row).
struct BwdLayout {
    size_t delta, total;
};

BwdLayout bwd_layout(int B, int H, int N) {
    const size_t BH = (size_t)B * H;
    BwdLayout L;
    L.delta = kHdr;
    L.total = L.delta + round_up(BH * N * sizeof(float), 256);
    return L;
}

ent_status check_common(int B, int H, int N, int d, int dtype, float alpha, int causal) {
    if (B < 0 || H < 0 || N < 0) return fail(ENT_EINVAL, "negative size (B=%d H=%d N=%d)", B, H, N);
    if (dtype != ENT_F32 && dtype != ENT_BF16) return fail(ENT_EINVAL, "unknown dtype %d", dtype);
    if (!(alpha > 1.f && alpha <= 2.f)) return fail(ENT_EINVAL, "alpha=%g outside (1, 2]", (double)alpha);
    if (causal != 0 && causal != 1) return fail(ENT_EINVAL, "causal must be 0 or 1 (got %d)", causal);
    if (d != 32 && d != 64 && d != 128)
        return fail(ENT_EUNSUPPORTED, "head dim d=%d (supported: 32, 64, 128)", d);
    if ((long long)B * H > 65535) return fail(ENT_EUNSUPPORTED, "B*H=%lld exceeds 65535", (long long)B * H);
    if (N > 130944) return fail(ENT_EUNSUPPORTED, "N=%d exceeds 130944", N);
    return ENT_OK;
}

// Copies a workspace header (status word and counters) to the host after the
// work queued on `stream` is done.
ent_status read_header(const void* ws, long long* counters, void* stream) {
    ent::WsHeader h;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemcpyAsync(&h, ws, sizeof(h), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess) return cuda_fail(e, "reading the workspace header");
    if (counters)
        for (int i = 0; i < 8; ++i) counters[i] = (long long)h.counters[i];
    if (h.status != 0)
        return fail(ENT_ETIMEOUT, "a bounded device wait gave up (site %u)", h.timeout_site);
    return ENT_OK;
}

}  // namespace

extern "C" {

int ent_attn_block_size(void) { return ent::kBlk; }

size_t ent_attn_fwd_workspace_size(int B, int H, int N, int d, int dtype) {
    (void)dtype;
    if (B < 0 || H < 0 || N < 0 || d < 0) return 0;
    return fwd_layout(B, H, N, d).total;
}

size_t ent_attn_bwd_workspace_size(int B, int H, int N, int d, int dtype) {
    (void)dtype;
    if (B < 0 || H < 0 || N < 0 || d < 0) return 0;
    return bwd_layout(B, H, N).total;
}

const char* ent_attn_last_error(void) { return g_err.c_str(); }

}  // extern "C"

namespace {

// Support lists of ent_attn_fwd_lists / ent_attn_bwd_lists (all null otherwise).
struct Lists {
    int32_t* key = nullptr;
    float* u = nullptr;
    uint8_t* n = nullptr;
    bool want = false;
};

// Sliding window of the *_window calls (want false otherwise).
struct Window {
    int window = 0, sinks = 0;
    bool want = false;
};

ent_status check_window(const Window& w) {
    if (w.want && (w.window < 1 || w.sinks < 0))
        return fail(ENT_EINVAL, "window=%d must be at least 1 and sinks=%d at least 0", w.window, w.sinks);
    return ENT_OK;
}

// The window that a call's kernels work under.  A bfloat16 window as long as the sequence is
// causal attention, which has the bound pass and the calibrated start (8 heads of 32768 x 128:
// 8.9 ms a forward; 9.8 under the window).  A shorter one has neither, and passes that much of
// the keys by: 9.0 ms at 24000, 7.2 at 16384.  (float32 windows have kernels of their own, faster
// than the general ones at any length that they take.)
Window effective(const Window& w, int N, int dtype) {
    return w.want && w.window >= N && dtype == ENT_BF16 ? Window() : w;
}

// Backward workspace of ent_attn_bwd_lists: the plain layout, then the per-tile flags
// and the fp32 dK, dV accumulators of the list kernel.
struct ListLayout {
    size_t tiles, dk, dv, total;
};

ListLayout list_layout(int B, int H, int N, int d) {
    const size_t BH = (size_t)B * H;
    ListLayout L;
    L.tiles = bwd_layout(B, H, N).total;
    L.dk = L.tiles + round_up(BH * (size_t)n_tiles(N), 256);
    L.dv = L.dk + round_up(BH * N * (size_t)d * 4, 256);
    L.total = L.dv + round_up(BH * N * (size_t)d * 4, 256);
    return L;
}

// Forward of ent_attn_fwd and, with a non-null otilde, of ent_attn_fwd_otilde.
ent_status fwd_impl(const void* q, const void* k, const void* v, int B, int H, int N, int d,
                    int dtype, float alpha, int causal, void* o, float* tau, uint8_t* block_mask,
                    uint8_t* iters, float* otilde, bool want_otilde, void* ws, size_t ws_bytes,
                    void* stream, const Lists& lists = Lists(), const Window& asked = Window()) {
    ent_status st = check_common(B, H, N, d, dtype, alpha, causal);
    if (st == ENT_OK) st = check_window(asked);
    if (st != ENT_OK) return st;
    const Window win = effective(asked, N, dtype);
    if (lists.want && dtype != ENT_BF16)
        return fail(ENT_EUNSUPPORTED, "support lists are built by the bf16 forward only");
    if (!ws) return fail(ENT_EINVAL, "null workspace");
    if (ws_bytes < ent_attn_fwd_workspace_size(B, H, N, d, dtype))
        return fail(ENT_EINVAL, "workspace of %zu bytes is below the required %zu", ws_bytes,
                    ent_attn_fwd_workspace_size(B, H, N, d, dtype));
    if (!aligned16(ws)) return fail(ENT_EINVAL, "workspace pointer not 16-byte aligned");
    const bool empty = (long long)B * H == 0 || N == 0;
    if (!empty && (!q || !k || !v || !o || !tau || !block_mask))
        return fail(ENT_EINVAL, "null q/k/v/o/tau/block_mask pointer");
    if (!empty && (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)))
        return fail(ENT_EINVAL, "q/k/v/o must be 16-byte aligned");
    if (!empty && want_otilde && (!otilde || !aligned16(otilde)))
        return fail(ENT_EINVAL, "otilde must be a non-null 16-byte aligned pointer");
    if (!empty && lists.want && (!lists.key || !lists.u || !lists.n))
        return fail(ENT_EINVAL, "null list_key/list_u/list_n pointer");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const FwdLayout FL = fwd_layout(B, H, N, d);
    // (no tile of a shorter sequence runs the bound pass, so its statistics are not computed)
    // (nor under a window, whose tiles visit few blocks: there the histogram start, the bound
    // pass and the calibrated start are all off)
    const bool bound = dtype == ENT_BF16 && hist_budget() == 0 && bound_enabled() && !empty &&
                       !win.want && n_tiles(N) >= ent::kBoundMinBlocks;
    // header, failure list (entries are tile + 1, 0 until written) and the per-head max |c|
    // start at 0, the per-head min R at all ones
    cudaError_t e = cudaMemsetAsync(ws, 0, bound ? FL.minr : (dtype == ENT_BF16 ? FL.maxc : kHdr), s);
    if (e == cudaSuccess && bound) e = cudaMemsetAsync(static_cast<char*>(ws) + FL.minr, 0xFF, (size_t)B * H * 4, s);
    if (e != cudaSuccess) return cuda_fail(e, "clearing the workspace header");
    if (empty) return ENT_OK;

    ent::FwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.o = o; a.tau = tau; a.mask = block_mask; a.iters = iters;
    a.otilde = want_otilde ? otilde : nullptr;
    a.list_key = lists.key; a.list_u = lists.u; a.list_n = lists.n;
    a.hdr = static_cast<ent::WsHeader*>(ws);
    a.BH = B * H; a.N = N; a.T = n_tiles(N); a.causal = causal; a.dr = d;
    a.alpha = alpha;
    const int gm = gamma_mode(alpha, &a.gamma);
    a.scale = 1.f / sqrtf((float)d);
    a.cx = (alpha - 1.f) * a.scale;
    // Stop rule: bf16 outputs resolve ~4e-3 relative, so |sum p - 1| <= 1e-5 is
    // far below their rounding; float32 outputs get 1e-6.
    a.ftol = dtype == ENT_F32 ? 1e-6f : 1e-5f;
    a.stol = dtype == ENT_F32 ? 4e-7f : 1e-6f;
    a.hist_budget = win.want ? 0 : hist_budget();
    if (win.want) {   // (a window or sinks beyond the sequence are the sequence)
        a.window = win.window < N ? win.window : N;
        a.sinks = win.sinks < N ? win.sinks : N;
    }
    if (dtype == ENT_BF16) {
        a.acc = accept_rule();
        a.verify_tol = verify_tol();
        a.spec = spec_enabled();
        a.fail_list = reinterpret_cast<int*>(static_cast<char*>(ws) + FL.fix);
    }
    if (dtype == ENT_BF16 && hist_budget() == 0 && calib_enabled() && !win.want && n_tiles(N) >= ent::kBoundMinBlocks) {
        char* base = static_cast<char*>(ws);
        a.gap = reinterpret_cast<float*>(base + FL.gap);
        a.calib = reinterpret_cast<float*>(base + FL.calib);
    }
    if (bound) {
        // statistics-pass skipping by key-block bounds; off with the histogram start, whose
        // windows must count every score down to their lowest bin
        char* base = static_cast<char*>(ws);
        a.head_words = reinterpret_cast<unsigned int*>(base + FL.maxc);
        a.bstats = reinterpret_cast<float2*>(base + FL.stats);
        a.cent = base + FL.cent;
    }
    if (dtype == ENT_F32) {
        if (win.want && ent::win_f32_fits(a.window, a.sinks, d)) {
            // its passes are cheap and each row stops for itself: near the rounding of the sums (24
            // rows of large scores: O 0.42e-6 off instead of 1.05e-6; the step costs 0 to 1 %).  The
            // general kernels start nearer and stop at 0.9e-6, and 2e-7 sends some row of most
            // tiles to the pass cap (4 times the time).
            a.ftol = 4e-7f;
            a.stol = 2e-7f;
            e = ent::win_fwd_f32(a, d, gm, s);
        } else {
            e = ent::simt_fwd_f32(a, d, gm, s);
        }
    } else {
        const char* why = nullptr;
        e = ent::tc_fwd(a, d, gm, s, &why);
        if (e != cudaSuccess && why) return fail(ENT_ECUDA, "forward launch: %s", why);
    }
    if (e != cudaSuccess) return cuda_fail(e, "forward launch");
    return ENT_OK;
}

// Backward of ent_attn_bwd and, with a non-null otilde, of ent_attn_bwd_otilde.
ent_status bwd_impl(const void* q, const void* k, const void* v, const float* otilde,
                    bool want_otilde, const void* dout, const float* tau,
                    const uint8_t* block_mask, int B, int H, int N, int d, int dtype, float alpha,
                    int causal, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                    void* stream, const Lists& lists = Lists(), const Window& asked = Window()) {
    ent_status st = check_common(B, H, N, d, dtype, alpha, causal);
    if (st == ENT_OK) st = check_window(asked);
    if (st != ENT_OK) return st;
    const Window win = effective(asked, N, dtype);
    if (lists.want && dtype != ENT_BF16)
        return fail(ENT_EUNSUPPORTED, "support lists are built by the bf16 forward only");
    if (!ws) return fail(ENT_EINVAL, "null workspace");
    const BwdLayout L = bwd_layout(B, H, N);
    const ListLayout LL = list_layout(B, H, N, d);
    const size_t need = lists.want ? LL.total : L.total;
    if (ws_bytes < need)
        return fail(ENT_EINVAL, "workspace of %zu bytes is below the required %zu", ws_bytes, need);
    if (!aligned16(ws)) return fail(ENT_EINVAL, "workspace pointer not 16-byte aligned");
    const bool empty = (long long)B * H == 0 || N == 0;
    if (!empty && (!q || !k || !v || !dout || !tau || !block_mask || !dq || !dk || !dv))
        return fail(ENT_EINVAL, "null q/k/v/dout/tau/block_mask/dq/dk/dv pointer");
    if (!empty && (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dout) ||
                   !aligned16(dq) || !aligned16(dk) || !aligned16(dv)))
        return fail(ENT_EINVAL, "q/k/v/dout/dq/dk/dv must be 16-byte aligned");
    if (!empty && want_otilde && (!otilde || !aligned16(otilde)))
        return fail(ENT_EINVAL, "otilde must be a non-null 16-byte aligned pointer");
    if (!empty && lists.want && (!lists.key || !lists.u || !lists.n))
        return fail(ENT_EINVAL, "null list_key/list_u/list_n pointer");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemsetAsync(ws, 0, kHdr, s);
    if (e != cudaSuccess) return cuda_fail(e, "clearing the workspace header");
    if (empty) return ENT_OK;
    if (lists.want) {   // the list kernel's dK, dV accumulators start at zero
        e = cudaMemsetAsync(static_cast<char*>(ws) + LL.dk, 0, LL.total - LL.dk, s);
        if (e != cudaSuccess) return cuda_fail(e, "clearing the list accumulators");
    }

    ent::BwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.dout = dout; a.tau = tau; a.mask = block_mask;
    a.dq = dq; a.dk = dk; a.dv = dv;
    a.otilde = want_otilde ? otilde : nullptr;
    char* base = static_cast<char*>(ws);
    a.hdr = reinterpret_cast<ent::WsHeader*>(base);
    a.delta = reinterpret_cast<float*>(base + L.delta);
    a.BH = B * H; a.N = N; a.T = n_tiles(N); a.causal = causal; a.dr = d;
    a.alpha = alpha;
    const int gm = gamma_mode(alpha, &a.gamma);
    a.scale = 1.f / sqrtf((float)d);
    a.cx = (alpha - 1.f) * a.scale;
    if (win.want) {
        a.window = win.window < N ? win.window : N;
        a.sinks = win.sinks < N ? win.sinks : N;
        // every query sees one key, whose weight is 1 whatever its score: dQ and dK are zero, not
        // what rounding leaves of dP - delta (dV is as ever)
        if (a.window == 1 && a.sinks == 0) a.scale = 0.f;
    }
    if (lists.want) {
        a.list_key = lists.key; a.list_u = lists.u; a.list_n = lists.n;
        a.tile_list = reinterpret_cast<uint8_t*>(base + LL.tiles);
        a.dk_acc = reinterpret_cast<float*>(base + LL.dk);
        a.dv_acc = reinterpret_cast<float*>(base + LL.dv);
    }
    if (dtype == ENT_F32) {
        e = win.want && ent::win_f32_fits(a.window, a.sinks, d) ? ent::win_bwd_f32(a, d, gm, s)
                                                                : ent::simt_bwd_f32(a, d, gm, s);
    } else {
        const char* why = nullptr;
        if (lists.want) {
            // the list kernel and dq take disjoint query tiles (both decide from the list
            // counts) and run at the same time, the list kernel on a side stream forked
            // from `s`; dkv, which adds the list kernel's accumulators, joins it
            cudaStream_t side = ent::side_stream();
            cudaEvent_t fork = nullptr, join = nullptr;
            if (!side) side = s;   // no side stream: the two run one after the other
            e = cudaEventCreateWithFlags(&fork, cudaEventDisableTiming);
            if (e == cudaSuccess) e = cudaEventCreateWithFlags(&join, cudaEventDisableTiming);
            if (e == cudaSuccess) e = cudaEventRecord(fork, s);
            if (e == cudaSuccess) e = cudaStreamWaitEvent(side, fork, 0);
            if (e == cudaSuccess) e = ent::list_bwd(a, d, gm, side);
            if (e == cudaSuccess) e = cudaEventRecord(join, side);
            if (e == cudaSuccess) e = ent::tc_bwd(a, d, gm, s, &why, join);
            if (fork) cudaEventDestroy(fork);   // released once the recorded work is done
            if (join) cudaEventDestroy(join);
        } else {
            e = ent::tc_bwd(a, d, gm, s, &why);
        }
        if (e != cudaSuccess && why) return fail(ENT_ECUDA, "backward launch: %s", why);
    }
    if (e != cudaSuccess) return cuda_fail(e, "backward launch");
    return ENT_OK;
}

}  // namespace

extern "C" {

ent_status ent_attn_fwd(const void* q, const void* k, const void* v, int B, int H, int N, int d,
                        int dtype, float alpha, int causal, void* o, float* tau,
                        uint8_t* block_mask, uint8_t* iters, void* ws, size_t ws_bytes,
                        void* stream) {
    return fwd_impl(q, k, v, B, H, N, d, dtype, alpha, causal, o, tau, block_mask, iters, nullptr,
                    false, ws, ws_bytes, stream);
}

ent_status ent_attn_fwd_otilde(const void* q, const void* k, const void* v, int B, int H, int N,
                               int d, int dtype, float alpha, int causal, void* o, float* tau,
                               uint8_t* block_mask, uint8_t* iters, float* otilde, void* ws,
                               size_t ws_bytes, void* stream) {
    return fwd_impl(q, k, v, B, H, N, d, dtype, alpha, causal, o, tau, block_mask, iters, otilde,
                    true, ws, ws_bytes, stream);
}

ent_status ent_attn_bwd(const void* q, const void* k, const void* v, const void* o,
                        const void* dout, const float* tau, const uint8_t* block_mask, int B,
                        int H, int N, int d, int dtype, float alpha, int causal, void* dq,
                        void* dk, void* dv, void* ws, size_t ws_bytes, void* stream) {
    (void)o;
    return bwd_impl(q, k, v, nullptr, false, dout, tau, block_mask, B, H, N, d, dtype, alpha,
                    causal, dq, dk, dv, ws, ws_bytes, stream);
}

ent_status ent_attn_bwd_otilde(const void* q, const void* k, const void* v, const float* otilde,
                               const void* dout, const float* tau, const uint8_t* block_mask,
                               int B, int H, int N, int d, int dtype, float alpha, int causal,
                               void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                               void* stream) {
    return bwd_impl(q, k, v, otilde, true, dout, tau, block_mask, B, H, N, d, dtype, alpha, causal,
                    dq, dk, dv, ws, ws_bytes, stream);
}

ent_status ent_attn_fwd_window(const void* q, const void* k, const void* v, int B, int H, int N,
                               int d, int dtype, float alpha, int window, int sinks, void* o,
                               float* tau, uint8_t* block_mask, uint8_t* iters, float* otilde,
                               void* ws, size_t ws_bytes, void* stream) {
    Window w;
    w.window = window; w.sinks = sinks; w.want = true;
    return fwd_impl(q, k, v, B, H, N, d, dtype, alpha, 1, o, tau, block_mask, iters, otilde,
                    otilde != nullptr, ws, ws_bytes, stream, Lists(), w);
}

ent_status ent_attn_bwd_window(const void* q, const void* k, const void* v, const float* otilde,
                               const void* dout, const float* tau, const uint8_t* block_mask,
                               int B, int H, int N, int d, int dtype, float alpha, int window,
                               int sinks, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                               void* stream) {
    Window w;
    w.window = window; w.sinks = sinks; w.want = true;
    return bwd_impl(q, k, v, otilde, otilde != nullptr, dout, tau, block_mask, B, H, N, d, dtype,
                    alpha, 1, dq, dk, dv, ws, ws_bytes, stream, Lists(), w);
}

int ent_attn_list_cap(void) { return ent::kListCap; }

size_t ent_attn_bwd_lists_workspace_size(int B, int H, int N, int d, int dtype) {
    (void)dtype;
    if (B < 0 || H < 0 || N < 0 || d < 0) return 0;
    return list_layout(B, H, N, d).total;
}

ent_status ent_attn_fwd_lists(const void* q, const void* k, const void* v, int B, int H, int N,
                              int d, int dtype, float alpha, int causal, void* o, float* tau,
                              uint8_t* block_mask, uint8_t* iters, int32_t* list_key,
                              float* list_u, uint8_t* list_n, void* ws, size_t ws_bytes,
                              void* stream) {
    Lists l;
    l.key = list_key; l.u = list_u; l.n = list_n; l.want = true;
    return fwd_impl(q, k, v, B, H, N, d, dtype, alpha, causal, o, tau, block_mask, iters, nullptr,
                    false, ws, ws_bytes, stream, l);
}

ent_status ent_attn_bwd_lists(const void* q, const void* k, const void* v, const int32_t* list_key,
                              const float* list_u, const uint8_t* list_n, const void* dout,
                              const float* tau, const uint8_t* block_mask, int B, int H, int N,
                              int d, int dtype, float alpha, int causal, void* dq, void* dk,
                              void* dv, void* ws, size_t ws_bytes, void* stream) {
    Lists l;
    l.key = const_cast<int32_t*>(list_key); l.u = const_cast<float*>(list_u);
    l.n = const_cast<uint8_t*>(list_n); l.want = true;
    return bwd_impl(q, k, v, nullptr, false, dout, tau, block_mask, B, H, N, d, dtype, alpha,
                    causal, dq, dk, dv, ws, ws_bytes, stream, l);
}

int ent_entmax_rows_max_n(void) { return 16384; }

}  // extern "C"

namespace {

static_assert(ENT_SOLVE_HIST == ent::kSolveHist && ENT_SOLVE_HALLEY == ent::kSolveHalley &&
                  ENT_SOLVE_BISECT == ent::kSolveBisect,
              "solver codes of the header and the kernels agree");

ent_status check_rows(int rows, int n, int dtype, float alpha) {
    if (rows < 0 || n < 0) return fail(ENT_EINVAL, "negative size (rows=%d n=%d)", rows, n);
    if (dtype != ENT_F32 && dtype != ENT_BF16) return fail(ENT_EINVAL, "unknown dtype %d", dtype);
    if (!(alpha > 1.f && alpha <= 2.f)) return fail(ENT_EINVAL, "alpha=%g outside (1, 2]", (double)alpha);
    if (n > ent_entmax_rows_max_n())
        return fail(ENT_EUNSUPPORTED, "n=%d exceeds %d", n, ent_entmax_rows_max_n());
    return ENT_OK;
}

ent::RowArgs row_args(int rows, int n, int dtype, float alpha) {
    ent::RowArgs a{};
    a.rows = rows; a.n = n; a.alpha = alpha;
    a.cx = alpha - 1.f;
    a.ftol = dtype == ENT_F32 ? 1e-6f : 1e-5f;
    a.stol = dtype == ENT_F32 ? 4e-7f : 1e-6f;
    return a;
}

}  // namespace

extern "C" {

ent_status ent_entmax_rows_fwd(const void* z, int rows, int n, int dtype, float alpha, int method,
                               void* p, float* tau, uint8_t* iters, void* stream) {
    ent_status st = check_rows(rows, n, dtype, alpha);
    if (st != ENT_OK) return st;
    if (method != ENT_SOLVE_HIST && method != ENT_SOLVE_HALLEY && method != ENT_SOLVE_BISECT)
        return fail(ENT_EINVAL, "unknown method %d", method);
    if (rows == 0 || n == 0) return ENT_OK;
    if (!z || !p || !tau) return fail(ENT_EINVAL, "null z/p/tau pointer");
    ent::RowArgs a = row_args(rows, n, dtype, alpha);
    a.z = z; a.p = p; a.tau = tau; a.iters = iters; a.method = method;
    const int gm = gamma_mode(alpha, &a.gamma);
    cudaError_t e = ent::rows_entmax(a, dtype == ENT_BF16, gm, false, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "row entmax launch");
    return ENT_OK;
}

ent_status ent_entmax_rows_bwd(const void* z, const float* tau, const void* dp, int rows, int n,
                               int dtype, float alpha, void* dz, void* stream) {
    ent_status st = check_rows(rows, n, dtype, alpha);
    if (st != ENT_OK) return st;
    if (rows == 0 || n == 0) return ENT_OK;
    if (!z || !tau || !dp || !dz) return fail(ENT_EINVAL, "null z/tau/dp/dz pointer");
    ent::RowArgs a = row_args(rows, n, dtype, alpha);
    a.z = z; a.tau_in = tau; a.dp = dp; a.dz = dz;
    const int gm = gamma_mode(alpha, &a.gamma);
    cudaError_t e = ent::rows_entmax(a, dtype == ENT_BF16, gm, true, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "row entmax backward launch");
    return ENT_OK;
}

ent_status ent_attn_read_status(const void* ws, long long* counters, void* stream) {
    if (!ws) return fail(ENT_EINVAL, "null workspace");
    return read_header(ws, counters, stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Backward with library-owned scratch (no workspace argument).
//
// Some callers cannot call cudaMalloc at the point where they run the
// backward: serving and training stacks that plan all device memory up front
// and treat any later allocation as an error (a cudaMalloc may synchronise the
// device and fragments a pre-sized pool), and plain-C callers with no device
// allocator of their own.  For them the backward's scratch (a 256-byte status
// and counter header plus delta, one float per query row) lives in the
// fixed-size array below, compiled into the library.  Every GPU that loads the
// library holds this array until the process exits.
namespace {

constexpr size_t kFixedScratchBytes = size_t(4) << 20;   // 4 MiB: header + 1,048,512 rows of delta
constexpr int kMaxScratchDevices = 64;

static __device__ __align__(256) unsigned char g_fixed_scratch[kFixedScratchBytes];

std::mutex g_fixed_scratch_mu;
void* g_fixed_scratch_addr[kMaxScratchDevices] = {};

// Device address of g_fixed_scratch on the current device.  The first call on
// a device looks it up with cudaGetSymbolAddress (the host-side name is only a
// stand-in, never a device address) and caches it.
cudaError_t fixed_scratch_address(void** out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxScratchDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_fixed_scratch_mu);
    if (!g_fixed_scratch_addr[dev]) {
        void* p = nullptr;
        e = cudaGetSymbolAddress(&p, g_fixed_scratch);
        if (e != cudaSuccess) return e;
        g_fixed_scratch_addr[dev] = p;
    }
    *out = g_fixed_scratch_addr[dev];
    return cudaSuccess;
}

}  // namespace

extern "C" ent_status ent_attn_bwd_noalloc(const void* q, const void* k, const void* v,
                                           const void* o, const void* dout, const float* tau,
                                           const uint8_t* block_mask, int B, int H, int N, int d,
                                           int dtype, float alpha, int causal, void* dq, void* dk,
                                           void* dv, void* stream) {
    (void)o;
    ent_status st = check_common(B, H, N, d, dtype, alpha, causal);
    if (st != ENT_OK) return st;
    const bool empty = (long long)B * H == 0 || N == 0;
    const size_t need = kHdr + round_up((size_t)B * H * N * sizeof(float), 256);
    if (need > kFixedScratchBytes)
        return fail(ENT_EUNSUPPORTED,
                    "ent_attn_bwd_noalloc: B*H*N = %lld rows exceed the %zu rows its fixed "
                    "scratch holds; use ent_attn_bwd with a workspace",
                    (long long)B * H * N, (kFixedScratchBytes - kHdr) / sizeof(float));
    if (!empty && (!q || !k || !v || !dout || !tau || !block_mask || !dq || !dk || !dv))
        return fail(ENT_EINVAL, "null q/k/v/dout/tau/block_mask/dq/dk/dv pointer");
    if (!empty && (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dout) ||
                   !aligned16(dq) || !aligned16(dk) || !aligned16(dv)))
        return fail(ENT_EINVAL, "q/k/v/dout/dq/dk/dv must be 16-byte aligned");
    void* base = nullptr;
    cudaError_t e = fixed_scratch_address(&base);
    if (e != cudaSuccess) return cuda_fail(e, "looking up the fixed scratch address");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // The scratch keeps the previous call's contents: the header (status and
    // counters) must start at zero; delta is fully rewritten before it is read.
    e = cudaMemsetAsync(base, 0, kHdr, s);
    if (e != cudaSuccess) return cuda_fail(e, "clearing the fixed scratch header");
    if (empty) return ENT_OK;

    ent::BwdArgs a{};
    a.q = q; a.k = k; a.v = v; a.dout = dout; a.tau = tau; a.mask = block_mask;
    a.dq = dq; a.dk = dk; a.dv = dv;
    a.otilde = nullptr;
    char* b = static_cast<char*>(base);
    a.hdr = reinterpret_cast<ent::WsHeader*>(b);
    a.delta = reinterpret_cast<float*>(b + kHdr);
    a.BH = B * H; a.N = N; a.T = n_tiles(N); a.causal = causal; a.dr = d;
    a.alpha = alpha;
    const int gm = gamma_mode(alpha, &a.gamma);
    a.scale = 1.f / sqrtf((float)d);
    a.cx = (alpha - 1.f) * a.scale;
    if (dtype == ENT_F32) {
        e = ent::simt_bwd_f32(a, d, gm, s);
    } else {
        const char* why = nullptr;
        e = ent::tc_bwd(a, d, gm, s, &why);
        if (e != cudaSuccess && why) return fail(ENT_ECUDA, "backward launch: %s", why);
    }
    if (e != cudaSuccess) return cuda_fail(e, "backward launch");
    return ENT_OK;
}

extern "C" ent_status ent_attn_noalloc_read_status(long long* counters, void* stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
    void* base = nullptr;
    {
        std::lock_guard<std::mutex> lock(g_fixed_scratch_mu);
        if (dev >= 0 && dev < kMaxScratchDevices) base = g_fixed_scratch_addr[dev];
    }
    if (!base)
        return fail(ENT_EINVAL,
                    "ent_attn_noalloc_read_status: no ent_attn_bwd_noalloc call on device %d yet", dev);
    return read_header(base, counters, stream);
}

// ---------------------------------------------------------------- 4-bit cache
namespace {

// Sizes of a call; `cover` the tokens its block table names or its max_len bounds.
ent_status check_kv4_sizes(int B, int Hkv, int L, int d, int dtype, long long cover) {
    if (B < 0 || Hkv < 1 || L < 0) return fail(ENT_EINVAL, "bad size (B=%d Hkv=%d L=%d)", B, Hkv, L);
    if (dtype != ENT_F32 && dtype != ENT_BF16) return fail(ENT_EINVAL, "unknown dtype %d", dtype);
    if (d != 32 && d != 64 && d != 128)
        return fail(ENT_EUNSUPPORTED, "head dim d=%d (supported: 32, 64, 128)", d);
    if ((long long)B * Hkv > 65535) return fail(ENT_EUNSUPPORTED, "B*Hkv=%lld exceeds 65535", (long long)B * Hkv);
    if (cover > 1ll << 30)   // positions and chunk ends stay clear of 31 bits
        return fail(ENT_EUNSUPPORTED, "%lld tokens a sequence exceed 2^30", cover);
    if ((long long)B * Hkv * L > 0x7fffffffll) return fail(ENT_EUNSUPPORTED, "B*Hkv*L exceeds 31 bits");
    return ENT_OK;
}

// Pool, block table and row counts of a call; fills a.g, a.Hkv, a.table, a.start, a.new_lens.
ent_status check_kv4(ent::Kv4Args& a, const void* kc, const void* km, const void* vc, const void* vm,
                     int pages, int page, const int32_t* table, int max_pages, const int32_t* start,
                     const int32_t* new_lens, int B, int Hkv, int L, int d, int dtype, int32_t* bad) {
    if (page < ent::kKvTile || (page & (page - 1)) != 0)
        return fail(ENT_EINVAL, "page of %d tokens (a power of two of at least %d)", page, ent::kKvTile);
    if (max_pages < 0) return fail(ENT_EINVAL, "negative size (max_pages=%d)", max_pages);
    const ent_status st = check_kv4_sizes(B, Hkv, L, d, dtype, (long long)max_pages * page);
    if (st != ENT_OK) return st;
    if (B > 0 && L > 0) {
        if ((!table && max_pages > 0) || !start) return fail(ENT_EINVAL, "null block_table/start pointer");
        if (pages < 1) return fail(ENT_EINVAL, "a pool without pages");
        if (!kc || !km || !vc || !vm) return fail(ENT_EINVAL, "null cache pointer");
        if (!aligned16(kc) || !aligned16(km) || !aligned16(vc) || !aligned16(vm))
            return fail(ENT_EINVAL, "cache arrays must be 16-byte aligned");
    }
    a.g.B = B; a.g.L = L; a.g.pages = pages; a.g.max_pages = max_pages;
    a.g.max_len = max_pages * page;
    while ((1 << a.g.page_shift) < page) ++a.g.page_shift;
    a.Hkv = Hkv;
    a.group = 1;
    a.table = table; a.start = start; a.new_lens = new_lens; a.bad = bad;
    a.k_codes = static_cast<uint8_t*>(const_cast<void*>(kc));
    a.v_codes = static_cast<uint8_t*>(const_cast<void*>(vc));
    a.k_meta = const_cast<void*>(km);
    a.v_meta = const_cast<void*>(vm);
    return ENT_OK;
}

// Workspace of the attention: per row and run of chunks its maximum and its count, then the
// candidates (score and key).  The rows of one key head share a scores warp, 4, 8, 16 or 32
// of them (the product is 8 queries wide; a warp of 4 holds two groups of dimensions in it and
// looks its scores through with twice the lanes a row; float32 rows at d = 128 take two parts
// each and stay at 16).
struct Kv4Layout {
    int block, blocks, chunk, nchunk, nrun;
    size_t n, cand, total;
};

bool kv4_layout(const ent::Kv4Geom& g, long long rows, int group, int d, int dtype, Kv4Layout* l) {
    const long long per = (long long)g.L * group;
    l->block = per <= 4 ? 4 : per <= 8 ? 8 : per <= 16 || (dtype == ENT_F32 && d == 128) ? 16 : 32;
    if (per > 65535ll * l->block || rows > 0x7fffffffll) return false;
    l->blocks = (int)((per + l->block - 1) / l->block);
    l->chunk = ent::kv4_chunk_keys(l->block);
    l->nchunk = ent::kv4_chunks(g, l->chunk);
    // runs: a warp each, enough of them for two rounds of 16 on each SM and no more (a longer
    // run pays its prologue once, and a higher maximum filters its later chunks).  16 are resident
    // where four rows share a warp; 12 or 8 for more rows, which so take up to four rounds.  Two
    // rounds of those measured better and worse: eight rows of 32 / 8 heads, 4 x 8192, 51 us
    // instead of 61, in float32 59 instead of 67, but 16 x 16384 in float32 330 instead of 300.
    const long long items = per > 0 ? rows / per * l->blocks : 0;
    long long want = items > 0 ? (2 * 16 * 148 + items - 1) / items : 1;
    if (want > ent::kKvMaxRuns) want = ent::kKvMaxRuns;
    l->nrun = (int)(want < l->nchunk ? want : l->nchunk);
    const size_t runs = (size_t)rows * l->nrun * 4;
    l->n = round_up(runs, 256);
    l->cand = l->n + round_up(runs, 256);
    l->total = l->cand + round_up((size_t)rows * l->nchunk * l->chunk * 8, 256);
    return true;
}

// Sizes of the attention alone; also its workspace's layout.
ent_status check_kv4_attn(ent::Kv4Geom& g, int Hq, int Hkv, int max_len, int window, int sinks, int d, int dtype,
                          Kv4Layout* l) {
    if (Hq < 1 || Hq % Hkv != 0) return fail(ENT_EINVAL, "Hq=%d is no multiple of Hkv=%d", Hq, Hkv);
    if (window < 0 || sinks < 0) return fail(ENT_EINVAL, "negative window=%d or sinks=%d", window, sinks);
    if (sinks > 0 && window == 0) return fail(ENT_EINVAL, "sinks=%d without a window", sinks);
    if (max_len < 0) return fail(ENT_EINVAL, "negative max_len=%d", max_len);
    g.max_len = max_len;
    g.window = window;
    g.sinks = sinks;
    if (!kv4_layout(g, (long long)g.B * Hq * g.L, Hq / Hkv, d, dtype, l))
        return fail(ENT_EUNSUPPORTED, "B*Hq*L=%lld rows, %lld of one key head, are too many",
                    (long long)g.B * Hq * g.L, (long long)g.L * (Hq / Hkv));
    return ENT_OK;
}

}  // namespace

extern "C" {

ent_status ent_attn_kv4_write(const void* k, const void* v, int B, int Hkv, int L, int d, int dtype,
                              const int32_t* block_table, int max_pages, const int32_t* start,
                              const int32_t* new_lens, void* k_codes, void* k_meta, void* v_codes,
                              void* v_meta, int pages, int page, int32_t* bad, void* stream) {
    ent::Kv4Args a{};
    ent_status st = check_kv4(a, k_codes, k_meta, v_codes, v_meta, pages, page, block_table, max_pages,
                              start, new_lens, B, Hkv, L, d, dtype, bad);
    if (st != ENT_OK) return st;
    if (B == 0 || L == 0) return ENT_OK;
    if (!k || !v) return fail(ENT_EINVAL, "null k/v pointer");
    if (!aligned16(k) || !aligned16(v)) return fail(ENT_EINVAL, "k/v must be 16-byte aligned");
    a.k = k; a.v = v;
    cudaError_t e = ent::kv4_write(a, d, dtype == ENT_BF16, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ENT_OK : cuda_fail(e, "cache write launch");
}

ent_status ent_attn_kv4_read(const void* k_codes, const void* k_meta, const void* v_codes,
                             const void* v_meta, int pages, int page, const int32_t* block_table,
                             int max_pages, const int32_t* start, const int32_t* new_lens, int B,
                             int Hkv, int L, int d, int dtype, void* k, void* v, int32_t* bad,
                             void* stream) {
    ent::Kv4Args a{};
    ent_status st = check_kv4(a, k_codes, k_meta, v_codes, v_meta, pages, page, block_table, max_pages,
                              start, new_lens, B, Hkv, L, d, dtype, bad);
    if (st != ENT_OK) return st;
    if (B == 0 || L == 0) return ENT_OK;
    if (!k || !v) return fail(ENT_EINVAL, "null k/v pointer");
    if (!aligned16(k) || !aligned16(v)) return fail(ENT_EINVAL, "k/v must be 16-byte aligned");
    a.k_out = k; a.v_out = v;
    cudaError_t e = ent::kv4_read(a, d, dtype == ENT_BF16, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ENT_OK : cuda_fail(e, "cache read launch");
}

size_t ent_attn_kv4_workspace_size(int B, int Hq, int Hkv, int L, int d, int dtype, int max_len,
                                   int window, int sinks) {
    ent::Kv4Geom g{};
    g.B = B; g.L = L;
    Kv4Layout l;
    const bool fine = check_kv4_sizes(B, Hkv, L, d, dtype, max_len) == ENT_OK &&
                      check_kv4_attn(g, Hq, Hkv, max_len, window, sinks, d, dtype, &l) == ENT_OK;
    return fine ? l.total : 0;
}

ent_status ent_attn_kv4_fwd(const void* q, int B, int Hq, int Hkv, int L, int d, int dtype,
                            float alpha, int window, int sinks, const void* k_codes,
                            const void* k_meta, const void* v_codes, const void* v_meta, int pages,
                            int page, const int32_t* block_table, int max_pages,
                            const int32_t* start, const int32_t* new_lens, int max_len, void* o,
                            float* tau, int32_t* bad, void* ws, size_t ws_bytes, void* stream) {
    ent::Kv4Args a{};
    ent_status st = check_kv4(a, k_codes, k_meta, v_codes, v_meta, pages, page, block_table, max_pages,
                              start, new_lens, B, Hkv, L, d, dtype, bad);
    if (st != ENT_OK) return st;
    if (!(alpha > 1.f && alpha <= 2.f)) return fail(ENT_EINVAL, "alpha=%g outside (1, 2]", (double)alpha);
    if (max_len > a.g.max_len)
        return fail(ENT_EINVAL, "max_len=%d exceeds max_pages * page = %d", max_len, a.g.max_len);
    Kv4Layout l;
    if ((st = check_kv4_attn(a.g, Hq, Hkv, max_len, window, sinks, d, dtype, &l)) != ENT_OK) return st;
    a.group = Hq / Hkv;
    if (B == 0 || L == 0) return ENT_OK;
    if (!q || !o) return fail(ENT_EINVAL, "null q/o pointer");
    if (!aligned16(q) || !aligned16(o)) return fail(ENT_EINVAL, "q/o must be 16-byte aligned");
    if (l.total > 0 && !ws) return fail(ENT_EINVAL, "null workspace");
    if (ws_bytes < l.total)
        return fail(ENT_EINVAL, "workspace of %zu bytes is below the required %zu", ws_bytes, l.total);
    if (!aligned16(ws)) return fail(ENT_EINVAL, "workspace pointer not 16-byte aligned");
    a.q = q; a.o = o; a.tau = tau;
    a.alpha = alpha;
    const int gm = gamma_mode(alpha, &a.gamma);
    a.cx = (alpha - 1.f) / sqrtf((float)d);
    a.block = l.block; a.blocks = l.blocks; a.chunk = l.chunk; a.nchunk = l.nchunk; a.nrun = l.nrun;
    char* base = static_cast<char*>(ws);
    a.run_max = reinterpret_cast<float*>(base);
    a.run_n = reinterpret_cast<int*>(base + l.n);
    a.cand = reinterpret_cast<int2*>(base + l.cand);
    cudaError_t e = ent::kv4_attn(a, d, dtype == ENT_BF16, gm, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ENT_OK : cuda_fail(e, "cache attention launch");
}

}  // extern "C"
