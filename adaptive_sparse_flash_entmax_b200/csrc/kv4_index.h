// kv4_index.h -- where things lie in the paged 4-bit key/value cache, and which keys a
// query row sees.  Plain C++ shared by the kernels (kv4.cu) and a host program that the
// CPU tests compile, so that every index is checked without a GPU.
//
// The cache is four arrays (keys and values alike): codes [pages][heads][page][d/2]
// bytes and meta [pages][heads][page][d/32] pairs (scale, zero) of bfloat16, one pair for
// each 32 consecutive dimensions; a value is zero + scale * code.  The 4-byte word
// c * (d/32) + w of a token's codes, c = 0..3, holds dimension 32 w + 8 c + i in bits
// 4i .. 4i+3: lane c of a quad reads its words of all groups with one load, and they are
// its part of the A operand of a 16-row matrix instruction (kv4.cu).
#pragma once
#include <stddef.h>
#include <stdint.h>

#ifdef __CUDACC__
#define ENT_HD __host__ __device__ __forceinline__
#else
#define ENT_HD inline
#endif

namespace ent {

constexpr int kKvGroup = 32;   // dimensions that share a (scale, zero) pair
constexpr int kKvTile = 16;    // keys of one matrix instruction; a page holds a multiple of it
constexpr int kKvBadPage = 1;  // bits of the caller's `bad` word: a page number outside the pool,
constexpr int kKvBadLen = 2;   // a start or length outside what the call covers,
constexpr int kKvBadWait = 4;  // a bounded device wait that gave up (the rows it served are NaN)

struct Kv4Geom {
    int B, L;                // sequences, new tokens of each (rows of q, k, v)
    int pages, page_shift;   // pages of the pool, log2 of the tokens in one
    int max_pages;           // columns of the block table
    int max_len;             // tokens the call covers, <= max_pages << page_shift
    int window, sinks;       // window 0: every earlier key is visible
};

// What sequence b of a call holds: rows 0 .. rows-1 at positions start .. start+rows-1,
// keys 0 .. end-1.  A start or length outside the call's cover gives no rows, or as many
// as fit, and sets bad.
struct Kv4Seq {
    int start, rows, end, bad;
};

ENT_HD Kv4Seq kv4_seq(const Kv4Geom& g, int start, int new_len) {
    Kv4Seq s;
    s.bad = 0;
    if (start < 0 || start > g.max_len || new_len < 0) {
        s.start = s.rows = s.end = 0;
        s.bad = kKvBadLen;
        return s;
    }
    s.start = start;
    s.rows = new_len;
    if (s.rows > g.L) { s.rows = g.L; s.bad = kKvBadLen; }
    if (s.rows > g.max_len - start) { s.rows = g.max_len - start; s.bad = kKvBadLen; }
    s.end = start + s.rows;
    return s;
}

// The pool's page of position pos of a sequence whose row of the block table is `table`,
// or -1 (0 <= pos < max_len).
ENT_HD int kv4_page(const Kv4Geom& g, const int* table, int pos) {
    const int p = table[pos >> g.page_shift];
    return (p >= 0 && p < g.pages) ? p : -1;
}

// Row of position pos in the arrays of one head: element offsets are this times d/2 (codes,
// bytes) or d/32 (meta, pairs).
ENT_HD size_t kv4_row(const Kv4Geom& g, int heads, int page, int head, int pos) {
    return (((size_t)page * heads + head) << g.page_shift) + (pos & ((1 << g.page_shift) - 1));
}

ENT_HD int kv4_min(int a, int b) { return a < b ? a : b; }
ENT_HD int kv4_max(int a, int b) { return a > b ? a : b; }

// The keys that some row of a sequence can see are split into chunks of `C` (a multiple
// of kKvTile): without a window [0, end) from 0 on; with one first the sinks, [0, sinks
// rounded up to a tile), then from the first key of the first row's window (rounded down
// to a tile) on.  Chunks start on tile boundaries, so a tile lies in one page.
ENT_HD int kv4_sink_end(const Kv4Geom& g) {
    if (!g.window || !g.sinks) return 0;
    const int s = kv4_min(g.sinks, g.max_len);
    return s > g.max_len - kKvTile ? g.max_len : (s + kKvTile - 1) / kKvTile * kKvTile;
}
ENT_HD int kv4_sink_chunks(const Kv4Geom& g, int C) { return (kv4_sink_end(g) + C - 1) / C; }

// First key of the part after the sinks.
ENT_HD int kv4_base(const Kv4Geom& g, int start) {
    if (!g.window) return 0;
    const int first = start >= g.window ? (start - g.window + 1) / kKvTile * kKvTile : 0;
    // (a sink end that is no multiple of the tile is max_len, past every key)
    return kv4_max(first, kv4_sink_end(g));
}

// Chunks that a call needs for any start and length it covers, and those of one sequence.
ENT_HD int kv4_chunks(const Kv4Geom& g, int C) {
    long long rest = g.max_len;
    if (g.window) {
        const long long w = (long long)g.window + g.L + kKvTile;
        if (w < rest) rest = w;
    }
    return kv4_sink_chunks(g, C) + (int)((rest + C - 1) / C);
}
ENT_HD int kv4_seq_chunks(const Kv4Geom& g, const Kv4Seq& s, int C) {
    const int base = kv4_base(g, s.start);
    return kv4_sink_chunks(g, C) + (s.end > base ? (s.end - base + C - 1) / C : 0);
}

// Keys of a sequence's chunks: chunk c holds first(c) .. end(c) - 1 (none where first >= end,
// for chunks of sinks that the sequence does not reach).
struct Kv4Chunks {
    int C, ns, sink_end, base, seq_end;
    ENT_HD Kv4Chunks(const Kv4Geom& g, const Kv4Seq& s, int C_)
        : C(C_), ns(kv4_sink_chunks(g, C_)), sink_end(kv4_min(kv4_sink_end(g), s.end)),
          base(kv4_base(g, s.start) - ns * C_), seq_end(s.end) {}
    ENT_HD int first(int c) const { return c * C + (c < ns ? 0 : base); }
    ENT_HD int end(int c) const { return kv4_min(first(c) + C, c < ns ? sink_end : seq_end); }
};

// The chunks of a sequence are dealt to `nrun` runs of equal length: run i holds chunks
// [i * kv4_run, (i + 1) * kv4_run) below kv4_seq_chunks.
ENT_HD int kv4_run(int seq_chunks, int nrun) { return (seq_chunks + nrun - 1) / nrun; }

// Whether the row at position pos sees key j.
ENT_HD bool kv4_sees(const Kv4Geom& g, int pos, int j) {
    return j <= pos && (!g.window || pos - j < g.window || j < g.sinks);
}

}  // namespace ent
