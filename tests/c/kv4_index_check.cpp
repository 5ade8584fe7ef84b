// Brute-force check of the cache's index arithmetic (csrc/kv4_index.h) on the CPU: every
// chunk of every sequence lies in the cover and on tile boundaries, each key that a row
// sees is in exactly one chunk, chunk counts are enough, pages outside the pool are never
// followed, and rows of the arrays never meet or leave the pool.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "kv4_index.h"

using namespace ent;

#define CHECK(x)                                                                       \
    do {                                                                               \
        if (!(x)) {                                                                    \
            std::printf("failed: %s (line %d)\n", #x, __LINE__);                       \
            return 1;                                                                  \
        }                                                                              \
    } while (0)

int main() {
    long long cases = 0;
    for (int C : {16, 32, 256})
        for (int max_len : {0, 1, 15, 16, 17, 40, 129, 300})
            for (int window : {0, 1, 2, 16, 17, 50, 1000})
                for (int sinks : {0, 1, 15, 16, 20, 130, 500}) {
                    if (sinks && !window) continue;
                    for (int L : {1, 2, 5, 40})
                        for (int start = -2; start <= max_len + 2; start += (max_len > 50 ? 7 : 1))
                            for (int nl : {-1, 0, 1, 3, L, L + 1}) {
                                Kv4Geom g{1, L, 4, 4, (max_len + 15) / 16, max_len, window, sinks};
                                const Kv4Seq s = kv4_seq(g, start, nl);
                                ++cases;
                                CHECK(s.rows >= 0 && s.rows <= L && s.start >= 0 && s.end <= max_len);
                                CHECK(s.end == s.start + s.rows);
                                const bool fine = start >= 0 && nl >= 0 && nl <= L && start + nl <= max_len;
                                CHECK((s.bad == 0) == fine);
                                if (fine) CHECK(s.start == start && s.rows == nl);
                                if (s.rows == 0) continue;   // no row reads a chunk
                                const int n = kv4_seq_chunks(g, s, C);
                                CHECK(n <= kv4_chunks(g, C));
                                std::vector<int> hits(max_len, 0);
                                for (int c = 0; c < n; ++c) {
                                    const int k0 = Kv4Chunks(g, s, C).first(c), k1 = Kv4Chunks(g, s, C).end(c);
                                    if (k0 >= k1) continue;
                                    CHECK(k0 >= 0 && k1 <= s.end && k1 - k0 <= C && k0 % kKvTile == 0);
                                    for (int j = k0; j < k1; ++j) ++hits[j];
                                }
                                for (int j = 0; j < max_len; ++j) {
                                    bool seen = false;
                                    for (int l = 0; l < s.rows; ++l) seen |= kv4_sees(g, s.start + l, j);
                                    CHECK(hits[j] <= 1);
                                    if (seen) CHECK(hits[j] == 1);
                                }
                            }
                }
    // pages and rows
    for (int shift : {4, 5, 7})
        for (int heads : {1, 3}) {
            const int pages = 5;
            Kv4Geom g{1, 1, pages, shift, 4, 4 << shift, 0, 0};
            const int table[4] = {4, -1, 5, 0};
            CHECK(kv4_page(g, table, 0) == 4 && kv4_page(g, table, (1 << shift) - 1) == 4);
            CHECK(kv4_page(g, table, 1 << shift) == -1 && kv4_page(g, table, 2 << shift) == -1);
            CHECK(kv4_page(g, table, (4 << shift) - 1) == 0);
            std::vector<int> hits((size_t)pages * heads << shift, 0);
            for (int p = 0; p < pages; ++p)
                for (int h = 0; h < heads; ++h)
                    for (int pos = 0; pos < (1 << shift); ++pos) {
                        const size_t r = kv4_row(g, heads, p, h, (3 << shift) + pos);
                        CHECK(r < hits.size());
                        ++hits[r];
                    }
            for (int x : hits) CHECK(x == 1);
            // far pages: past 32 bits of elements
            Kv4Geom far{1, 1, 2000000000, 20, 1, 1 << 20, 0, 0};
            CHECK(kv4_row(far, 8, 1999999999, 7, 5) == ((1999999999ull * 8 + 7) << 20) + 5);
        }
    // runs: every chunk in one, and no more runs than there are places
    for (int n : {1, 2, 3, 7, 64, 1000, 16384})
        for (int nrun : {1, 2, 3, 37, 1024}) {
            const int run = kv4_run(n, nrun);
            CHECK(run >= 1 && (long long)run * nrun >= n && (n + run - 1) / run <= nrun);
        }
    // the largest cover
    for (int window : {0, 1, 1 << 30, 2147483647}) {
        Kv4Geom g{1, 3, 1, 4, 1 << 26, 1 << 30, window, window ? 2147483647 : 0};
        const Kv4Seq s = kv4_seq(g, (1 << 30) - 3, 3);
        CHECK(s.rows == 3 && s.end == 1 << 30);
        const int n = kv4_seq_chunks(g, s, 512);
        CHECK(n > 0 && n <= kv4_chunks(g, 512));
        const int k0 = Kv4Chunks(g, s, 512).first(n - 1), k1 = Kv4Chunks(g, s, 512).end(n - 1);
        CHECK(k0 >= 0 && k0 < k1 && k1 <= s.end);
    }
    std::printf("kv4 index ok (%lld sequences)\n", cases);
    return 0;
}
