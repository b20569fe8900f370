// units_check.cpp -- the division of a call of the paged prompt attention (units.cuh),
// whose sums have closed forms, against enumeration: units' tiles and costs, the place
// of a cost, and the ranges that the CTAs own.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "units.cuh"

using namespace kvattn;

#define CHECK(x)                                             \
    do {                                                     \
        if (!(x)) {                                          \
            printf("line %d: %s (case %d)\n", __LINE__, #x, it); \
            exit(1);                                         \
        }                                                    \
    } while (0)

namespace {

std::mt19937 rng(1);
int pick(int a, int b) { return a + (int)(rng() % (unsigned)(b - a + 1)); }

// Sequences: what their blocks cost, one after the other.
void sequences(int cases) {
    for (int it = 0; it < cases; ++it) {
        UnitSeq s;
        s.causal = pick(0, 1);
        s.len = pick(1, pick(1, 3000));
        s.shift = s.causal ? pick(0, pick(0, 5000)) : pick(1, 6000);
        s.window = s.causal && pick(0, 1) ? pick(1, pick(1, 7000)) : 1 << 25;
        s.tpu_lg = pick(0, 8);
        const int tpu = 1 << s.tpu_lg;
        s.piece = pick(0, 25);
        s.tpt = std::max(1, tpu >> pick(0, 1));
        s.w1 = pick(1, 5);
        s.w2 = s.w1 + pick(0, 2);
        const int nb = seq_blocks(s);
        CHECK(nb == (s.len + tpu - 1) / tpu);
        long long cost = 0;
        for (int b = 0; b < nb; ++b) {
            if (b < 40 || b > nb - 40 || pick(0, 9) == 0) {
                CHECK(blocks_cost(s, b) == cost);
                CHECK(block_at_cost(s, cost) == b);
            }
            const int tokens = std::min(tpu, s.len - b * tpu);
            int first = 1 << 30, last = 0;  // keys that some token of the block attends
            for (int t : {b * tpu, b * tpu + tokens - 1}) {
                const int end = s.shift + (s.causal ? t + 1 : 0);
                first = std::min(first, std::max(0, end - s.window));
                last = std::max(last, end);
            }
            const int tiles = (last + kUnitKeys - 1) / kUnitKeys - first / kUnitKeys;
            CHECK(tiles >= 1);
            CHECK(unit_first(s, b) == first / kUnitKeys);
            CHECK(unit_tiles(s, b) == tiles);
            CHECK(unit_weight(s, b) == (tokens > s.tpt ? s.w2 : s.w1));
            cost += unit_weight(s, b) * (long long)tiles + s.piece;
            if (pick(0, 9) == 0) CHECK(block_at_cost(s, cost - 1) == b);
        }
        CHECK(blocks_cost(s, nb) == cost);
    }
}

// Partitions: every tile has one CTA, every CTA a tile, a CTA at most the end of one
// unit and the start of another, and who starts a cut unit knows how many pieces it has.
void partitions(int cases) {
    for (int it = 0; it < cases; ++it) {
        const int piece = pick(0, 25), n = pick(1, 60);
        std::vector<int> nt(n), w(n), done(n, 0), pieces(n, 0), start(n, -1), said(n, 0);
        long long total = 0;
        for (int i = 0; i < n; ++i) {
            nt[i] = pick(0, 3) ? pick(1, 5) : pick(1, 200);
            w[i] = pick(4, 5);
            total += w[i] * nt[i] + piece;
        }
        const int grid = pick(1, 160), least = std::max(5 + piece, pick(1, 30));
        const int ranges = (int)std::max(1LL, std::min<long long>(total / least, grid));
        for (int c = 0; c < ranges; ++c) {
            const long long x0 = range_start(total, ranges, c), x1 = range_start(total, ranges, c + 1);
            CHECK(c + 1 < ranges || x1 == total);
            long long u = 0;
            int tiles = 0, units = 0;
            for (int i = 0; i < n; ++i) {
                const int ta = tiles_before(u, nt[i], w[i], piece, x0), tb = tiles_before(u, nt[i], w[i], piece, x1);
                if (ta < tb) {
                    CHECK(done[i] == ta);
                    done[i] = tb;
                    tiles += tb - ta;
                    ++pieces[i];
                    if (ta == 0 && tb < nt[i]) {
                        start[i] = c;
                        said[i] = range_of(total, ranges, u + piece + (long long)w[i] * (nt[i] - 1)) - c + 1;
                    }
                    if (ta > 0) {  // goes on with a cut unit: its first, and the next CTA's turn
                        CHECK(units == 0);
                        CHECK(start[i] >= 0 && c == start[i] + pieces[i] - 1);
                    }
                    ++units;
                }
                u += w[i] * nt[i] + piece;
            }
            CHECK(tiles > 0);
        }
        for (int i = 0; i < n; ++i) {
            CHECK(done[i] == nt[i]);
            CHECK(pieces[i] > 1 ? said[i] == pieces[i] : start[i] < 0);
        }
    }
}

void ranges(int cases) {
    for (int it = 0; it < cases; ++it) {
        // (totals in 32 bits and past them)
        const long long total = pick(0, 1) ? pick(1, 1000000) : (1LL << pick(31, 55)) + pick(0, 1 << 30);
        const int n = (int)std::min<long long>(pick(1, 3000), total);
        CHECK(range_start(total, n, 0) == 0 && range_start(total, n, n) == total);
        const int c = pick(0, n - 1);
        const long long a = range_start(total, n, c), z = range_start(total, n, c + 1);
        CHECK(a == (long long)((__int128)total * c / n) && a < z);
        CHECK(range_of(total, n, a) == c && range_of(total, n, z - 1) == c);
    }
}

}  // namespace

int main() {
    sequences(200000);
    partitions(20000);
    ranges(300000);
    puts("ok");
    return 0;
}
