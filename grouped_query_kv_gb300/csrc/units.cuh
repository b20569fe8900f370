// units.cuh -- how the paged prompt attention divides a call: key tiles of all
// units (a block of a sequence's tokens, one head group), in the order (sequence,
// head group, block of tokens), cut into equal ranges of cost, a CTA each.  A
// unit of nt key tiles costs w nt + piece, the latter at its first tile: tile 0
// starts at the unit's start u, tile t > 0 at u + piece + w t, and a CTA owns the
// tiles that start in its range.  w is less for a unit with one query tile of two.  Everything follows from the lengths
// in a few operations, so that a CTA finds its place without a list.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define KVATTN_HD __host__ __device__ __forceinline__
#else
#define KVATTN_HD inline
#endif

namespace kvattn {

constexpr int kUnitKeys = 128, kUnitLg = 7;  // keys of a tile

// One sequence of a call: token t (of `len`) attends the positions
// [max(0, e - window), e), e = shift + (causal ? t + 1 : 0).
struct UnitSeq {
    int len, shift, causal, window;
    int tpu_lg;  // log2 of the tokens of a unit, up to 8
    int tpt;     // tokens of a query tile
    int w1, w2;  // cost of a key tile of a unit with up to tpt tokens, and with more
    int piece;   // cost of a unit's start and end
};

KVATTN_HD int seq_blocks(const UnitSeq &s) { return (s.len + (1 << s.tpu_lg) - 1) >> s.tpu_lg; }
KVATTN_HD int seq_end(const UnitSeq &s, int t) { return s.shift + (s.causal ? t + 1 : 0); }

// First key tile of a block of tokens, and how many there are.
KVATTN_HD int unit_first(const UnitSeq &s, int blk) {
    const int lo = seq_end(s, blk << s.tpu_lg) - s.window;
    return lo > 0 ? lo >> kUnitLg : 0;
}
KVATTN_HD int unit_tiles(const UnitSeq &s, int blk) {
    const long long past = (long long)(blk + 1) << s.tpu_lg;
    const int last = (int)(past < s.len ? past : s.len) - 1;
    return ((seq_end(s, last) + kUnitKeys - 1) >> kUnitLg) - unit_first(s, blk);
}

KVATTN_HD int unit_weight(const UnitSeq &s, int blk) {
    const int left = s.len - (blk << s.tpu_lg), all = 1 << s.tpu_lg;
    return (left < all ? left : all) > s.tpt ? s.w2 : s.w1;
}

// sum of ceil(y / 2^lg), 1 <= y <= x, and of floor(y / 2^lg), 0 <= y <= x (x >= -1)
KVATTN_HD long long sum_ceil(long long x, int lg) {
    const long long q = x >> lg, r = x & ((1 << lg) - 1);
    return ((q * (q + 1) / 2) << lg) + r * (q + 1);
}
KVATTN_HD long long sum_floor(long long x, int lg) {
    const long long q = (x + 1) >> lg, r = (x + 1) & ((1 << lg) - 1);
    return ((q * (q - 1) / 2) << lg) + r * q;
}

// Cost of a sequence's first m blocks (of one head group).
KVATTN_HD long long blocks_cost(const UnitSeq &s, int m) {
    if (m <= 0) return 0;
    const int nb = seq_blocks(s);
    const int f = m < nb ? m : nb - 1;  // full blocks; the last may end early
    long long c = (long long)m * s.piece;
    if (m == nb) c += (long long)unit_weight(s, nb - 1) * unit_tiles(s, nb - 1);
    if (f == 0) return c;
    const int w = unit_weight(s, 0);  // (of all full blocks)
    if (!s.causal) return c + (long long)f * w * unit_tiles(s, 0);
    long long t = 0;  // their tiles
    const long long lo = (long long)s.shift + 1 - s.window;  // where block 0's window starts
    if (s.tpu_lg > kUnitLg) {                                // two key tiles a block
        t += (long long)f * ((s.shift + kUnitKeys - 1) >> kUnitLg) + (long long)f * (f + 1);
        const long long a = lo >> kUnitLg;                   // (rounded down, below 0 too)
        const long long i0 = a >= 0 ? 0 : (-a + 1) / 2;      // blocks whose window starts at 0
        if (f > i0) t -= (f - i0) * a + (f - i0) * (f + i0 - 1);
    } else {  // 2^lg blocks a key tile
        const int lg = kUnitLg - s.tpu_lg;
        const long long up = ((long long)s.shift + (1 << s.tpu_lg) - 1) >> s.tpu_lg;
        t += sum_ceil(up + f, lg) - sum_ceil(up, lg);
        const long long a = lo >> s.tpu_lg;
        const long long i0 = a >= 0 ? 0 : -a;
        if (f > i0) t -= sum_floor(a + f - 1, lg) - sum_floor(a + i0 - 1, lg);
    }
    return c + w * t;
}

// The block that cost r (less than that of all) falls in.
KVATTN_HD int block_at_cost(const UnitSeq &s, long long r) {
    int lo = 0, hi = seq_blocks(s) - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (blocks_cost(s, mid) <= r) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Range c of C equal ones of a call's cost starts here (no product passes 64
// bits; in 32 where they do, which the device divides in several times faster).
KVATTN_HD long long range_start(long long total, int C, int c) {
    if (total < 1LL << 31 && C < 1 << 15) {
        const unsigned t = (unsigned)total, n = (unsigned)C, i = (unsigned)c;
        const unsigned q = t / n;
        return (long long)q * i + (t - q * n) * i / n;
    }
    return total / C * c + total % C * c / C;
}
// The last range that starts at or before e.
KVATTN_HD int range_of(long long total, int C, long long e) {
    long long c;
    if (total < 1LL << 31) {
        const unsigned q = (unsigned)total / (unsigned)C;
        c = q > 0 ? (unsigned)e / q : C - 1;
    } else {
        c = e / (total / C);
    }
    if (c > C - 1) c = C - 1;
    while (range_start(total, C, (int)c) > e) --c;
    return (int)c;
}

// Tiles of a unit at cost u, of nt of weight w, that start before x.
KVATTN_HD int tiles_before(long long u, int nt, int w, int piece, long long x) {
    if (x <= u) return 0;
    const long long d = x - u - piece;
    if (d <= w) return 1;
    if (d > (long long)w * (nt - 1)) return nt;
    return (int)(((unsigned)d + w - 1) / (unsigned)w);  // (d is below nt w, which fits)
}

}  // namespace kvattn
