// units.cuh -- how the paged prompt attention divides a call: key tiles of all
// units (a block of a sequence's tokens, one head group), in the order (sequence,
// head group, block of tokens), cut into equal ranges of cost, a CTA each.  A
// unit of nt key tiles costs nt + cost_piece, the latter at its first tile: tile
// 0 starts at the unit's start u, tile t > 0 at u + cost_piece + t, and a CTA
// owns the tiles that start in its range.  Everything follows from the lengths
// in a few operations, so that a CTA finds its place without a list.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define KVATTN_HD __host__ __device__ __forceinline__
#else
#define KVATTN_HD inline
#endif

namespace kvattn {

constexpr int kUnitKeys = 128;  // keys of a tile

// One sequence of a call: token t (of `len`) attends the positions
// [max(0, e - window), e), e = shift + (causal ? t + 1 : 0).
struct UnitSeq {
    int len, shift, causal, window;
    int tpu;    // tokens of a unit, a power of two up to 256
    int piece;  // cost_piece
};

KVATTN_HD int seq_blocks(const UnitSeq &s) { return (s.len + s.tpu - 1) / s.tpu; }
KVATTN_HD int seq_end(const UnitSeq &s, int t) { return s.shift + (s.causal ? t + 1 : 0); }

// First key tile of a block of tokens, and how many there are.
KVATTN_HD int unit_first(const UnitSeq &s, int blk) {
    const int lo = seq_end(s, blk * s.tpu) - s.window;
    return lo > 0 ? lo / kUnitKeys : 0;
}
KVATTN_HD int unit_tiles(const UnitSeq &s, int blk) {
    const long long past = (long long)(blk + 1) * s.tpu;
    const int last = (int)(past < s.len ? past : s.len) - 1;
    return (seq_end(s, last) + kUnitKeys - 1) / kUnitKeys - unit_first(s, blk);
}

// sum of ceil(y / k), 1 <= y <= x, and of floor(y / k), 0 <= y <= x (x >= -1)
KVATTN_HD long long sum_ceil(long long x, int k) {
    const long long q = x / k, r = x % k;
    return k * (q * (q + 1) / 2) + r * (q + 1);
}
KVATTN_HD long long sum_floor(long long x, int k) {
    const long long q = (x + 1) / k, r = (x + 1) % k;
    return k * (q * (q - 1) / 2) + r * q;
}

// Cost of a sequence's first m blocks (of one head group).
KVATTN_HD long long blocks_cost(const UnitSeq &s, int m) {
    if (m <= 0) return 0;
    const int nb = seq_blocks(s);
    const int f = m < nb ? m : nb - 1;  // full blocks; the last may end early
    long long c = (long long)m * s.piece;
    if (m == nb) c += unit_tiles(s, nb - 1);
    if (!s.causal) return c + (long long)f * ((s.shift + kUnitKeys - 1) / kUnitKeys - unit_first(s, 0));
    const long long lo = (long long)s.shift + 1 - s.window;  // where block 0's window starts
    if (s.tpu > kUnitKeys) {                                 // two key tiles a block
        c += (long long)f * ((s.shift + kUnitKeys - 1) / kUnitKeys) + (long long)f * (f + 1);
        const long long a = lo >= 0 ? lo / kUnitKeys : -((-lo + kUnitKeys - 1) / kUnitKeys);  // floor
        const long long i0 = a >= 0 ? 0 : (-a + 1) / 2;      // blocks whose window starts at 0
        if (f > i0) c -= (f - i0) * a + (f - i0) * (f + i0 - 1);
    } else {  // k blocks a key tile
        const int k = kUnitKeys / s.tpu;
        const long long up = ((long long)s.shift + s.tpu - 1) / s.tpu;
        c += sum_ceil(up + f, k) - sum_ceil(up, k);
        const long long a = lo >= 0 ? lo / s.tpu : -((-lo + s.tpu - 1) / s.tpu);
        const long long i0 = a >= 0 ? 0 : -a;
        if (f > i0) c -= sum_floor(a + f - 1, k) - sum_floor(a + i0 - 1, k);
    }
    return c;
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

// Range c of C equal ones of a call's cost starts here (no product passes 64 bits).
KVATTN_HD long long range_start(long long total, int C, int c) {
    return total / C * c + total % C * c / C;
}
// The last range that starts at or before e.
KVATTN_HD int range_of(long long total, int C, long long e) {
    const long long q = total / C;
    long long c = q > 0 ? e / q : C - 1;
    if (c > C - 1) c = C - 1;
    while (range_start(total, C, (int)c) > e) --c;
    return (int)c;
}

// Tiles of a unit at cost u, of nt, that start before x.
KVATTN_HD int tiles_before(long long u, int nt, int piece, long long x) {
    if (x <= u) return 0;
    const long long t = x - u - piece;
    return t <= 1 ? 1 : t < nt ? (int)t : nt;
}

}  // namespace kvattn
