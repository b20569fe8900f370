// blocks.cu -- forking, freeing and compacting the blocks of a paged cache, and
// copying the ones that these calls name ("Machine Learning Engineering and AI
// Systems at Scale", section "The key and value cache", on PagedAttention:
// sequences that share a prefix point at the same blocks).
//
// What they compute.  refs[b] counts the holders of block b beyond the first, so
// that a block fresh from the free stack has none and kv_block_tables needs no
// count of its own.  A fork shares the parent's whole blocks (refs + 1 each) and
// takes one block for the last, partly filled one, whose copy the caller makes
// in every layer.  Freeing takes refs - 1 per entry; a block that falls below
// zero has lost its last holder and is pushed, in ascending order of the ids, so
// that the result does not depend on the order of the atomics (their sums do not
// either).  Compaction: with `used` blocks held, the k-th held block at or past
// `used` moves to the k-th free one below it.
//
// Layout.  Some kilobytes of integers, or some hundred, and four to six steps that
// each need all of the one before: one CTA of 1024 threads does all steps of a
// small call (a CTA's barriers cost less than a cluster's: 64 forks of up to 128
// blocks 7.6 us for 8.7, dropping them 7.4 for 9.9), one cluster of eight those of a
// large one, the counts of the CTAs exchanged through distributed shared memory; a
// kernel per step would cost a launch each.  No workspace.  What bounds a call: the
// chain of barriers and dependent loads; a pool of 65 536 blocks compacted 24 us, of
// which the scattered marks, moves and table entries of eight SMs are 12 (more SMs for
// them, in a second launch, have not been tried).
//
// kv_copy_blocks is a copy of 16-byte vectors of K and V, four of each in flight
// per thread, and bound by HBM: 7680 blocks of 16 x 8 x 128 150 us, 0.98 of the
// measured copy rate.
#include <climits>
#include <cooperative_groups.h>

#include "../../include/kvattn.h"
#include "internal.h"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace kvattn {

namespace {

constexpr int kCtas = 8;                       // of a large call's cluster
constexpr int kThr = 1024;
constexpr int kPer = 8;                        // requests per thread at most (65535 / (kCtas kThr))
constexpr int kTile = 4 * kThr;                // blocks of a CTA's step, four to a thread
constexpr int kSmallNames = 256, kSmallBlocks = 1 << 15;  // a call up to these is one CTA's

// ------------------------------------------------------------------- scans

struct Scan {
    int warp[32];
    int total;
    long long cta[3];  // this CTA's sums, read by the others (each place once)
};

// The CTAs of a call, NC of them: one or a cluster.
template <int NC>
struct Team {
    static constexpr int kAll = NC * kThr, kWarps = kAll / 32;
    int rank = 0;
    __device__ __forceinline__ Team() {
        if constexpr (NC > 1) rank = (int)cg::this_cluster().block_rank();
    }
    __device__ __forceinline__ void sync() const {
        if constexpr (NC > 1)
            cg::this_cluster().sync();
        else
            __syncthreads();
    }
    // (a barrier) the sums of the CTAs before this one, given its own, and of all
    __device__ __forceinline__ long long scan(long long mine, Scan &s, int place, long long *all) const {
        if constexpr (NC > 1) {
            cg::cluster_group cl = cg::this_cluster();
            if (threadIdx.x == 0) s.cta[place] = mine;
            cl.sync();
            long long before = 0, sum = 0;
#pragma unroll
            for (int r = 0; r < NC; ++r) {
                const long long x = *cl.map_shared_rank(&s.cta[place], r);
                if (r < rank) before += x;
                sum += x;
            }
            *all = sum;
            return before;
        } else {
            __syncthreads();
            *all = mine;
            return 0;
        }
    }
};

// Exclusive prefix sum over a CTA's threads, and their sum.  (Its barriers also
// end the use of s before.)
__device__ __forceinline__ int cta_scan(int v, Scan &s, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
    }
    __syncthreads();
    if (lane == 31) s.warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const int mine = s.warp[lane];
        int w = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += x;
        }
        s.warp[lane] = w - mine;
        if (lane == 31) s.total = w;
    }
    __syncthreads();
    *total = s.total;
    return s.warp[warp] + incl - v;
}

__device__ __forceinline__ void blk_error(unsigned int *err) { atomicCAS(err, 0u, (unsigned int)DEV_ERR_BOUNDS); }

// Four consecutive counts of blocks from b on (b a multiple of 4), `pad` past the end.
__device__ __forceinline__ void load_blocks(const int32_t *a, int b, int n, int pad, int (&v)[4]) {
    if (b + 4 <= n) {
        const int4 x = __ldcg(reinterpret_cast<const int4 *>(a + b));
        v[0] = x.x;
        v[1] = x.y;
        v[2] = x.z;
        v[3] = x.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = b + i < n ? __ldcg(a + b + i) : pad;
    }
}

// ------------------------------------------------------------------- forks

struct ForkParams {
    int32_t *table, *lens, *refs;
    const int32_t *free_ids, *free_count, *parents, *children;
    int32_t *copies, *count_out;
    unsigned int *err;
    int n, R, max_blocks, lg, num_blocks, num_free;
};

template <int NC>
__global__ void __launch_bounds__(kThr) fork_kernel(const ForkParams p) {
    using T = Team<NC>;
    __shared__ Scan s;
    pdl_launch_dependents();
    pdl_wait_prior();
    const T team;
    const int t = team.rank * kThr + threadIdx.x;
    const int per = (p.n + T::kAll - 1) / T::kAll;  // consecutive forks of a thread
    const int i0 = min(t * per, p.n), i1 = min(i0 + per, p.n);
    int count = __ldcg(p.free_count);
    bool bad = count < 0 || count > p.num_free;
    const int said = count;
    if (bad) count = 0;

    // whose row is free (its length 0) and within the table
    unsigned able = 0;
    for (int i = i0; i < i1; ++i) {
        const int a = p.parents[i], c = p.children[i];
        if (a >= 0 && a < p.R && c >= 0 && c < p.R && __ldcg(p.lens + c) == 0) able |= 1u << (i - i0);
    }
    team.sync();
    // of forks into one row the first has it: it leaves the smallest mark in the
    // row's length.  A parent that is marked is some fork's child.
    for (int i = i0; i < i1; ++i)
        if (able >> (i - i0) & 1) atomicMin(p.lens + p.children[i], INT_MIN + i);
    team.sync();
    int need = 0;
    unsigned parts = 0;
    const int cap = p.max_blocks << p.lg, rest = (1 << p.lg) - 1;
    for (int i = i0; i < i1; ++i) {
        if (!(able >> (i - i0) & 1)) continue;
        const int len = __ldcg(p.lens + p.parents[i]);
        if (__ldcg(p.lens + p.children[i]) != INT_MIN + i || len < 0 || len > cap) {
            able &= ~(1u << (i - i0));
        } else if (len & rest) {
            parts |= 1u << (i - i0);
            ++need;
        }
    }
    int cta;
    long long all;
    const int in_cta = cta_scan(need, s, &cta);
    int before = (int)team.scan(cta, s, 0, &all) + in_cta;
    // (a barrier: every length and mark has been read)
    __shared__ int served[NC == 1 ? kSmallNames : 1];  // (one CTA) a fork's length, or -1
    for (int i = i0; i < i1; ++i) {
        const bool own = able >> (i - i0) & 1, part = parts >> (i - i0) & 1;
        const int a = p.parents[i], c = p.children[i];
        bool ok = own;
        int len = own ? __ldcg(p.lens + a) : -1, fresh = -1;
        if (part) {
            ok = before < count;
            if (ok) fresh = p.free_ids[count - 1 - before];
            ok = ok && fresh >= 0 && fresh < p.num_blocks;
            ++before;
        }
        if (!ok) {
            bad = true;
            len = -1;
            fresh = -1;
        }
        if constexpr (NC == 1)
            served[i] = len;
        else  // (what the fork's warp is to know waits in its place of the copies)
            p.copies[2 * i] = len, p.copies[2 * i + 1] = fresh;
        if constexpr (NC == 1) {
            int src = -1;
            if (fresh >= 0) {
                src = p.table[(size_t)a * p.max_blocks + (len >> p.lg)];
                p.table[(size_t)c * p.max_blocks + (len >> p.lg)] = fresh;
                if (src < 0 || src >= p.num_blocks) {  // nothing to copy
                    src = -1;
                    bad = true;
                }
            }
            p.copies[2 * i] = src;
            p.copies[2 * i + 1] = src < 0 ? -1 : fresh;
        }
    }
    if (t == 0) p.count_out[0] = said == count ? count - (int)min(all, (long long)count) : said;
    team.sync();
    // (nobody reads the marks and the parents' lengths any more, but a refused fork
    // its own mark)
    const int gw = t >> 5, lane = t & 31;
    // a warp per fork, or several for its entries where there are few forks
    const int ways = max(1, T::kWarps / p.n);
    for (int i = gw / ways; i < p.n; i += T::kWarps / ways) {
        const int way = gw % ways;
        const int len = NC == 1 ? served[i] : __ldcg(p.copies + 2 * i);
        const int a = p.parents[i], c = p.children[i];
        if (len >= 0) {
            const int32_t *from = p.table + (size_t)a * p.max_blocks;
            int32_t *to = p.table + (size_t)c * p.max_blocks;
            const int whole = len >> p.lg;
            for (int e0 = lane + 128 * way; e0 < whole; e0 += 128 * ways) {
                int b[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) b[q] = e0 + 32 * q < whole ? from[e0 + 32 * q] : -1;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (e0 + 32 * q < whole) {
                        to[e0 + 32 * q] = b[q];
                        if (b[q] >= 0 && b[q] < p.num_blocks)
                            atomicAdd(p.refs + b[q], 1);
                        else
                            bad = true;
                    }
            }
            if (way == 0 && lane == 0) p.lens[c] = len;
        } else if (way == 0 && lane == 0 && c >= 0 && c < p.R && __ldcg(p.lens + c) == INT_MIN + i) {
            p.lens[c] = 0;  // the row that this fork had marked
        }
        if constexpr (NC > 1) {  // (one warp a fork)
            int src = -1, dst = -1;
            if (len >= 0 && (len & rest)) {
                dst = __ldcg(p.copies + 2 * i + 1);
                src = p.table[(size_t)a * p.max_blocks + (len >> p.lg)];
                if (lane == 0) p.table[(size_t)c * p.max_blocks + (len >> p.lg)] = dst;
                if (src < 0 || src >= p.num_blocks) {  // nothing to copy
                    src = dst = -1;
                    bad = true;
                }
            }
            __syncwarp();
            if (lane == 0) {
                p.copies[2 * i] = src;
                p.copies[2 * i + 1] = dst;
            }
        }
    }
    if (bad) blk_error(p.err);
}

// ----------------------------------------------------------------- freeing

struct FreeParams {
    int32_t *table, *lens, *refs, *free_ids;
    const int32_t *free_count, *requests;
    int32_t *count_out;
    unsigned int *err;
    int n, R, max_blocks, lg, num_blocks, num_free;
};

// A CTA's share of the blocks: whole tiles, the same order as the CTAs'.
template <int NC>
__device__ __forceinline__ void share_of(int num_blocks, int rank, int *b0, int *b1) {
    const int tiles = (int)(((long long)num_blocks + kTile - 1) / kTile);
    const int each = (tiles + NC - 1) / NC;
    *b0 = (int)min((long long)num_blocks, (long long)rank * each * kTile);
    *b1 = (int)min((long long)num_blocks, (long long)*b0 + (long long)each * kTile);
}

template <int NC>
__global__ void __launch_bounds__(kThr) free_kernel(const FreeParams p) {
    using T = Team<NC>;
    __shared__ Scan s;
    pdl_launch_dependents();
    pdl_wait_prior();
    const T team;
    const int t = team.rank * kThr + threadIdx.x, gw = t >> 5, lane = t & 31;
    const int count = __ldcg(p.free_count);
    const bool refuse = count < 0 || count > p.num_free;  // nothing is done
    bool bad = refuse;
    const int cap = p.max_blocks << p.lg, rest = (1 << p.lg) - 1;

    // lets go of the entries of row r from e0 on, 128 of every `every`
    auto let_go = [&](int r, int nb, int e0, int every) {
        int32_t *row = p.table + (size_t)r * p.max_blocks;
        for (e0 += lane; e0 < nb; e0 += every) {
            int b[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) b[q] = e0 + 32 * q < nb ? row[e0 + 32 * q] : 0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (e0 + 32 * q < nb) {
                    row[e0 + 32 * q] = -1;
                    if (b[q] >= 0 && b[q] < p.num_blocks)
                        atomicSub(p.refs + b[q], 1);
                    else
                        bad = true;
                }
        }
    };
    // the length of the i-th request, 0 if there is nothing to free, and its row
    auto length_of = [&](int i, int *r) {
        int len = 0;
        *r = -1;
        if (i < p.n && !refuse) {
            *r = p.requests[i];
            if (*r >= 0 && *r < p.R) {
                len = __ldcg(p.lens + *r);
                if (len < 0 || len > cap) {
                    len = 0;
                    bad = true;
                }
            } else {
                bad = true;
            }
        }
        return len;
    };
    // A request named twice is freed once: the first name leaves the smallest mark in
    // its length.
    if (NC == 1 || p.n <= kSmallNames) {
        // every CTA has the whole list, and all warps share the entries
        __shared__ int rows[kSmallNames], lens[kSmallNames];
        int r;
        const int i = threadIdx.x, len = length_of(i, &r);
        team.sync();
        if (team.rank == 0 && len > 0) atomicMin(p.lens + r, INT_MIN + i);
        team.sync();
        if (i < kSmallNames) {
            rows[i] = r;
            lens[i] = len > 0 && __ldcg(p.lens + r) == INT_MIN + i ? len : 0;
        }
        __syncthreads();
        const int ways = max(1, T::kWarps / p.n);
        for (int k = gw / ways; k < p.n; k += T::kWarps / ways)
            let_go(rows[k], (lens[k] + rest) >> p.lg, 128 * (gw % ways), 128 * ways);
        team.sync();
        if (team.rank == 0 && len > 0) p.lens[r] = 0;  // (every mark has been compared)
    } else {
        // request gw + kWarps (lane + 32 u) is this lane's u-th, and its warp's to free
        int len[kPer], req[kPer];
#pragma unroll
        for (int u = 0; u < kPer; ++u) len[u] = length_of(gw + T::kWarps * (lane + 32 * u), &req[u]);
        team.sync();
#pragma unroll
        for (int u = 0; u < kPer; ++u)
            if (len[u] > 0) atomicMin(p.lens + req[u], INT_MIN + gw + T::kWarps * (lane + 32 * u));
        team.sync();
#pragma unroll
        for (int u = 0; u < kPer; ++u) {
            const int i = gw + T::kWarps * (lane + 32 * u);
            const bool mine = len[u] > 0 && __ldcg(p.lens + req[u]) == INT_MIN + i;
            unsigned todo = __ballot_sync(0xffffffffu, mine);
            while (todo) {
                const int src = __ffs(todo) - 1;
                todo &= todo - 1;
                const int r = __shfl_sync(0xffffffffu, req[u], src);
                let_go(r, (__shfl_sync(0xffffffffu, len[u], src) + rest) >> p.lg, 0, 128);
            }
        }
        team.sync();
#pragma unroll
        for (int u = 0; u < kPer; ++u)
            if (len[u] > 0) p.lens[req[u]] = 0;
    }

    // the blocks without a holder, in the order of their ids
    int b0, b1;
    share_of<NC>(p.num_blocks, team.rank, &b0, &b1);
    int mine = 0;
    for (int b = b0 + 4 * (int)threadIdx.x; b < b1; b += kTile) {
        int v[4];
        load_blocks(p.refs, b, b1, 0, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) mine += v[i] < 0;
    }
    int cta;
    long long all;
    cta_scan(mine, s, &cta);
    long long at = count + team.scan(cta, s, 0, &all);
    if (cta > 0 && !refuse) {
        for (int b = b0; b < b1; b += kTile) {
            const int mb = b + 4 * (int)threadIdx.x;
            int v[4] = {0, 0, 0, 0};
            if (mb < b1) load_blocks(p.refs, mb, b1, 0, v);
            int k = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) k += v[i] < 0;
            if (!__syncthreads_or(k)) continue;
            int tile;
            const int rank = cta_scan(k, s, &tile);
            long long to = at + rank;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (v[i] < 0) {
                    if (v[i] < -1) bad = true;  // let go more often than it was held
                    p.refs[mb + i] = 0;
                    if (to < p.num_free)
                        p.free_ids[to] = mb + i;
                    else
                        bad = true;  // no room: the stack is smaller than the pool
                    ++to;
                }
            at += tile;
        }
    }
    if (t == 0) p.count_out[0] = refuse ? count : (int)min(count + all, (long long)p.num_free);
    if (bad) blk_error(p.err);
    if (NC > 1) team.sync();  // (the others may still read this CTA's sum)
}

// -------------------------------------------------------------- compaction

struct CompactParams {
    const int32_t *table, *lens, *refs, *free_ids, *free_count;
    int32_t *table_out, *refs_out, *free_out, *count_out, *moves, *remap;
    unsigned int *err;
    int R, max_blocks, lg, num_blocks, num_free;
};

template <int NC>
__global__ void __launch_bounds__(kThr) compact_kernel(const CompactParams p) {
    using T = Team<NC>;
    __shared__ Scan s;
    pdl_launch_dependents();
    pdl_wait_prior();
    const T team;
    const int t = team.rank * kThr + threadIdx.x, gw = t >> 5, lane = t & 31;
    const int n = p.num_blocks;
    const int said = __ldcg(p.free_count);
    bool bad = said < 0 || said > p.num_free;
    const int count = bad ? 0 : said;

    // remap: -1 for the blocks on the stack, each other block itself
    int b0, b1, cta;
    long long all;
    share_of<NC>(n, team.rank, &b0, &b1);
    for (int b = b0 + 4 * (int)threadIdx.x; b < b1; b += kTile) {
        if (b + 4 <= b1)
            *reinterpret_cast<int4 *>(p.remap + b) = make_int4(b, b + 1, b + 2, b + 3);
        else
            for (int i = b; i < b1; ++i) p.remap[i] = i;
    }
    team.sync();
    // (here and below four loads of a thread are in flight: a step is some loads long)
    for (int k0 = t; k0 < count; k0 += 4 * T::kAll) {
        int b[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) b[q] = k0 + q * T::kAll < count ? p.free_ids[k0 + q * T::kAll] : 0;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (k0 + q * T::kAll < count) {
                if (b[q] >= 0 && b[q] < n)
                    p.remap[b[q]] = -1;
                else
                    bad = true;
            }
    }
    team.sync();
    int mine = 0;
    for (int b = b0 + 4 * (int)threadIdx.x; b < b1; b += kTile) {
        int v[4];
        load_blocks(p.remap, b, b1, 0, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) mine += v[i] < 0;
    }
    cta_scan(mine, s, &cta);
    team.scan(cta, s, 0, &all);
    const int used = n - (int)all;
    if ((int)all != count) bad = true;  // an id twice

    // holes: free blocks below `used`; movers: held ones from there on
    auto kind = [&](int b, int v) { return v < 0 ? (b < used ? 1 : 0) : (b >= used && b < n ? 1 << 16 : 0); };
    int holes = b1 <= used ? cta : 0, movers = b0 >= used ? b1 - b0 - cta : 0;
    if (b0 < used && used < b1) {  // (one CTA's share has the border)
        int h = 0, m = 0;
        for (int b = b0 + 4 * (int)threadIdx.x; b < b1; b += kTile) {
            int v[4];
            load_blocks(p.remap, b, b1, 0, v);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int k = b + i < b1 ? kind(b + i, v[i]) : 0;
                h += k & 1;
                m += k >> 16;
            }
        }
        cta_scan(h, s, &holes);
        cta_scan(m, s, &movers);
    }
    const long long first = team.scan((long long)holes << 32 | (unsigned)movers, s, 1, &all);
    int hole = (int)(first >> 32), mover = (int)first;
    const int moved = (int)(all >> 32);
    if (holes + movers > 0)
        for (int b = b0; b < b1; b += kTile) {
            const int mb = b + 4 * (int)threadIdx.x;
            int v[4], k[4] = {0, 0, 0, 0}, sum = 0;
            if (mb < b1) {
                load_blocks(p.remap, mb, b1, 0, v);
#pragma unroll
                for (int i = 0; i < 4; ++i) k[i] = mb + i < b1 ? kind(mb + i, v[i]) : 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) sum += k[i];
            int tile;
            const int rank = cta_scan(sum, s, &tile);  // (4096 of a kind at most: 16 bits each)
            int h = hole + (rank & 0xffff), m = mover + (rank >> 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (k[i] == 1) p.moves[2 * h++ + 1] = mb + i;
                if (k[i] > 1) p.moves[2 * m++] = mb + i;
            }
            hole += tile & 0xffff;
            mover += tile >> 16;
        }
    for (int k = 2 * moved + t; k < n / 2 * 2; k += T::kAll) p.moves[k] = -1;
    team.sync();
    // references: a hole's are its mover's, and nobody holds what lies from `used` on.
    // (Holes and movers are left to the second loop; a mover's place of the map says
    // that it is held before and after it.)
    for (int b = b0 + 4 * (int)threadIdx.x; b < b1; b += kTile) {
        int v[4], r[4] = {0, 0, 0, 0};
        load_blocks(p.remap, b, b1, 0, v);
        if (b < used && p.refs_out != p.refs) load_blocks(p.refs, b, b1, 0, r);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (b + i < b1) {
                if (b + i >= used ? v[i] < 0 : v[i] >= 0 && p.refs_out != p.refs)
                    p.refs_out[b + i] = b + i >= used ? 0 : r[i];
            }
    }
    for (int k0 = t; k0 < moved; k0 += 4 * T::kAll) {
        int2 m[4];  // (from, to)
        int r[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (k0 + q * T::kAll < moved) m[q] = __ldcg(reinterpret_cast<const int2 *>(p.moves) + k0 + q * T::kAll);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (k0 + q * T::kAll < moved) r[q] = p.refs[m[q].x];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (k0 + q * T::kAll < moved) {
                p.refs_out[m[q].y] = r[q];
                p.refs_out[m[q].x] = 0;
                p.remap[m[q].x] = m[q].y;
            }
    }
    const int left = n - used;
    for (int k = t; k < min(left, p.num_free); k += T::kAll) p.free_out[k] = n - 1 - k;  // the lowest id on top
    if (p.free_out != p.free_ids)
        for (int k0 = left + t; k0 < p.num_free; k0 += 4 * T::kAll) {
            int b[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) b[q] = k0 + q * T::kAll < p.num_free ? p.free_ids[k0 + q * T::kAll] : 0;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (k0 + q * T::kAll < p.num_free) p.free_out[k0 + q * T::kAll] = b[q];
        }
    if (t == 0) p.count_out[0] = said == count ? left : said;
    team.sync();
    const int cap = p.max_blocks << p.lg, rest = (1 << p.lg) - 1;
    const bool in_place = p.table_out == p.table;
    // four requests a warp, or several warps for their entries where there are few
    const int fours = (p.R + 3) / 4, ways = max(1, T::kWarps / fours);
    for (int r0 = gw / ways * 4; r0 < p.R; r0 += T::kWarps / ways * 4) {
        int len = lane < 4 && r0 + lane < p.R ? p.lens[r0 + lane] : 0;
        if (len < 0 || len > cap) {
            bad = true;
            len = 0;
        }
        int nb[4], last = in_place ? 0 : p.max_blocks;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            nb[q] = (__shfl_sync(0xffffffffu, len, q) + rest) >> p.lg;
            if (in_place) last = max(last, nb[q]);
        }
        for (int e = lane + 32 * (gw % ways); e < last; e += 32 * ways) {
            int b[4], to[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const bool here = r0 + q < p.R && (!in_place || e < nb[q]);
                b[q] = here ? p.table[(size_t)(r0 + q) * p.max_blocks + e] : -1;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                to[q] = b[q];
                if (e < nb[q] && b[q] >= 0 && b[q] < n) to[q] = __ldcg(p.remap + b[q]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
                if (r0 + q < p.R && (!in_place || e < nb[q])) {
                    if (e < nb[q] && (to[q] < 0 || to[q] >= n)) bad = true;  // no block, or a free one
                    p.table_out[(size_t)(r0 + q) * p.max_blocks + e] = to[q];
                }
        }
    }
    if (bad) blk_error(p.err);
}

// ------------------------------------------------------------------ copies

constexpr int kCopyThreads = 256;
constexpr int kCopyVecs = 4;  // of K, and of V, per thread

template <class T>
struct CopyParams {
    T *k, *v;
    const int32_t *copies;
    unsigned int *err;
    int n, num_blocks;
    unsigned vecs;  // of a block
};

template <class T>
__global__ void __launch_bounds__(kCopyThreads) copy_blocks_kernel(const CopyParams<T> p) {
    pdl_launch_dependents();
    pdl_wait_prior();
    const unsigned long long v0 = (unsigned long long)blockIdx.x * (kCopyThreads * kCopyVecs);
    const unsigned long long first = v0 / p.vecs;
    const unsigned off0 = (unsigned)(v0 - first * p.vecs);
    T k[kCopyVecs], v[kCopyVecs];
    long long dst[kCopyVecs];
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i) {
        const unsigned x = off0 + i * kCopyThreads + threadIdx.x;  // (vecs is at most 2^30)
        const unsigned more = x / p.vecs, c = x - more * p.vecs;
        const unsigned long long pair = first + more;
        dst[i] = -1;
        if (pair < (unsigned long long)p.n) {
            const int2 m = reinterpret_cast<const int2 *>(p.copies)[pair];
            if (m.x >= 0 && m.y >= 0 && m.x < p.num_blocks && m.y < p.num_blocks) {
                dst[i] = (long long)m.y * p.vecs + c;
                k[i] = __ldcs(p.k + (long long)m.x * p.vecs + c);
                v[i] = __ldcs(p.v + (long long)m.x * p.vecs + c);
            } else if (m.x != -1 || m.y != -1) {
                blk_error(p.err);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kCopyVecs; ++i)
        if (dst[i] >= 0) {
            p.k[dst[i]] = k[i];
            p.v[dst[i]] = v[i];
        }
}

template <class Kernel, class Params>
cudaError_t launch_pdl(Kernel kernel, unsigned grid, unsigned block, cudaStream_t stream, const Params &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// One CTA, or a cluster of kCtas.
template <class Kernel, class Params>
cudaError_t launch_team(Kernel one, Kernel many, bool small, cudaStream_t stream, const Params &p) {
    if (small) return launch_pdl(one, 1, kThr, stream, p);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCtas);
    cfg.blockDim = dim3(kThr);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCtas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, many, p);
}

template <class T>
cudaError_t launch_copies(void *k, void *v, const int32_t *copies, unsigned int *err, int n, int num_blocks,
                          long long block_bytes, cudaStream_t stream) {
    CopyParams<T> p = {};
    p.k = static_cast<T *>(k);
    p.v = static_cast<T *>(v);
    p.copies = copies;
    p.err = err;
    p.n = n;
    p.num_blocks = num_blocks;
    p.vecs = (unsigned)(block_bytes / sizeof(T));
    const unsigned long long all = (unsigned long long)n * p.vecs;
    const unsigned grid = (unsigned)((all + kCopyThreads * kCopyVecs - 1) / (kCopyThreads * kCopyVecs));
    return launch_pdl(copy_blocks_kernel<T>, grid, kCopyThreads, stream, p);
}

bool off(const void *p, unsigned mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

// The sizes that fork, free and compaction share.
int check_pool(const int32_t *table, int R, int max_blocks, int block_size, int num_blocks, int num_free,
               const char *who, int *lg) {
    if (R <= 0 || num_free <= 0)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: R and num_free must be positive (%d, %d)", who, R, num_free);
    if (R > 65535 || num_blocks > (1 << 28) || num_free > (1 << 28))
        return api_failf(KVATTN_ERR_UNSUPPORTED,
                         "%s: sizes beyond limits (R <= 65535, num_blocks and num_free <= 2^28)", who);
    int lmax;
    return api_check_paged(table, 1, block_size, max_blocks, num_blocks, who, lg, &lmax);
}

int check_names(int n, const char *who) {
    if (n < 1) return api_failf(KVATTN_ERR_INVALID_ARG, "%s: n must be positive (got %d)", who, n);
    if (n > 65535) return api_failf(KVATTN_ERR_UNSUPPORTED, "%s: n = %d beyond 65535", who, n);
    return KVATTN_OK;
}

}  // namespace

}  // namespace kvattn

using namespace kvattn;

extern "C" {

int kv_fork_blocks(int32_t *block_table, int32_t *seq_lens, int32_t *refs, const int32_t *free_blocks,
                   const int32_t *free_count, const int32_t *parents, const int32_t *children, int32_t *copies,
                   int32_t *free_count_out, int n, int R, int max_blocks, int block_size, int num_blocks,
                   int num_free, kvattn_stream_t stream) {
    const char *who = "kv_fork_blocks";
    api_begin();
    if (!block_table || !seq_lens || !refs || !free_blocks || !free_count || !parents || !children || !copies ||
        !free_count_out)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: null pointer", who);
    if (off(block_table, 3) || off(seq_lens, 3) || off(refs, 15) || off(free_blocks, 3) || off(free_count, 3) ||
        off(parents, 3) || off(children, 3) || off(copies, 7) || off(free_count_out, 3))
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: int32 arrays must be 4-byte, copies 8, refs 16-byte aligned",
                         who);
    ForkParams p = {};
    int rc, ctas;
    unsigned int wait_limit;
    if ((rc = check_names(n, who)) ||
        (rc = check_pool(block_table, R, max_blocks, block_size, num_blocks, num_free, who, &p.lg)) ||
        (rc = api_device(&ctas, &p.err, &wait_limit)))
        return rc;
    p.table = block_table;
    p.lens = seq_lens;
    p.refs = refs;
    p.free_ids = free_blocks;
    p.free_count = free_count;
    p.parents = parents;
    p.children = children;
    p.copies = copies;
    p.count_out = free_count_out;
    p.n = n; p.R = R;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.num_free = num_free;
    cudaError_t e = launch_team(fork_kernel<1>, fork_kernel<kCtas>, n <= kSmallNames,
                                reinterpret_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess) return api_cuda_fail(e, "fork launch");
    return KVATTN_OK;
}

int kv_free_blocks(int32_t *block_table, int32_t *seq_lens, int32_t *refs, int32_t *free_blocks,
                   const int32_t *free_count, const int32_t *requests, int32_t *free_count_out, int n, int R,
                   int max_blocks, int block_size, int num_blocks, int num_free, kvattn_stream_t stream) {
    const char *who = "kv_free_blocks";
    api_begin();
    if (!block_table || !seq_lens || !refs || !free_blocks || !free_count || !requests || !free_count_out)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: null pointer", who);
    if (off(block_table, 3) || off(seq_lens, 3) || off(refs, 15) || off(free_blocks, 3) || off(free_count, 3) ||
        off(requests, 3) || off(free_count_out, 3))
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: int32 arrays must be 4-byte, refs 16-byte aligned", who);
    FreeParams p = {};
    int rc, ctas;
    unsigned int wait_limit;
    if ((rc = check_names(n, who)) ||
        (rc = check_pool(block_table, R, max_blocks, block_size, num_blocks, num_free, who, &p.lg)) ||
        (rc = api_device(&ctas, &p.err, &wait_limit)))
        return rc;
    p.table = block_table;
    p.lens = seq_lens;
    p.refs = refs;
    p.free_ids = free_blocks;
    p.free_count = free_count;
    p.requests = requests;
    p.count_out = free_count_out;
    p.n = n; p.R = R;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.num_free = num_free;
    cudaError_t e = launch_team(free_kernel<1>, free_kernel<kCtas>, n <= kSmallNames && num_blocks <= kSmallBlocks,
                                reinterpret_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess) return api_cuda_fail(e, "free launch");
    return KVATTN_OK;
}

int kv_compact_blocks(const int32_t *block_table, const int32_t *seq_lens, const int32_t *refs,
                      const int32_t *free_blocks, const int32_t *free_count, int32_t *block_table_out,
                      int32_t *refs_out, int32_t *free_blocks_out, int32_t *free_count_out, int32_t *moves,
                      int32_t *remap, int R, int max_blocks, int block_size, int num_blocks, int num_free,
                      kvattn_stream_t stream) {
    const char *who = "kv_compact_blocks";
    api_begin();
    if (!block_table || !seq_lens || !refs || !free_blocks || !free_count || !block_table_out || !refs_out ||
        !free_blocks_out || !free_count_out || !moves || !remap)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: null pointer", who);
    if (off(block_table, 3) || off(seq_lens, 3) || off(refs, 15) || off(free_blocks, 3) || off(free_count, 3) ||
        off(block_table_out, 3) || off(refs_out, 15) || off(free_blocks_out, 3) || off(free_count_out, 3) ||
        off(moves, 7) || off(remap, 15))
        return api_failf(KVATTN_ERR_INVALID_ARG,
                         "%s: int32 arrays must be 4-byte, moves 8, refs and remap 16-byte aligned", who);
    CompactParams p = {};
    int rc, ctas;
    unsigned int wait_limit;
    if ((rc = check_pool(block_table, R, max_blocks, block_size, num_blocks, num_free, who, &p.lg))) return rc;
    if ((rc = api_device(&ctas, &p.err, &wait_limit))) return rc;
    p.table = block_table;
    p.lens = seq_lens;
    p.refs = refs;
    p.free_ids = free_blocks;
    p.free_count = free_count;
    p.table_out = block_table_out;
    p.refs_out = refs_out;
    p.free_out = free_blocks_out;
    p.count_out = free_count_out;
    p.moves = moves;
    p.remap = remap;
    p.R = R;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.num_free = num_free;
    cudaError_t e = launch_team(compact_kernel<1>, compact_kernel<kCtas>, R <= kSmallNames && num_blocks <= kSmallBlocks,
                                reinterpret_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess) return api_cuda_fail(e, "compaction launch");
    return KVATTN_OK;
}

int kv_copy_blocks(void *k_pool, void *v_pool, const int32_t *copies, int n, int num_blocks, long long block_bytes,
                   kvattn_stream_t stream) {
    const char *who = "kv_copy_blocks";
    api_begin();
    if (!k_pool || !v_pool || !copies) return api_failf(KVATTN_ERR_INVALID_ARG, "%s: null pointer", who);
    if (block_bytes < 4 || block_bytes % 4)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: block_bytes must be a positive multiple of 4 (got %lld)", who,
                         block_bytes);
    const bool wide = block_bytes % 16 == 0;
    if (off(k_pool, wide ? 15 : 3) || off(v_pool, wide ? 15 : 3) || off(copies, 7))
        return api_failf(KVATTN_ERR_INVALID_ARG,
                         "%s: pools must be 16-byte aligned (4 where block_bytes is no multiple of 16), copies 8", who);
    if (n < 1 || num_blocks < 1)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: n and num_blocks must be positive (%d, %d)", who, n, num_blocks);
    if (n > (1 << 28) || block_bytes > (1LL << 32))
        return api_failf(KVATTN_ERR_UNSUPPORTED, "%s: sizes beyond limits (n <= 2^28, block_bytes <= 2^32)", who);
    const unsigned long long vecs = (unsigned long long)n * (unsigned long long)(block_bytes / (wide ? 16 : 4));
    if (vecs / (kCopyThreads * kCopyVecs) >= 0x7fffffffULL)
        return api_failf(KVATTN_ERR_UNSUPPORTED, "%s: too many bytes for one launch", who);
    int rc, ctas;
    unsigned int *err, wait_limit;
    if ((rc = api_device(&ctas, &err, &wait_limit))) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e = wide ? launch_copies<uint4>(k_pool, v_pool, copies, err, n, num_blocks, block_bytes, st)
                         : launch_copies<uint32_t>(k_pool, v_pool, copies, err, n, num_blocks, block_bytes, st);
    if (e != cudaSuccess) return api_cuda_fail(e, "block copy launch");
    return KVATTN_OK;
}

}  // extern "C"
