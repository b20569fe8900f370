// prefill.cuh -- the prompt-attention kernel: over packed K/V rows (PG = false,
// prefill.cu), which this comment is about, and over a paged pool (PG = true,
// extend.cu and extend_few.cu, whose comment says what differs).
//
// Causal grouped-query attention over whole prompts, packed one
// after the other ("The Basics of Transformer Inference", the prefill phase:
// every prompt token attends itself and the tokens before it, in one pass):
//     out[i,h,:] = sum_j softmax_j(scale q[i,h] . k[j,h/G]) v[j,h/G,:]
// over max(first, i - window + 1) <= j <= i of the token's own sequence.
//
// Mathematics.  One pass over the keys with a running maximum m and sum l per
// row (base-2 exponentials, scores scaled by |scale| log2 e):
//     p_j = 2^(s_j - m),  l += p_j,  O += p_j v_j,   out = O / l.
// m moves only when a score passes it by more than 2^8 (then O and l are
// rescaled by 2^(m - m')), so O is rarely touched between products; p stays
// below 2^8 and l in 32 bits.  p enters the second product as bf16 (the
// output is bf16: the weights' rounding, at most 2^-8 of each, averages out below
// the output's own).
//
// Layout.  A tile is 128 query rows: hpg = gcd(G, 128) heads of one K/V head
// by 128 / hpg consecutive tokens, so heads that share K/V share every key
// tile, and the causal diagonal is only 128 / hpg tokens wide.  Rows are
// tensor-memory lanes: thread r of a softmax warpgroup owns row r and its 128
// scores of a key tile, so row maxima and sums need no exchange.
//   S (tile)  = Q K^T     [128 x 128 keys]   both operands in shared memory
//   O (tile) += P V       [128 x D]          P in tensor memory, over S
// D = 64, 128: two query tiles per CTA, each with its S, O and warpgroup;
// while one is in its softmax the tensor cores work for the other, and both
// read the same K/V tiles.  D = 256: O takes 256 of the 512 columns, so one
// query tile per CTA with two S buffers: Q K^T of the next key tile runs
// during the softmax of this one.
//
// Warps: 0 issues the copies (TMA), 1 and 2 the MMAs (D = 64, 128: one per
// query tile, in strict turns; D = 256: one for Q K^T, one for P V), 3 walks
// the work list (and at D = 256 copies V), then one softmax warpgroup per
// query tile.
//
// What bounds it: the tensor pipe, which idles some 300 cycles between one
// query tile's products and the next's; below a few hundred tokens the chain
// of one unit (copy, Q K^T, softmax, P V, rows out: 8 us for four prompts of
// up to 97 tokens).  Measured in a graph of calls: 8192 tokens of 64 heads
// over 8 of 128 720 us (1527 TFLOP/s, 0.80 of the cuBLAS bf16 rate; called one
// after the other, with other inputs each, 760 us, 1447), of 16 heads over 1 of
// 256 340 us (1620, 0.85); eight ragged prompts of that layout 320 us (1396,
// 0.73; 331 called).  D = 64 some 905 TFLOP/s: a key tile's MMAs take 678
// cycles (64 an MMA at N = 128, 53 at N = 64) where D = 128 takes 1027 for
// twice the operations, but its softmax takes as long, and the tensor pipe is
// busy a third of the time.
//
// Work list.  A unit is (sequence, block of NQ x 128 / hpg tokens, K/V head,
// head group); its cost grows with its block's index.  Every CTA of the
// persistent grid sorts the blocks of all sequences into buckets of that
// index (from cu_seqlens, in shared memory: no workspace, no atomics on
// global memory, the same order in every run) and takes units from the
// largest down, every second round in reverse.
#pragma once

#include <climits>
#include <cuda_bf16.h>
#include <type_traits>

#include "../../include/kvattn.h"
#include "internal.h"
#include "ptx.cuh"
#include "units.cuh"

namespace kvattn {

namespace {

constexpr int kRows = 128;      // query rows of a tile = keys of a tile
constexpr int kSlab = 16384;    // 128 rows x 64 columns of bf16
constexpr int kSmemMax = 232448;
constexpr float kTauPf = 8.f;   // log2 headroom before the running max must move
constexpr int kBuckets = 128;
constexpr int kDesc = 4;        // units in flight between the work list and its readers
constexpr int kBarEndPf = 1;

// Where the keys of a unit's queries end: token t of a sequence attends the
// positions [max(0, e - window), e) with e = key_end(t).
struct PrefillParams {
    const int32_t *cu;  // [B + 1] first rows of the sequences
    uint16_t *out;      // bf16 [N, Hq, D]
    unsigned int *err;
    int B, N, Hq, Hkv, G;
    // query heads of a tile and their log2, and its tokens, 128 / hpg.  (Over a pool hpg
    // may be a whole group of another size, with a power of two of tokens, and the tile
    // have less than 128 rows; there is no log2 then.)
    int hpg, hpg_lg;
    int tpt;
    int passes;         // G / hpg
    int window;         // keys one query attends at most (N: all)
    float sl;           // |scale| log2(e), at least the smallest normal number
    int neg;            // scale < 0: the MMA negates q
    unsigned int wait_limit;
};

// Over a paged pool, units cut into pieces of their key tiles (schedule below).
struct PagedPrefillParams : PrefillParams {
    const int32_t *table;    // [B, max_blocks]
    const int32_t *kv_lens;  // [B] positions of the pool that a sequence attends
    float *ws_o;             // [2 * CTAs] partial O (unnormalised), see Partial
    float *ws_ml;            // [2 * CTAs, rows of a unit, 2] partial (m in log2 units, l)
    int4 *split;             // [CTAs] split units, see MergeParams
    int lg, max_blocks, num_blocks;
    int box, box_lg;         // rows of a copy, min(block size, 128), and their log2
    int rows;                // query rows of a tile, hpg * tpt
    int q_bytes;             // bytes of a query tile's copy
    // A unit of at most few_tok tokens (32 query rows) has them four times in
    // its tile, 32 lanes each, and every warp of the softmax takes a quarter of a
    // key tile's columns for its copy: four partial results that are joined.
    int few_tok, few_bytes;  // (0: no such units, as at D = 256 or hpg > 32)
    int tpu_lg;              // log2 of a unit's tokens
    int causal;              // token t sees up to itself; else the whole pool rows
    int w1, w2, cost_piece;  // costs, see UnitSeq
    int min_range;           // cost of a CTA's range at least
};

// One unit of work as its readers see it.
struct Unit {
    int row0;    // first packed row of the sequence
    int len;     // its length
    int t0;      // first token of the unit
    int kvh;     // K/V head
    int h0;      // first query head
    int kbeg;    // first key of the unit's key tiles
    int n[2];    // key tiles of each query tile; n[0] = 0 ends the list
};
// A piece of one over a paged pool: n[0] < 0 ends the list.
struct PagedUnit : Unit {
    int b;       // row of the block table
    int shift;   // cached positions before token 0 (causal), or all of them
    int kend;    // end of the piece's keys
    int slot;    // workspace slot of its partial result; -1: it is a whole unit
    int few;     // its rows are in the tile four times
};
template <bool PG>
using ParamsOf = std::conditional_t<PG, PagedPrefillParams, PrefillParams>;
struct NoMap {};
template <bool PG>
using QuarterMap = std::conditional_t<PG, CUtensorMap, NoMap>;  // of q, a few_tok box
template <bool PG>
using UnitOf = std::conditional_t<PG, PagedUnit, Unit>;

// A place in a ring of N slots from slot OFF: the slot and the parity of its
// present fill (counted up: a division by N of every place took a tenth of the
// time).
template <int N_, int OFF>
struct Ring {
    static constexpr int N = N_;
    int slot = OFF;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++slot == OFF + N) {
            slot = OFF;
            parity ^= 1;
        }
    }
};

// The same for the copy warp that fills the ring, with its fills counted.
template <int N_, int OFF_>
struct CopyRing {
    static constexpr int N = N_, OFF = OFF_;
    int slot = OFF_, pos = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        ++pos;
        if (++slot >= OFF + N) {
            slot -= N;
            parity ^= 1;
        }
    }
};

template <int D, bool PG = false>
struct PfCfg {
    static constexpr int NQ = D == 256 ? 1 : 2;         // query tiles
    static constexpr int SLABS = D / 64;
    static constexpr int QT = SLABS * kSlab;            // one query tile
    static constexpr int KC = D < 128 ? D : 128;        // head dims of a ring slot
    static constexpr int CPT = D / KC;                  // slots per K (or V) tile
    static constexpr int SLOT = KC / 64 * kSlab;
    static constexpr int FIXED = NQ * QT + 1024 + 2048;
    static constexpr int NS_FIT = (kSmemMax - FIXED) / SLOT;
    static constexpr int NS = NS_FIT > 10 ? 10 : NS_FIT;  // ring slots
    // the first four warps are a warpgroup of their own; with two query tiles
    // it hands registers to the softmax warpgroups
    static constexpr int SOFT0 = 4;                     // first softmax warp
    static constexpr int THREADS = 32 * SOFT0 + 128 * NQ;
    [[maybe_unused]] static constexpr int REGS_SERVICE = 88, REGS_SOFT = 208;  // 128 x 88 + 256 x 208 = 384 x 168
    static constexpr int off_q = 0;
    static constexpr int off_ring = NQ * QT;
    static constexpr int off_bar = off_ring + NS * SLOT;
    static constexpr int nbar = 2 * NS + 2 * 2 + 3 * 2 + 2 * kDesc + 1 + 2 + (PG ? 1 : 0);
    static constexpr int off_misc = off_bar + nbar * 8;          // tmem base, abort flag
    static constexpr int off_unit = (off_misc + 32 + 15) / 16 * 16;
    static constexpr int off_cnt = off_unit + kDesc * (int)sizeof(UnitOf<PG>);
    static constexpr int off_sum = off_cnt + 2 * kBuckets * 4;
    static constexpr int bytes = off_sum + 64;
    static constexpr int alloc = bytes + 1024;
    // Two query tiles: one ring, K0 V0 K1 V1 ..., which each MMA warp takes
    // whole.  One: a ring of K and one of V, each with a copy warp and an MMA
    // warp of its own (one copy warp for both took some 2700 cycles a key tile,
    // longer than its MMAs).  Either way a slot's waits see every fill in
    // order: a barrier's parity cannot tell a fill from the one two before.
    static constexpr int KN = NQ == 2 ? NS : NS - CPT, VN = NQ == 2 ? NS : CPT;
    using KRing = Ring<KN, 0>;
    using VRing = Ring<VN, NQ == 2 ? 0 : KN>;
    // Over a pool, where a slot's boxes are a lane's each (a copy warp each for K and
    // V at D = 64 and 128: 8192 tokens of 64 heads over 8 of 128 950 us for 800).
    using KCopies = CopyRing<KN, 0>;
    using VCopies = CopyRing<VN, NQ == 2 ? 0 : KN>;
    static_assert(NS > 2 * CPT && NS >= 4, "the ring holds more than one K and one V tile");
    static_assert(alloc <= kSmemMax, "shared memory");
    // TMEM: S0, S1 (128 columns each; P over the first 64), then O per tile
    static constexpr int O0 = 256;
    static_assert(O0 + NQ * D <= 512, "tensor memory");
};

__device__ __forceinline__ void pf_error(unsigned int *err, unsigned int code) { atomicCAS(err, 0u, code); }

// A bounded wait by one lane.  (The copies' end, after a role gave up; mbar_wait
// there has the compiler lay the whole kernel out otherwise: 8192 tokens of 64
// heads over 8 of 128 724 us with this, 742 with that.)
__device__ __forceinline__ bool pf_wait(uint64_t *bar, uint32_t parity, volatile int *abort_flag) {
    for (uint32_t it = 0; it < KVATTN_SPIN_LIMIT; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((it & 255u) == 255u && *abort_flag) return false;
    }
    *abort_flag = 1;
    return false;
}

// D[tmem] (+)= A[tmem] * B[smem], bf16 inputs (A packed two to a column), fp32 accumulate.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                             uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// Warp: 32 consecutive 32-bit columns of this warp's 32 TMEM lanes.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Warp: 16 packed columns.
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

__device__ __forceinline__ float max_of(const float (&x)[32]) {
    float mx[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) mx[i] = max3(x[i], x[4 + i], x[8 + i]);
#pragma unroll
    for (int c = 12; c < 28; c += 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], x[c + i], x[c + 4 + i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], x[28 + i]);
    return fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
}

// 32 bytes, a whole sector, from one thread (dst 32-byte aligned).
__device__ __forceinline__ void st_global_32b(void *dst, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

__device__ __forceinline__ void ld_global_32b(const float *src, float (&v)[8]) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(src)
                 : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// (by a warp) a row of 32 V values times f, V consecutive ones of each lane from dst on.
template <int V>
__device__ __forceinline__ void store_row(uint16_t *dst, const float *o, float f) {
    uint32_t w[V / 2];
#pragma unroll
    for (int k = 0; k < V / 2; ++k) w[k] = bf16x2_of(o[2 * k] * f, o[2 * k + 1] * f);
    if constexpr (V == 2)
        *reinterpret_cast<uint32_t *>(dst) = w[0];
    else if constexpr (V == 4)
        *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    else
        *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Where a row of a workspace slot begins, and how far from eight values of it to the
// next eight: a thread stores its own row, and with eight values of one row beside
// those of the next a warp's stores are whole lines (at D = 64, 128: 21 single tokens
// and 3 x 256 of 32 heads over 8 of 128 68 us for 74; at D = 256, where the compiler
// then lays the softmax out worse, 8192 tokens of 16 heads over 1 443 for 415).  With
// few rows a warp stores and loads a row.
template <int D, bool FEW>
struct Partial {
    static constexpr bool WHOLE = FEW || D == 256;  // rows in one piece
    static constexpr int ROWS = (D == 256 ? 1 : 2) * kRows, STEP = WHOLE ? 8 : ROWS * 8;
    static __device__ __forceinline__ size_t row(int slot, int r) {
        return WHOLE ? ((size_t)slot * ROWS + r) * D : (size_t)slot * ROWS * D + (size_t)r * 8;
    }
    static __device__ __forceinline__ size_t ml(int slot, int r) { return ((size_t)slot * ROWS + r) * 2; }
};

// (by a warp) 128 bytes of each lane's row, w, to off[r] (lane 4 i + r's) from dst on:
// four lanes exchange their rows' pieces of 32 bytes, so that they store whole lines
// together.  off < 0: nobody's row.
__device__ __forceinline__ void store_lines(void *dst, const long long (&off)[4], uint32_t (&w)[32]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o <= 2; o *= 2) {
        const bool up = lane & o;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c & o) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t &a = w[c * 8 + i], &b = w[(c + o) * 8 + i];
                const uint32_t x = __shfl_xor_sync(0xffffffffu, up ? a : b, o);
                if (up) a = x;
                else b = x;
            }
        }
    }
    char *mine = static_cast<char *>(dst) + (lane & 3) * 32;
#pragma unroll
    for (int r = 0; r < 4; ++r)
        if (off[r] >= 0) st_global_32b(mine + off[r], w + r * 8);
}

// A published unit, the same in every lane.
template <class U>
__device__ __forceinline__ U read_unit(const U &from) {
    U u;
    const int *src = reinterpret_cast<const int *>(&from);
    int *dst = reinterpret_cast<int *>(&u);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(U) / 4); ++i) dst[i] = __shfl_sync(0xffffffffu, src[i], 0);
    return u;
}

__device__ __forceinline__ bool ends_list(const Unit &u) { return u.n[0] == 0; }
__device__ __forceinline__ bool ends_list(const PagedUnit &u) { return u.n[0] < 0; }
__device__ __forceinline__ bool few_of(const Unit &) { return false; }
__device__ __forceinline__ bool few_of(const PagedUnit &u) { return u.few; }

// First of the unit's key tiles that query tile s attends: its window may start
// behind whole tiles that the first query tile needs (one of ten in a window of
// 1024 with 128 tokens a tile: three prompts of 16 heads of 64, 78.3 us with them
// computed, 74.1 without; full prompts lose 0.4 % to the test).
__device__ __forceinline__ int first_tile(const PrefillParams &p, const Unit &u, int s) {
    return max(0, u.t0 + s * p.tpt + 1 - p.window - u.kbeg) / kRows;
}
// Where the keys of token t end.
__device__ __forceinline__ int key_end(const PagedPrefillParams &p, int shift, int t) {
    return shift + (p.causal ? t + 1 : 0);
}
__device__ __forceinline__ int first_tile(const PagedPrefillParams &p, const PagedUnit &u, int s) {
    return max(0, key_end(p, u.shift, u.t0 + s * p.tpt) - p.window - u.kbeg) / kRows;
}
// First position that a token of the unit attends: rows before it are not read,
// or, in its tile, zeroed.
__device__ __forceinline__ int first_key(const PagedPrefillParams &p, const PagedUnit &u) {
    return max(0, key_end(p, u.shift, u.t0) - p.window);
}
// Keys of the whole sequence.
__device__ __forceinline__ int seq_keys(const PrefillParams &, const Unit &u) { return u.len; }
__device__ __forceinline__ int seq_keys(const PagedPrefillParams &p, const PagedUnit &u) {
    return key_end(p, u.shift, u.len - 1);
}
// Keys of the unit's key tiles that query tile s attends at most.
__device__ __forceinline__ int last_key(const PrefillParams &p, const Unit &u, int s) {
    return min(u.t0 + (s + 1) * p.tpt, u.len) - u.kbeg;
}
__device__ __forceinline__ int last_key(const PagedPrefillParams &p, const PagedUnit &u, int s) {
    return min(u.kend, key_end(p, u.shift, min(u.t0 + (s + 1) * p.tpt, u.len) - 1)) - u.kbeg;
}

// Length of sequence b (0 where its bounds are not 0 <= cu[b] <= cu[b+1] <= N).
__device__ __forceinline__ int pf_len(const PrefillParams &p, int b, int *row0) {
    const int a = p.cu[b], e = p.cu[b + 1];
    *row0 = a;
    return (a < 0 || e < a || e > p.N) ? -1 : e - a;
}

// ------------------------------------------------- schedule over a paged pool

// Where a CTA is in its range of the call's cost.
struct PagedRange {
    long long x0, x1;  // its range
    long long total;   // of all
    long long u0;      // where the unit (seq, hh, blk) starts
    UnitSeq seq;
    int row0;          // packed row of the sequence's token 0
    int b, hh, blk;
    int ranges;
    int4 record;       // its last unit, if others go on with it (see merge_kernel)
};

// Sequence b: its tokens that attend something, their first packed row, and how
// many before them (*none) attend nothing and become zeros.  False: bounds that
// are not 0 <= cu[b] <= cu[b+1] <= N (nothing is done), or a length outside the
// table row (as 0).
__device__ __forceinline__ bool load_seq(const PagedPrefillParams &p, int b, UnitSeq *s, int *row0, int *none) {
    const int a = p.cu[b], e = p.cu[b + 1];
    int kv = p.kv_lens[b];
    bool ok = kv >= 0 && kv <= p.max_blocks << p.lg;
    if (!ok) kv = 0;
    int n = e - a;
    if (a < 0 || e < a || e > p.N) {
        ok = false;
        n = 0;
    }
    *none = p.causal ? max(0, n - kv) : kv == 0 ? n : 0;
    *row0 = a + *none;
    s->len = n - *none;
    s->shift = p.causal ? kv - s->len : kv;
    return ok;
}

// Rows that attend nothing, dealt out by sequence.
__device__ __forceinline__ void zero_rows(const PagedPrefillParams &p, int D, int thread, int threads) {
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        UnitSeq s;
        int row0, none;
        load_seq(p, b, &s, &row0, &none);
        uint4 *dst = reinterpret_cast<uint4 *>(p.out + (size_t)(row0 - none) * p.Hq * D);
        const size_t n = none > 0 ? (size_t)none * p.Hq * D / 8 : 0;
        for (size_t i = thread; i < n; i += threads) dst[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// (by all threads) this CTA's range: prefix sums of the sequences' costs, as many
// consecutive ones to a thread as it takes; the thread that has the range's start
// leaves its sequence in shared memory.
__device__ __forceinline__ PagedRange find_range(const PagedPrefillParams &p, int heads, long long *sm, int threads) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *found = reinterpret_cast<int *>(sm + 33);
    const int per = (p.B + threads - 1) / threads;
    const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
    PagedRange r = {};
    r.seq.causal = p.causal;
    r.seq.window = p.window;
    r.seq.tpu_lg = p.tpu_lg;
    r.seq.tpt = p.tpt;
    r.seq.w1 = p.w1;
    r.seq.w2 = p.w2;
    r.seq.piece = p.cost_piece;
    auto cost_of = [&](int b) {
        int none;
        if (!load_seq(p, b, &r.seq, &r.row0, &none) && blockIdx.x == 0) pf_error(p.err, DEV_ERR_BOUNDS);
        return r.seq.len > 0 ? blocks_cost(r.seq, seq_blocks(r.seq)) * heads : 0LL;
    };
    long long mine = 0;
    for (int b = b0; b < b1; ++b) mine += cost_of(b);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) sm[warp] = incl;
    __syncthreads();
    long long before = incl - mine;
    for (int w = 0; w < threads / 32; ++w) {
        if (w < warp) before += sm[w];
        r.total += sm[w];
    }
    const long long most = r.total < 1LL << 31 ? (long long)((unsigned)r.total / (unsigned)p.min_range)
                                               : r.total / p.min_range;
    r.ranges = most < 1 ? 1 : most < gridDim.x ? (int)most : (int)gridDim.x;
    if ((int)blockIdx.x < r.ranges && r.total > 0) {
        r.x0 = range_start(r.total, r.ranges, blockIdx.x);
        r.x1 = range_start(r.total, r.ranges, blockIdx.x + 1);
        if (before <= r.x0 && r.x0 < before + mine) {
            int b = b0;
            if (per > 1)
                for (;; ++b) {
                    const long long c = cost_of(b);
                    if (r.x0 < before + c) break;
                    before += c;
                }
            sm[32] = before;
            found[0] = b;
            found[1] = r.row0;
            found[2] = r.seq.len;
            found[3] = r.seq.shift;
        }
    }
    __syncthreads();
    if (r.x0 < r.x1 && warp == 3) {
        r.b = found[0];
        r.row0 = found[1];
        r.seq.len = found[2];
        r.seq.shift = found[3];
        const long long off = r.x0 - sm[32], each = blocks_cost(r.seq, seq_blocks(r.seq));
        r.hh = off < 1LL << 31 && each < 1LL << 31 ? (int)((unsigned)off / (unsigned)each) : (int)(off / each);
        r.blk = block_at_cost(r.seq, off - r.hh * each);
        r.u0 = sm[32] + r.hh * each + blocks_cost(r.seq, r.blk);
    }
    return r;
}

// (by a warp) the CTA's next piece.
__device__ __forceinline__ void next_piece(const PagedPrefillParams &p, PagedRange &r, int tpu, int heads,
                                           PagedUnit *u) {
    const int lane = threadIdx.x & 31;
    u->n[0] = -1;
    while (r.u0 < r.x1) {
        if (r.blk == seq_blocks(r.seq)) {
            r.blk = 0;
            if (++r.hh == heads) {
                r.hh = 0;
                unsigned hit = 0;
                for (int from = r.b + 1; from < p.B && !hit; from += 32) {  // the next that has tokens
                    UnitSeq s = r.seq;
                    int row0 = 0, none;
                    s.len = 0;
                    if (from + lane < p.B) load_seq(p, from + lane, &s, &row0, &none);
                    hit = __ballot_sync(0xffffffffu, s.len > 0);
                    if (hit) {
                        const int src = __ffs(hit) - 1;
                        r.b = from + src;
                        r.row0 = __shfl_sync(0xffffffffu, row0, src);
                        r.seq.len = __shfl_sync(0xffffffffu, s.len, src);
                        r.seq.shift = __shfl_sync(0xffffffffu, s.shift, src);
                    }
                }
                if (!hit) {  // (not reached: the range ends with the last unit)
                    r.u0 = r.x1;
                    return;
                }
            }
        }
        const int nt = unit_tiles(r.seq, r.blk), w = unit_weight(r.seq, r.blk);
        const int ta = tiles_before(r.u0, nt, w, p.cost_piece, r.x0);
        const int tb = tiles_before(r.u0, nt, w, p.cost_piece, r.x1);
        if (ta < tb) {
            const int first = unit_first(r.seq, r.blk);
            u->row0 = r.row0;
            u->len = r.seq.len;
            u->t0 = r.blk * tpu;
            u->kvh = r.hh / p.passes;
            u->h0 = u->kvh * p.G + (r.hh - u->kvh * p.passes) * p.hpg;
            u->kbeg = (first + ta) * kRows;
            u->b = r.b;
            u->shift = r.seq.shift;
            const int stop = min(u->t0 + tpu, u->len);
            u->few = stop - u->t0 <= p.few_tok;  // (both query tiles have the same rows then)
            u->kend = min((first + tb) * kRows, key_end(p, u->shift, stop - 1));
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                u->n[s] = 0;
                if (s * p.tpt < tpu && u->t0 + s * p.tpt < u->len) {
                    const int n = max(0, last_key(p, *u, s) + kRows - 1) / kRows;
                    if (first_tile(p, *u, s) < n) u->n[s] = n;
                }
            }
            if (u->few && p.tpt < tpu) u->n[1] = u->n[0];
            u->slot = -1;
            if (ta > 0) {
                u->slot = 2 * blockIdx.x;
            } else if (tb < nt) {
                u->slot = 2 * blockIdx.x + 1;
                const int last = range_of(r.total, r.ranges, r.u0 + p.cost_piece + (long long)w * (nt - 1));
                r.record = make_int4(u->row0 + u->t0, stop - u->t0, u->h0, last - (int)blockIdx.x + 1);
            }
        }
        r.u0 += p.cost_piece + (long long)w * nt;
        ++r.blk;
        if (ta < tb) return;
    }
}

// PG: over a paged pool; FEW: with units of few rows (by their own loop over key
// tiles, beside which the other spills registers: 8192 tokens of 64 heads over 8 of
// 128 812 us without it, 894 with).
template <int D, bool PG, bool FEW>
__global__ void __launch_bounds__(PfCfg<D, PG>::THREADS, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv, const ParamsOf<PG> p,
                   const __grid_constant__ QuarterMap<PG> tmq4) {
    using C = PfCfg<D, PG>;
    using Unit = UnitOf<PG>;
    static_assert(!FEW || (PG && C::NQ == 2), "few rows: two query tiles over a pool");
    constexpr int NQ = C::NQ, NS = C::NS, CPT = C::CPT;

    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *qbuf = smem + C::off_q;
    uint8_t *ring = smem + C::off_ring;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::off_bar);
    uint64_t *slot_full = bars, *slot_empty = slot_full + NS;
    uint64_t *q_full = slot_empty + NS, *q_empty = q_full + 2;
    // s_full, p_full, pv_done: of query tile s (two tiles) or of S buffer s (one)
    uint64_t *s_full = q_empty + 2, *p_full = s_full + 2, *pv_done = p_full + 2;
    uint64_t *u_full = pv_done + 2, *u_empty = u_full + kDesc, *drain = u_empty + kDesc;
    uint64_t *turn = drain + 1;  // the MMA warps' turns
    [[maybe_unused]] uint64_t *join = turn + 2;  // (few rows) the softmax warps' steps of a join
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::off_misc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::off_misc + 16);
    [[maybe_unused]] volatile int *joined = abort_flag + 1;  // (few rows) units joined so far
    Unit *units = reinterpret_cast<Unit *>(smem + C::off_unit);
    int *cnt = reinterpret_cast<int *>(smem + C::off_cnt);  // [kBuckets] full, [kBuckets] rest
    unsigned long long *sum_pairs = reinterpret_cast<unsigned long long *>(smem + C::off_sum);
    int *max_nb = reinterpret_cast<int *>(sum_pairs + 1);

    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int tpu = NQ * p.tpt;          // tokens of a unit
    const int heads = p.Hkv * p.passes;  // units of one block of tokens

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&slot_full[s], 1);
            mbar_init(&slot_empty[s], NQ);  // K and V tiles serve every query tile
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 1);
            mbar_init(&q_empty[s], 1);
            mbar_init(&s_full[s], 1);
            mbar_init(&p_full[s], 4);
            mbar_init(&pv_done[s], 1);
            mbar_init(&turn[s], 1);
        }
        for (int s = 0; s < kDesc; ++s) {
            mbar_init(&u_full[s], 1);
            // readers of a unit: the copy warps, the MMA warps, the softmax warps
            mbar_init(&u_empty[s], (NQ == 2 ? 3 : 4) + 4 * NQ);
        }
        mbar_init(drain, 2);  // warps 1 and 2
        if (FEW) {
            mbar_init(join, 4 * NQ);
            *joined = 0;
        }
        *abort_flag = 0;
        *sum_pairs = 0;
        *max_nb = 0;
        fence_barrier_init();
        prefetch_tmap(&tmq);
        prefetch_tmap(&tmk);
        prefetch_tmap(&tmv);
    }
    for (int i = tid; i < 2 * kBuckets; i += C::THREADS) cnt[i] = 0;
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait_prior();  // inputs and lengths may come from the previous kernel

    // ------------------------------------------------ the work list's buckets
    long long total = 0;
    int width = 0, nbk = 0;
    PagedRange range;  // (paged: this CTA's range of the call's cost, and where it starts)
    if constexpr (PG) {
        range = find_range(p, heads, reinterpret_cast<long long *>(cnt), C::THREADS);
    } else {
    {
        unsigned long long s = 0;
        int m = 0;
        for (int b = tid; b < p.B; b += C::THREADS) {
            int row0;
            const int len = pf_len(p, b, &row0);
            if (len < 0) {
                if (blockIdx.x == 0) pf_error(p.err, DEV_ERR_BOUNDS);
                continue;
            }
            const int nb = (len + tpu - 1) / tpu;
            s += nb;
            m = max(m, nb);
        }
        if (m > 0) {
            atomicAdd(sum_pairs, s);
            atomicMax(max_nb, m);
        }
    }
    __syncthreads();
    total = (long long)*sum_pairs * heads;
    const int mnb = *max_nb;
    // one wave of units: any order does
    width = total <= gridDim.x ? max(mnb, 1) : (mnb + kBuckets - 1) / kBuckets;
    nbk = width > 0 ? (mnb + width - 1) / width : 0;
    if (nbk > 1) {
        for (int b = tid; b < p.B; b += C::THREADS) {
            int row0;
            const int len = pf_len(p, b, &row0);
            if (len <= 0) continue;
            const int nb = (len + tpu - 1) / tpu;
            const int k = nb / width;
            // buckets below k hold `width` blocks of this sequence, bucket k the rest
            if (k > 0) atomicAdd(&cnt[k - 1], 1);
            if (nb % width) atomicAdd(&cnt[kBuckets + k], nb % width);
        }
        __syncthreads();
    }
    }

    const uint32_t ring_s = smem_u32(ring), qbuf_s = smem_u32(qbuf);

    const uint32_t wlim = p.wait_limit ? p.wait_limit : KVATTN_SPIN_LIMIT;
    // (by a whole warp) unit k of this CTA's list
    auto next_unit = [&](int k, Unit *u) {
        if (!mbar_wait_warp(&u_full[k % kDesc], (uint32_t)((k / kDesc) & 1), abort_flag)) return false;
        *u = read_unit(units[k % kDesc]);
        __syncwarp();
        if (lane == 0) mbar_arrive(&u_empty[k % kDesc]);
        return true;
    };
    // (by a whole warp) one slot's copies: a uniform wait, then one lane issues
    [[maybe_unused]] int fills = 0;  // (packed rows) slots filled by this warp
    auto issue = [&](const void *tm, int c, int head, int row, auto &r) -> bool {
        const int slot = r.slot;
        if (fills >= r.N && !mbar_wait_warp(&slot_empty[slot], r.parity ^ 1, abort_flag)) return false;
        if (elect_one()) {
            mbar_arrive_expect_tx(&slot_full[slot], C::SLOT);
#pragma unroll
            for (int sl = 0; sl < C::KC / 64; ++sl)
                tma_load_3d_plain(ring + slot * C::SLOT + sl * kSlab, tm, &slot_full[slot],
                                  c * C::KC + sl * 64, head, row);
        }
        __syncwarp();
        ++fills;
        r.next();
        return true;
    };
    // (paged) the same from the boxes of a tile's blocks, a lane each
    struct Boxes {
        int z, row;   // the lane's block and K/V head in the pool, its first row there
        bool mine;    // the lane has one
        int bytes;    // of all, per 64 head dims
    };
    [[maybe_unused]] auto issue_paged = [&](const void *tm, int c, const Boxes &t, auto &r) -> bool {
        if constexpr (PG) {
            const int slot = r.slot;
            if (r.pos >= r.N && !mbar_wait_warp(&slot_empty[slot], r.parity ^ 1, abort_flag)) return false;
            if (lane == 0) mbar_arrive_expect_tx(&slot_full[slot], t.bytes * (C::KC / 64));
            __syncwarp();
            if (t.mine) {
#pragma unroll
                for (int sl = 0; sl < C::KC / 64; ++sl)
                    tma_load_3d_plain(ring + slot * C::SLOT + sl * kSlab + lane * p.box * 128, tm, &slot_full[slot],
                                      c * C::KC + sl * 64, t.row, t.z);
            }
            __syncwarp();
            r.next();
        }
        return true;
    };
    // (paged) The blocks of a unit's tiles, 32 table entries at a time and 32 ahead,
    // so that a copy warp does not wait for memory at each tile.
    struct Blocks {
        int now, then;  // entry first + lane of the unit's row, and first + 32 + lane
        int first;
    };
    [[maybe_unused]] auto entry = [&](const Unit &u, int e) -> int {
        if constexpr (PG) return e <= (u.kend - 1) >> p.lg ? p.table[(size_t)u.b * p.max_blocks + e] : 0;
        return 0;
    };
    [[maybe_unused]] auto blocks_of = [&](const Unit &u) -> Blocks {
        Blocks x = {};
        if constexpr (PG) {
            x.first = u.kbeg >> p.lg;
            x.now = entry(u, x.first + lane);
            x.then = entry(u, x.first + 32 + lane);
        }
        return x;
    };
    // the boxes of the unit's rows of the tile at position kb (whose blocks are in one
    // group of 32); a block that is none reads as zeros, from past the pool
    [[maybe_unused]] auto boxes_at = [&](const Unit &u, Blocks &x, int kb) -> Boxes {
        Boxes t = {};
        if constexpr (PG) {
            int e = (kb >> p.lg) - x.first;
            if (e >= 32) {
                x.first += 32;
                e -= 32;
                x.now = x.then;
                x.then = entry(u, x.first + 32 + lane);
            }
            const int blk = __shfl_sync(0xffffffffu, x.now, (e + lane) & 31);
            const int b0 = max(0, first_key(p, u) - kb) >> p.box_lg;
            const int b1 = (min(kRows, u.kend - kb) + p.box - 1) >> p.box_lg;
            t.mine = lane >= b0 && lane < b1;
            t.bytes = (b1 - b0) << p.box_lg << 7;
            t.row = kb & ((1 << p.lg) - 1);
            const bool bad = blk < 0 || blk >= p.num_blocks;
            if (t.mine && bad) pf_error(p.err, DEV_ERR_BOUNDS);
            t.z = bad ? p.num_blocks * p.Hkv : blk * p.Hkv + u.kvh;
        }
        return t;
    };
    // (by one lane) the last fills of a ring of n slots from slot `off` have landed
    auto landed = [&](int n, int off) {
        volatile int never = 0;
        for (int i = fills > n ? fills - n : 0; i < fills; ++i)
            pf_wait(&slot_full[off + i % n], (uint32_t)((i / n) & 1), &never);
    };
    // (paged, by one lane) the last fills of r have landed
    [[maybe_unused]] auto landed_paged = [&](const auto &r) {
        volatile int never = 0;
        for (int pos = r.pos - 1, i = 0; pos >= 0 && i < r.N; --pos, ++i)
            pf_wait(&slot_full[r.OFF + pos % r.N], (uint32_t)((pos / r.N) & 1), &never);
    };
    // A walk over the key tiles of all units (where a copy warp has K or V alone).
    struct Walk {
        Unit u;
        int k = -1, g = -1;  // unit, key tile of the CTA
        int j = 0;           // key tile of the unit
        bool done = false;
    };
    auto step = [&](Walk &w) -> bool {
        ++w.g;
        if (w.k >= 0 && ++w.j < (PG && NQ == 2 ? max(w.u.n[0], w.u.n[1]) : w.u.n[0])) return true;
        w.j = 0;
        if (!next_unit(++w.k, &w.u)) return false;
        w.done = ends_list(w.u);
        return true;
    };
    if (warp < C::SOFT0) {
    if constexpr (NQ == 2) regs_dec<C::REGS_SERVICE>();

    // ============================================================ work list
    if (warp == 3) {
        bool ok = true;
        // the walk: bucket kb holds pairs [pb0, pb0 + its count), `cover` sequences reach past it
        int kb = nbk;
        long long pb0 = 0, pbn = 0;
        int cover = 0;
        int sb = 0;                  // the bucket's scan: sequences before sb hold sp pairs
        long long sp = 0;
        auto find = [&](long long k, Unit *u) {
            if constexpr (PG) {
                next_piece(p, range, tpu, heads, u);
            } else {
            const long long rank = k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
            if (rank >= total) {
                u->n[0] = 0;
                return;
            }
            const long long pair = rank / heads;
            const int hh = (int)(rank - pair * heads);
            while (pair >= pb0 + pbn) {  // the next bucket down
                pb0 += pbn;
                --kb;
                if (nbk == 1) {
                    pbn = (long long)*sum_pairs;
                } else {
                    cover += cnt[kb];
                    pbn = (long long)cover * width + cnt[kBuckets + kb];
                }
                sb = 0;
                sp = 0;
            }
            const long long off = pair - pb0;
            for (;; sb += 32) {  // the chunk of 32 sequences that holds the pair
                const int b = sb + lane;
                int row0 = 0, len = 0, mine = 0;
                if (b < p.B) {
                    len = max(pf_len(p, b, &row0), 0);
                    mine = min(max((len + tpu - 1) / tpu - kb * width, 0), width);
                }
                int incl = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o) incl += v;
                }
                const long long before = sp + incl - mine;
                const unsigned hit = __ballot_sync(0xffffffffu, off >= before && off < before + mine);
                if (hit) {
                    const int src = __ffs(hit) - 1;
                    u->row0 = __shfl_sync(0xffffffffu, row0, src);
                    u->len = __shfl_sync(0xffffffffu, len, src);
                    const int blk = kb * width + (int)(off - __shfl_sync(0xffffffffu, before, src));
                    u->t0 = blk * tpu;
                    break;
                }
                sp += __shfl_sync(0xffffffffu, incl, 31);
                if (sb + 32 >= p.B) {  // (not reached: every pair has a sequence)
                    u->n[0] = 0;
                    return;
                }
            }
            u->kvh = hh / p.passes;
            u->h0 = u->kvh * p.G + (hh - u->kvh * p.passes) * p.hpg;
            u->kbeg = max(0, u->t0 + 1 - p.window);
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int a = u->t0 + s * p.tpt, e = min(a + p.tpt, u->len);
                u->n[s] = (s < NQ && a < e) ? (e - u->kbeg + kRows - 1) / kRows : 0;
            }
            }
        };
        // publishes unit k; with one query tile only if its place is free, unless it must
        auto publish = [&](int k, const Unit &u, bool must, bool *done) -> bool {
            uint64_t *place = &u_empty[k % kDesc];
            const uint32_t parity = (uint32_t)((k / kDesc - 1) & 1);
            *done = false;
            if (k >= kDesc) {
                if (!must && !__all_sync(0xffffffffu, mbar_test(place, parity))) return true;
                if (!mbar_wait_warp(place, parity, abort_flag)) return false;
            }
            if (lane == 0) {
                units[k % kDesc] = u;
                mbar_arrive(&u_full[k % kDesc]);
            }
            __syncwarp();
            *done = true;
            return true;
        };
        [[maybe_unused]] typename C::VCopies vcopies;
        Unit u = {};
        int k = 0;
        bool more = true, done;  // the last unit published does not end the list
        find(0, &u);
        auto pump = [&](bool must) {  // publishes the next unit and finds the one after
            if (!more) return true;
            if (!publish(k, u, must, &done)) return false;
            if (done) {
                more = !ends_list(u);
                ++k;
                if (more) find(k, &u);
            }
            return true;
        };
        if (NQ == 2) {
            while (ok && more) ok = pump(true);
        } else if constexpr (PG) {
            // this warp copies V, too, and publishes units as their places come free
            Walk w;
            ok = pump(true) && pump(true) && pump(true) && step(w);
            Blocks x = {};
            while (ok && !w.done) {
                if (w.j == 0) x = blocks_of(w.u);
                const Boxes t = boxes_at(w.u, x, w.u.kbeg + w.j * kRows);
                const bool last = w.j + 1 == max(w.u.n[0], w.u.n[1]);
                for (int c = 0; c < CPT && ok; ++c) ok = issue_paged(&tmv, c, t, vcopies);
                if (ok) ok = pump(last && w.k + 1 >= k);
                if (ok) ok = step(w);
            }
        } else {
            // (the same over packed rows)
            typename C::VRing rc;
            Walk w;
            ok = pump(true) && pump(true) && pump(true) && step(w);
            while (ok && !w.done) {
                for (int c = 0; c < CPT && ok; ++c)
                    ok = issue(&tmv, c, w.u.kvh, w.u.row0 + w.u.kbeg + w.j * kRows, rc);
                if (ok) ok = pump(w.j + 1 == w.u.n[0] && w.k + 1 >= k);
                if (ok) ok = step(w);
            }
        }
        if constexpr (PG) {
            if (lane == 0) p.split[blockIdx.x] = range.record;
        }
        if (!ok && lane == 0) {
            pf_error(p.err, DEV_ERR_TIMEOUT);
            *abort_flag = 1;
        }
        __syncwarp();
        named_bar_sync(kBarEndPf, C::THREADS);
        if constexpr (PG) {
            if (NQ == 1 && *abort_flag && lane == 0) landed_paged(vcopies);
        } else {
            if (NQ == 1 && *abort_flag && lane == 0) landed(C::VN, C::KN);
        }
        return;
    }

    // ================================================================== TMA
    if (warp == 0) {
        bool ok = true;
        uint32_t qn[2] = {0, 0};     // query tiles issued
        typename C::KRing rc;
        [[maybe_unused]] int joins = 0;  // units of few rows so far
        // (a count, not a barrier's phase, which says nothing to who comes late)
        [[maybe_unused]] auto joins_over = [&]() -> bool {
            for (uint32_t it = 0; it < KVATTN_SPIN_LIMIT; ++it) {
                if (__all_sync(0xffffffffu, *joined >= joins)) {
                    __threadfence_block();
                    return true;
                }
                if ((it & 255u) == 255u && __any_sync(0xffffffffu, *abort_flag)) return false;
                __nanosleep(32);
            }
            *abort_flag = 1;
            return false;
        };
        auto load_q = [&](const Unit &u) -> bool {
            if constexpr (FEW) {
                // units of few rows are joined in query tile 1's place
                if (u.few)
                    ++joins;
                else if (u.n[1] > 0 && joins > 0 && !joins_over())
                    return false;
            }
#pragma unroll(PG ? 2 : 1)
            for (int s = 0; s < NQ; ++s) {
                if (u.n[s] == 0 || (FEW && s > 0 && few_of(u))) continue;  // (few rows: one tile for both)
                if (qn[s] && !mbar_wait_warp(&q_empty[s], (qn[s] - 1) & 1, abort_flag)) return false;
                if (elect_one()) {
                    bool few = false;
                    if constexpr (PG) {
                        few = FEW && u.few;
                        mbar_arrive_expect_tx(&q_full[s], few ? 4 * p.few_bytes : p.q_bytes);
                        if (few)
#pragma unroll
                            for (int sl = 0; sl < C::SLABS; ++sl)
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    tma_load_3d_plain(qbuf + s * C::QT + sl * kSlab + c * (32 * 128), &tmq4,
                                                      &q_full[s], sl * 64, u.h0, u.row0 + u.t0);
                    } else {
                        mbar_arrive_expect_tx(&q_full[s], C::QT);
                    }
                    if (!few)
#pragma unroll
                        for (int sl = 0; sl < C::SLABS; ++sl)
                            tma_load_3d_plain(qbuf + s * C::QT + sl * kSlab, &tmq, &q_full[s], sl * 64, u.h0,
                                              u.row0 + u.t0 + s * p.tpt);
                }
                __syncwarp();
                ++qn[s];
            }
            return true;
        };
        [[maybe_unused]] typename C::KCopies kcopies;
        if constexpr (PG) {
            Walk w;
            ok = step(w);
            Blocks x = {};
            while (ok && !w.done) {
                if (w.j == 0) x = blocks_of(w.u);
                const Boxes t = boxes_at(w.u, x, w.u.kbeg + w.j * kRows);
                for (int c = 0; c < CPT && ok; ++c) ok = issue_paged(&tmk, c, t, kcopies);
                if (ok && w.j == 0) ok = load_q(w.u);
                if (NQ == 2 && ok) ok = issue_paged(&tmv, 0, t, kcopies);
                if (ok) ok = step(w);
            }
        } else if (NQ == 2) {
            Unit u;
            for (int k = 0; ok; ++k) {
                ok = next_unit(k, &u);
                if (!ok || ends_list(u)) break;
                const int n = max(u.n[0], u.n[1]);
                const int kv0 = u.row0 + u.kbeg;
                for (int j = 0; j < n && ok; ++j) {
                    ok = issue(&tmk, 0, u.kvh, kv0 + j * kRows, rc);
                    if (ok && j == 0) ok = load_q(u);
                    if (ok) ok = issue(&tmv, 0, u.kvh, kv0 + j * kRows, rc);
                }
            }
        } else {
            Walk w;
            ok = step(w);
            while (ok && !w.done) {
                for (int c = 0; c < CPT && ok; ++c)
                    ok = issue(&tmk, c, w.u.kvh, w.u.row0 + w.u.kbeg + w.j * kRows, rc);
                if (ok && w.j == 0) ok = load_q(w.u);
                if (ok) ok = step(w);
            }
        }
        if (!ok && lane == 0) {
            pf_error(p.err, DEV_ERR_TIMEOUT);
            *abort_flag = 1;
        }
        __syncwarp();
        pdl_launch_dependents();
        named_bar_sync(kBarEndPf, C::THREADS);
        if (*abort_flag && lane == 0) {
            // a role gave up: let the copies in flight land before the CTA exits
            if constexpr (PG)
                landed_paged(kcopies);
            else
                landed(C::KN, 0);
            volatile int never = 0;
            for (int s = 0; s < NQ; ++s)
                if (qn[s]) pf_wait(&q_full[s], (qn[s] - 1) & 1, &never);
        }
        return;
    }

    // ================================================================== MMA
    // With two query tiles a warp for each, so that one's waits do not drain the
    // tensor pipe of the other's MMAs.
    if (warp <= 2) {
        constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, C::KC, false, true);
        // bit 13: A enters negated (a negative scale)
        const uint32_t idesc_qk = (IDESC_QK | (p.neg ? 1u << 13 : 0u)) & ~(0x3fu << 17);
        const int s = NQ == 2 ? warp - 1 : 0;  // query tile
        bool ok = true;
        uint32_t units_q = 0;         // query tiles consumed
        uint32_t g = 0;               // key tiles so far, its last bit
        uint32_t it = 0;              // turns taken, the last bit
        bool first_turn = true;

        // S[buf] = Q_s K_j^T from the slots at r; keys past the tile's last are
        // left out, 16 at a time
        auto qk = [&](int buf, typename C::KRing r, int keys, bool last) {
            const uint32_t idesc = idesc_qk | ((uint32_t)((keys + 15) / 16 * 2) << 17);
            const uint32_t d = tmem + buf * 128;
            if (elect_one()) {
#pragma unroll
                for (int c = 0; c < CPT; ++c, r.next()) {
                    const uint64_t kd = smem_desc(ring_s + r.slot * C::SLOT, 16, 1024, 2);
                    const uint64_t qd = smem_desc(qbuf_s + s * C::QT + c * (C::KC / 64) * kSlab, 16, 1024, 2);
#pragma unroll
                    for (int kk = 0; kk < C::KC / 16; ++kk) {
                        const uint64_t o = ((kk >> 2) * kSlab + (kk & 3) * 32) >> 4;
                        umma_bf16(d, qd + o, kd + o, idesc, c != 0 || kk != 0);
                    }
                    umma_commit(&slot_empty[r.slot]);
                }
                umma_commit(&s_full[buf]);
                if (last) umma_commit(&q_empty[s]);
            }
            __syncwarp();
        };
        // O_s (+)= P[buf] V_j from the slots at r
        auto pv = [&](int buf, typename C::VRing r, int keys, bool first, int acc = -1) {
            const uint32_t a = tmem + buf * 128, d = tmem + C::O0 + (acc < 0 ? s : acc) * D;
            if (elect_one()) {
#pragma unroll
                for (int c = 0; c < CPT; ++c, r.next()) {
                    const uint64_t vd = smem_desc(ring_s + r.slot * C::SLOT, kSlab, 1024, 2);
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk) {
                        if (kk * 16 < keys)
                            umma_bf16_ts(d + c * C::KC, a + kk * 8, vd + kk * (2048 >> 4), IDESC_PV,
                                         !(first && kk == 0));
                    }
                    umma_commit(&slot_empty[r.slot]);
                }
                umma_commit(&pv_done[buf]);
            }
            __syncwarp();
        };

        if constexpr (NQ == 2) {
            Unit u;
            // The two query tiles' MMAs go out in turns, the products of one key
            // tile together: P V of the step before, then Q K^T of this one (of
            // the next unit's first key tile, too).  The query tiles then keep
            // half a period apart, each in its softmax while the other's
            // products run.  Measured at 8192 tokens, 64 heads over 8 of 128:
            // left to share the tensor cores, both finish together and both
            // wait for both, 1009 us; in turns 869 us.
            typename C::KRing rc;    // the next slot that this warp has not waited for
            auto slot_ready = [&]() {
                const bool go = mbar_wait_warp(&slot_full[rc.slot], rc.parity, abort_flag);
                rc.next();
                return go;
            };
            int owed = 0;            // the step before: 1 its P V is due, 2 its V tile was not needed
            int owed_keys = 0;
            bool owed_first = false;
            // (key tiles from j0 to n are the query tile's; j = nmax: the last P V alone)
            auto turn_of = [&](int j0, int n, int nmax, int j, int end) {
                // (one uniform wait after the other: what comes early is waited for
                // while the other tile's MMAs are still running)
                bool go = true;
                const auto rv = rc;
                if (owed) go = slot_ready();
                const auto rk = rc;
                if (go && j < nmax) go = slot_ready();
                if (go && j == j0 && j < n) go = mbar_wait_warp(&q_full[s], units_q++ & 1, abort_flag);
                if (go && (s == 1 || !first_turn)) go = mbar_wait_warp(&turn[s], s == 0 ? it ^ 1 : it, abort_flag);
                if (go && owed == 1) go = mbar_wait_warp(&p_full[s], g ^ 1, abort_flag, wlim);
                if (!go) return false;
                tc_fence_after();
                if (owed == 1)
                    pv(s, rv, owed_keys, owed_first);
                else if (owed == 2 && lane == 0)
                    mbar_arrive(&slot_empty[rv.slot]);
                owed = 0;
                if (j0 <= j && j < n) {
                    const int keys = min(kRows, end - j * kRows);
                    qk(s, rk, keys, j == n - 1);
                    g ^= 1;
                    owed = 1;
                    owed_keys = keys;
                    owed_first = j == j0;
                } else if (j < nmax) {
                    if (lane == 0) mbar_arrive(&slot_empty[rk.slot]);
                    owed = 2;
                }
                if (lane == 0) mbar_arrive(&turn[s ^ 1]);
                it ^= 1;
                first_turn = false;
                return true;
            };
            // With units of few rows.  The even key tiles of one go through S and O of
            // query tile 0 and its softmax warps, the odd ones through those of query
            // tile 1; warp 1 issues Q K^T of all, warp 2 P V of all, as at D = 256, so
            // that the chains of copy, Q K^T, softmax, P V of several key tiles overlap
            // (one chain alone leaves memory idle: 64 requests of 16 heads of 64 over up
            // to 2048 states 96 us).  Each gives its slots back for both.
            uint32_t tiles[2] = {0, 0};  // through S buffer 0 and 1 so far
            bool after_few = false;
            [[maybe_unused]] auto turn_few = [&](bool visit, bool own, bool first, bool last, int keys) {
                bool go = true;
                const auto rv = rc;
                if (owed) go = slot_ready();
                const auto rk = rc;
                if (go && visit) go = slot_ready();
                if (go && own && first) go = mbar_wait_warp(&q_full[s], units_q++ & 1, abort_flag);
                if (go && own && after_few) {  // (P V of the last few rows was the other warp's)
                    after_few = false;
                    if (tiles[s] > 0) go = mbar_wait_warp(&pv_done[s], (tiles[s] - 1) & 1, abort_flag);
                }
                if (go && (s == 1 || !first_turn)) go = mbar_wait_warp(&turn[s], s == 0 ? it ^ 1 : it, abort_flag);
                if (go && owed == 1) go = mbar_wait_warp(&p_full[s], (tiles[s] - 1) & 1, abort_flag, wlim);
                if (!go) return false;
                tc_fence_after();
                if (owed == 1)
                    pv(s, rv, owed_keys, owed_first);
                else if (owed == 2 && lane == 0)
                    mbar_arrive(&slot_empty[rv.slot]);
                owed = 0;
                if (own) {
                    qk(s, rk, keys, last);
                    ++tiles[s];
                    owed = 1;
                    owed_keys = keys;
                    owed_first = first;
                } else if (visit) {
                    if (lane == 0) mbar_arrive(&slot_empty[rk.slot]);
                    owed = 2;
                }
                if (lane == 0) mbar_arrive(&turn[s ^ 1]);
                it ^= 1;
                first_turn = false;
                return true;
            };
            for (int k = 0; FEW && ok; ++k) {
                ok = next_unit(k, &u);
                if (!ok) break;
                if (owed && (ends_list(u) || few_of(u))) ok = turn_few(false, false, false, false, 0);
                if (!ok || ends_list(u)) break;
                const int end = last_key(p, u, few_of(u) ? 0 : s);
                if (few_of(u)) {
                    const int n = u.n[0];
                    if (s == 0) ok = mbar_wait_warp(&q_full[0], units_q++ & 1, abort_flag);
                    for (int j = 0; j < n && ok; ++j) {
                        // (what is waited for first has every fill of the slot before its
                        // present one behind it: its parity means this one)
                        const int buf = j & 1, keys = min(kRows, end - j * kRows);
                        const bool before = tiles[buf] > 0;
                        const uint32_t par = tiles[buf] & 1;
                        if (s == 1) rc.next();
                        const auto r = rc;
                        if (s == 0 && before) ok = mbar_wait_warp(&pv_done[buf], par ^ 1, abort_flag);
                        if (s == 1) ok = mbar_wait_warp(&p_full[buf], par, abort_flag, wlim);
                        ok = ok && mbar_wait_warp(&slot_full[r.slot], r.parity, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        if (s == 0)
                            qk(buf, r, keys, j == n - 1);
                        else
                            pv(buf, r, keys, j < 2, buf);
                        if (elect_one()) umma_commit(&slot_empty[r.slot]);  // (the other warp's)
                        __syncwarp();
                        rc.next();
                        if (s == 0) rc.next();
                        ++tiles[buf];
                    }
                    after_few = true;
                } else {
                    const int n = s == 0 ? u.n[0] : u.n[1], nmax = max(u.n[0], u.n[1]), j0 = first_tile(p, u, s);
                    for (int j = 0; j < nmax && ok; ++j)
                        ok = turn_few(true, j0 <= j && j < n, j == j0, j == n - 1, min(kRows, end - j * kRows));
                    const int other = s == 0 ? u.n[1] : u.n[0];
                    if (other > 0) tiles[s ^ 1] += other - first_tile(p, u, s ^ 1);
                }
            }
            for (int k = 0; !FEW && ok; ++k) {
                ok = next_unit(k, &u);
                if (!ok) break;
                if (ends_list(u)) {
                    if (owed) ok = turn_of(0, 0, 0, 0, 0);
                    break;
                }
                const int nmax = max(u.n[0], u.n[1]), j0 = first_tile(p, u, s);
                int n;
                if constexpr (PG)
                    n = s == 0 ? u.n[0] : u.n[1];
                else
                    n = u.n[s];
                const int end = last_key(p, u, s);
                for (int j = 0; j < nmax && ok; ++j) ok = turn_of(j0, n, nmax, j, end);
            }
        } else {
            // One warp issues Q K^T, the other P V, so that each one's waits pass
            // under the other's MMAs.  Q K^T of key tile g goes into the S buffer
            // that P V of g - 2 reads its P from: it is issued behind that (a
            // fence on both sides of the barrier keeps the MMAs' order).
            Walk w;
            auto tile = [&](auto &rc) {
                ok = step(w);
                while (ok && !w.done) {
                    const int buf = w.g & 1;
                    const uint32_t parity = (w.g >> 1) & 1;
                    const auto r = rc;
                    if (warp == 1 && w.j == 0) ok = mbar_wait_warp(&q_full[0], units_q++ & 1, abort_flag);
#pragma unroll
                    for (int c = 0; c < CPT; ++c, rc.next())
                        ok = ok && mbar_wait_warp(&slot_full[rc.slot], rc.parity, abort_flag);
                    if (ok && warp == 1 && w.g >= 2) ok = mbar_wait_warp(&turn[buf], parity ^ 1, abort_flag);
                    if (ok && warp == 2) ok = mbar_wait_warp(&p_full[buf], parity, abort_flag, wlim);
                    if (!ok) break;
                    tc_fence_after();
                    const int keys = min(kRows, last_key(p, w.u, 0) - w.j * kRows);
                    if constexpr (std::is_same_v<std::remove_const_t<decltype(r)>, typename C::KRing>) {
                        qk(buf, r, keys, w.j == w.u.n[0] - 1);
                    } else {
                        pv(buf, r, keys, w.j == 0);
                        if (elect_one()) {  // (the lane that issued)
                            tc_fence_before();
                            mbar_arrive(&turn[buf]);
                        }
                        __syncwarp();
                    }
                    ok = step(w);
                }
            };
            if constexpr (NQ == 1) {
                if (warp == 1) {
                    typename C::KRing rc;
                    tile(rc);
                } else {
                    typename C::VRing rc;
                    tile(rc);
                }
            }
        }
        if (!ok) {
            pf_error(p.err, DEV_ERR_TIMEOUT);
            *abort_flag = 1;
        }
        // every MMA issued so far has finished before tensor memory is freed
        if (elect_one()) umma_commit(drain);
        __syncwarp();
        volatile int never = 0;
        mbar_wait_warp(drain, 0, &never);
        __syncwarp();
        named_bar_sync(kBarEndPf, C::THREADS);
        if (warp == 1) {
            tc_fence_after();
            tmem_dealloc(tmem, 512);
        }
        return;
    }

    }

    // ============================================================== softmax
    if constexpr (NQ == 2) regs_inc<C::REGS_SOFT>();
    const int s = (warp - C::SOFT0) >> 2;          // query tile
    const int q4 = warp & 3;                       // TMEM lane quarter this warp may access
    const int row = q4 * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(q4 * 32) << 16);
    const uint32_t o_t = lanes + C::O0 + s * D;
    int r_tok, r_head;
    constexpr int kNobody = 1 << 20;
    [[maybe_unused]] int few_tok_of = 0;  // (paged) the token of the lane's row in a copy of few rows
    if constexpr (PG) {  // (any number of heads; rows past the tile's are nobody's)
        zero_rows(p, D, tid - 32 * C::SOFT0, 128 * NQ);
        r_tok = row < p.rows ? row / p.hpg : kNobody;
        r_head = row % p.hpg;
        if (FEW) few_tok_of = lane < p.few_tok * p.hpg ? lane / p.hpg : kNobody;
    } else {
        r_tok = row >> p.hpg_lg;
        r_head = row & (p.hpg - 1);
    }
    long long g = 0;      // key tiles so far
    long long base = 0;   // ring slots of the units before this one
    bool ok = true;
    [[maybe_unused]] uint32_t joins = 0;  // (few rows) steps of joins so far

    Unit u;
    for (int k = 0;; ++k) {
        ok = next_unit(k, &u);
        if (!ok || (PG ? u.n[0] < 0 : u.n[0] == 0)) break;  // (ends_list, which takes u's address, spills here)
        const int nmax = max(u.n[0], u.n[1]);
        int n;
        if constexpr (PG)
            n = NQ == 2 && s == 1 ? u.n[1] : u.n[0];  // (an index known when it is compiled keeps u in registers)
        else
            n = u.n[s];
        int first_tok = u.t0 + s * p.tpt;
        if constexpr (FEW)
            if (u.few) first_tok = u.t0;  // (both tiles)
        const int end_tok = min(first_tok + p.tpt, u.len);
        int tok = first_tok + r_tok;
        if constexpr (PG)
            if (FEW && u.few) tok = first_tok + few_tok_of;
        const int tq = min(tok, u.len - 1);
        float m = -INFINITY, l = 0.f;
        bool alive = true;  // (paged) some row of the warp is a token's
        [[maybe_unused]] int e_row, e_first, e_last;  // (paged) where the row's keys end, the tile's first and last
        if constexpr (PG) {
            alive = (FEW && u.few) || q4 * 32 < (end_tok - first_tok) * p.hpg;
            e_row = key_end(p, u.shift, tq);
            e_first = key_end(p, u.shift, first_tok);
            e_last = key_end(p, u.shift, end_tok - 1);
        }

        const int j0 = first_tile(p, u, s);
        // the running maximum follows mn where it is far behind; O and l with it
        auto move_max = [&](float mn, bool more, int buf) -> bool {
            const bool grow = (mn - m) * p.sl > kTauPf;  // (both -inf: no)
            if (__any_sync(0xffffffffu, grow)) {
                const float alpha = (grow && m != -INFINITY) ? fast_exp2((m - mn) * p.sl) : 1.f;
                if (grow) m = mn;
                l *= alpha;
                if (more && __any_sync(0xffffffffu, alpha != 1.f)) {
                    // O holds the tiles up to j - 1
                    const int pb = NQ == 2 ? s : buf ^ 1;
                    const uint32_t pp = (uint32_t)((NQ == 2 ? g - 1 : (g - 1) >> 1) & 1);
                    ok = mbar_wait_warp(&pv_done[pb], pp, abort_flag, wlim);
                    if (!ok) return false;
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        float o[16];
                        tmem_ld16(o_t + c * 16, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= alpha;
                        tmem_st16(o_t + c * 16, o);
                    }
                }
            }
            return true;
        };
        // (few rows) the weights of 32 scores to column `to` of P, and into l
        [[maybe_unused]] auto weigh = [&](const float (&x)[32], uint32_t to) {
            const float neg_m = m == -INFINITY ? 0.f : -m * p.sl;
            const float2 sl2 = make_float2(p.sl, p.sl), nm2 = make_float2(neg_m, neg_m);
            float2 ls[2] = {make_float2(l, 0.f), make_float2(0.f, 0.f)};
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float2 y = fma2(make_float2(x[2 * i], x[2 * i + 1]), sl2, nm2);
                const float2 e = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                ls[i & 1] = add2(ls[i & 1], e);
                pk[i] = bf16x2_of(e.x, e.y);
            }
            tmem_st16u(to, pk);
            ls[0] = add2(ls[0], ls[1]);
            l = ls[0].x + ls[0].y;
        };
        auto hide_rows = [&](int j, int buf, int kb, int keys) -> bool {
            // rows past the sequence's end that the last 16 keys of P V would
            // read belong to another sequence (or to none) and may hold
            // anything, which a weight of zero does not hide: they are zeroed
            const int stop = (keys + 15) / 16 * 16, past = seq_keys(p, u) - kb;
            // (paged: so are those before the first that a token of the unit attends)
            int before = 0;
            if constexpr (PG) before = first_key(p, u) - kb;
            if (past < stop || (PG && before > 0)) {
                const long long iv = NQ == 2 ? base + 2 * j + 1 : g * CPT;  // (of the ring that V is in)
                // (one query tile: the scores may be two tiles ahead of P V, and
                // the slot's parity says something once the V tile before is done with)
                if (NQ == 1 && g > 0) ok = mbar_wait_warp(&pv_done[buf ^ 1], (uint32_t)(((g - 1) >> 1) & 1), abort_flag);
                for (int c = 0; c < CPT && ok; ++c) {
                    const int slot = (NQ == 2 ? 0 : C::KN) + (int)((iv + c) % C::VN);
                    ok = mbar_wait_warp(&slot_full[slot], (uint32_t)(((iv + c) / C::VN) & 1), abort_flag);
                    if constexpr (PG) {
                        if (ok)
                            for (int i = row; i < before * (C::KC / 64) * 8; i += 128) {
                                const int r = (i >> 3) / (C::KC / 64), sl = (i >> 3) % (C::KC / 64);
                                *reinterpret_cast<uint4 *>(ring + slot * C::SLOT + sl * kSlab + r * 128 +
                                                           (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                            }
                    }
                    if (ok)
                        for (int i = row; i < (stop - past) * (C::KC / 64) * 8; i += 128) {
                            const int r = past + (i >> 3) / (C::KC / 64), sl = (i >> 3) % (C::KC / 64);
                            *reinterpret_cast<uint4 *>(ring + slot * C::SLOT + sl * kSlab + r * 128 +
                                                       (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                }
                if (!ok) return false;
                fence_proxy_async_smem();
            }
            return true;
        };
        if constexpr (FEW) {
            for (int j = s; u.few && j < n; j += 2, ++g) {
            const int buf = s;
            const uint32_t par = (uint32_t)(g & 1);
            ok = mbar_wait_warp(&s_full[buf], par, abort_flag, wlim);
            if (!ok) break;
            tc_fence_after();
            const uint32_t s_t = lanes + buf * 128;
            const int kb = u.kbeg + j * kRows, keys = min(kRows, min(u.kend, e_last) - kb);
            const int hi = e_row - kb, lo = hi - p.window, sure_hi = e_first - kb, sure_lo = e_last - p.window - kb;
            // this warp's quarter of the columns, for its copy of the rows; the
            // other columns of P are zero
            float x[32];
            const int c0 = q4 * 32;
            float mn = m;
            if (c0 < keys) {
                tmem_ld32(s_t + c0, x);
                tmem_ld_wait();
                if (c0 + 32 > sure_hi || c0 < sure_lo) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = (c0 + i < hi && c0 + i >= lo) ? x[i] : -INFINITY;
                }
                mn = fmaxf(mn, max_of(x));
            }
            if (!move_max(mn, j > s, buf)) break;
            {
                uint32_t none[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) none[i] = 0u;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c != q4 && c * 32 < keys) tmem_st16u(s_t + c * 16, none);
            }
            if (c0 < keys) weigh(x, s_t + c0 / 2);
            if (!hide_rows(j, buf, kb, keys)) break;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[buf]);
            }
            if (!ok) break;
        }
        for (int j = j0; j < n && !(FEW && few_of(u)); ++j, ++g) {
            const int buf = NQ == 2 ? s : (int)(g & 1);
            const uint32_t par = (uint32_t)((NQ == 2 ? g : g >> 1) & 1);
            ok = mbar_wait_warp(&s_full[buf], par, abort_flag, wlim);
            if (!ok) break;
            tc_fence_after();
            const uint32_t s_t = lanes + buf * 128;
            // The tile's keys in four parts of 32: parts past the last key that
            // any row attends are left out (the MMAs stop there too), and only
            // parts at the diagonal or the window's edge hide some keys from
            // some rows: a row's are [lo, hi).
            [[maybe_unused]] float v[FEW ? 1 : 128];
            const int kb = u.kbeg + j * kRows;
            int keys, hi, lo, sure_hi, sure_lo;
            if constexpr (PG) {
                keys = min(kRows, min(u.kend, e_last) - kb);
                hi = e_row - kb;
                lo = hi - p.window;
                sure_hi = e_first - kb;
                sure_lo = e_last - p.window - kb;
            } else {
                keys = min(kRows, end_tok - kb);
                hi = tq + 1 - kb, lo = tq + 1 - p.window - kb;
                sure_hi = first_tok + 1 - kb, sure_lo = end_tok - p.window - kb;
            }
            // (a whole tile that hides nothing takes the straight path)
            const bool whole = !FEW && keys == kRows && kRows <= sure_hi && sure_lo <= 0;
            if (PG && !whole) {
                // 32 columns at a time, twice: code of a few hundred instructions (unrolled
                // over the tile its first turn, and each after the straight path's, waits for
                // instructions)
                if (alive) {
                    auto scores = [&](int c, float (&x)[32]) {
                        tmem_ld32(s_t + c * 32, x);
                        tmem_ld_wait();
                        if (c * 32 + 32 > sure_hi || c * 32 < sure_lo) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                x[i] = (c * 32 + i < hi && c * 32 + i >= lo) ? x[i] : -INFINITY;
                        }
                    };
                    float mn = m;
#pragma unroll 1
                    for (int c = 0; c * 32 < keys; ++c) {
                        float x[32];
                        scores(c, x);
                        mn = fmaxf(mn, max_of(x));
                    }
                    if (!move_max(mn, j > j0, buf)) break;
#pragma unroll 1
                    for (int c = 0; c * 32 < keys; ++c) {  // (P of a part lies over scores of the parts before)
                        float x[32];
                        scores(c, x);
                        weigh(x, s_t + c * 16);
                    }
                }
            } else if constexpr (!FEW) {
            if (!PG || alive) {
            float mn;
            if (PG || whole) {
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(s_t + c * 32, v + c * 32);
                tmem_ld_wait();
                float mx[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mx[i] = max3(v[i], v[8 + i], v[16 + i]);
#pragma unroll
                for (int c = 24; c < 120; c += 16) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) mx[i] = max3(mx[i], v[c + i], v[c + 8 + i]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) mx[i] = fmaxf(mx[i], v[120 + i]);
                mn = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), max3(mx[6], mx[7], m));
            } else {
                mn = m;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float *x = v + c * 32;
                    if (c * 32 < keys) {
                        tmem_ld32(s_t + c * 32, x);
                        tmem_ld_wait();
                        if (c * 32 + 32 > sure_hi || c * 32 < sure_lo) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                x[i] = (c * 32 + i < hi && c * 32 + i >= lo) ? x[i] : -INFINITY;
                        }
                        float mx[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) mx[i] = max3(x[i], x[4 + i], x[8 + i]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], x[12 + i], x[16 + i]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) mx[i] = max3(mx[i], x[20 + i], x[24 + i]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], x[28 + i]);
                        mn = max3(mn, max3(mx[0], mx[1], mx[2]), mx[3]);
                    }
                }
            }
            if (!move_max(mn, j > j0, buf)) break;
            const float neg_m = m == -INFINITY ? 0.f : -m * p.sl;
            const float2 sl2 = make_float2(p.sl, p.sl), nm2 = make_float2(neg_m, neg_m);
            float2 ls[2] = {make_float2(l, 0.f), make_float2(0.f, 0.f)};
            auto weights = [&](int c) {  // of the part's 32 keys
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 x = fma2(make_float2(v[c * 32 + 2 * i], v[c * 32 + 2 * i + 1]), sl2, nm2);
                    const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                    ls[i & 1] = add2(ls[i & 1], e);
                    pk[i] = bf16x2_of(e.x, e.y);
                }
                tmem_st16u(s_t + c * 16, pk);
            };
            if (PG || whole) {
#pragma unroll
                for (int c = 0; c < 4; ++c) weights(c);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c * 32 < keys) weights(c);
            }
            ls[0] = add2(ls[0], ls[1]);
            l = ls[0].x + ls[0].y;
            }
            }
            if (!hide_rows(j, buf, kb, keys)) break;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[buf]);
        }
        if (!ok) break;
        // (paged) the rows as they are, and what they stand for
        [[maybe_unused]] auto store_partial = [&](int slot) {
            if constexpr (PG) {
                const size_t at = (size_t)slot * (NQ * kRows) + s * kRows + row;
                float *dst = p.ws_o + at * D;
                if constexpr (!Partial<D, FEW>::WHOLE) dst = p.ws_o + Partial<D, FEW>::row(slot, s * kRows + row);
                if (tok < end_tok)
                    *reinterpret_cast<float2 *>(p.ws_ml + at * 2) =
                        make_float2(m == -INFINITY ? -INFINITY : m * p.sl, l);
                [[maybe_unused]] long long off[4];
                if constexpr (D == 256) {
                    const long long mine = tok < end_tok ? (long long)at * (D * 4) : -1;
#pragma unroll
                    for (int r = 0; r < 4; ++r) off[r] = __shfl_sync(0xffffffffu, mine, (lane & ~3) + r);
                }
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {  // (unrolled, it spills at D = 256)
                    float o[32];
                    tmem_ld32(o_t + c * 32, o);
                    tmem_ld_wait();
                    if constexpr (D == 256) {
                        uint32_t w[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i]);
                        store_lines(p.ws_o + c * 32, off, w);
                    } else if (tok < end_tok) {
                        uint32_t w[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i]);
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
                            st_global_32b(dst + (c * 32 + i) / 8 * Partial<D, FEW>::STEP, w + i);
                    }
                }
                tc_fence_before();
                __syncwarp();
            }
        };
        [[maybe_unused]] auto store_nothing = [&](int slot) {
            if constexpr (PG)
                if (tok < end_tok)
                    *reinterpret_cast<float2 *>(p.ws_ml + ((size_t)slot * (NQ * kRows) + s * kRows + row) * 2) =
                        make_float2(-INFINITY, 0.f);
        };
        if constexpr (FEW) {
            if (u.few) {
                // The copies of a row, each with the keys of its columns, are joined in
                // shared memory (through the workspace it took some 6 us a unit under
                // load): maxima, then sums and the rows scaled to the joint maximum, a
                // group of rows at a time, which all warps add up, one row each.
                constexpr int COPIES = 4 * NQ, GROUP = C::QT / (COPIES * D * 4), V = D / 32;
                const int copy = s * 4 + q4, rows = (end_tok - first_tok) * p.hpg;
                float *exch = reinterpret_cast<float *>(cnt);                     // [COPIES][32]
                float *part = reinterpret_cast<float *>(qbuf + C::QT);  // [COPIES][GROUP][D]: query tile 1's place
                auto all_here = [&]() -> bool {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(join);
                    return mbar_wait_warp(join, joins++ & 1, abort_flag);
                };
                const bool own = n > s;
                if (own) {
                    ok = mbar_wait_warp(&pv_done[s], (uint32_t)((g - 1) & 1), abort_flag, wlim);
                    if (!ok) break;
                    tc_fence_after();
                }
                exch[copy * 32 + lane] = m;
                if (!(ok = all_here())) break;
                float top = -INFINITY;
#pragma unroll
                for (int c = 0; c < COPIES; ++c) top = fmaxf(top, exch[c * 32 + lane]);
                const float w = m == -INFINITY ? 0.f : fast_exp2((m - top) * p.sl);
                if (!(ok = all_here())) break;
                exch[copy * 32 + lane] = l * w;
                for (int r0 = 0; r0 < rows; r0 += GROUP) {
                    // (16-byte pieces of a row change places by its number: the lanes'
                    // stores, a row apart, meet different banks)
                    float *mine = part + (copy * GROUP + lane - r0) * D;
                    const bool here = lane >= r0 && lane < min(rows, r0 + GROUP);
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        float o[16];
                        if (own) {
                            tmem_ld16(o_t + c * 16, o);
                            tmem_ld_wait();
                        }
                        if (here) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int at = ((c * 4 + i) ^ (lane & 7)) * 4;
                                *reinterpret_cast<float4 *>(mine + at) =
                                    own ? make_float4(o[4 * i] * w, o[4 * i + 1] * w, o[4 * i + 2] * w, o[4 * i + 3] * w)
                                        : make_float4(0.f, 0.f, 0.f, 0.f);
                            }
                        }
                    }
                    if (!(ok = all_here())) break;
                    for (int r = r0 + copy; r < min(rows, r0 + GROUP); r += COPIES) {
                        float o[V], sum = 0.f;
#pragma unroll
                        for (int i = 0; i < V; ++i) o[i] = 0.f;
#pragma unroll
                        for (int c = 0; c < COPIES; ++c) {
                            const float *from = part + (c * GROUP + r - r0) * D;
                            sum += exch[c * 32 + r];
                            if constexpr (V == 2) {
                                const float2 x = *reinterpret_cast<const float2 *>(from + ((lane >> 1) ^ (r & 7)) * 4 + (lane & 1) * 2);
                                o[0] += x.x;
                                o[1] += x.y;
                            } else {
#pragma unroll
                                for (int i = 0; i < V; i += 4) {
                                    const float4 x = *reinterpret_cast<const float4 *>(from + ((lane * (V / 4) + i / 4) ^ (r & 7)) * 4);
                                    o[i] += x.x;
                                    o[i + 1] += x.y;
                                    o[i + 2] += x.z;
                                    o[i + 3] += x.w;
                                }
                            }
                        }
                        const float of_row = __shfl_sync(0xffffffffu, top, r);
                        if (u.slot >= 0) {
                            const size_t at = (size_t)u.slot * (NQ * kRows) + r;
                            float *dst = p.ws_o + at * D + lane * V;
                            if constexpr (V == 2)
                                *reinterpret_cast<float2 *>(dst) = make_float2(o[0], o[1]);
                            else
#pragma unroll
                                for (int i = 0; i < V; i += 4)
                                    *reinterpret_cast<float4 *>(dst + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                            if (lane == 0)
                                *reinterpret_cast<float2 *>(p.ws_ml + at * 2) =
                                    make_float2(of_row == -INFINITY ? -INFINITY : of_row * p.sl, sum);
                        } else {
                            const int t = r / p.hpg;
                            store_row<V>(p.out + ((size_t)(u.row0 + u.t0 + t) * p.Hq + u.h0 + r - t * p.hpg) * D + lane * V,
                                         o, 1.f / sum);
                        }
                    }
                    // (the next to write here is a copy of query rows)
                    fence_proxy_async_smem();
                    if (!(ok = all_here())) break;
                }
                if (!ok) break;
                if (copy == 0 && lane == 0) {
                    __threadfence_block();
                    *joined = *joined + 1;
                }
                base += 2 * nmax;
                continue;
            }
        }
        if (n > 0) {
            const int buf = NQ == 2 ? s : (int)((g - 1) & 1);
            const uint32_t par = (uint32_t)((NQ == 2 ? g - 1 : (g - 1) >> 1) & 1);
            ok = mbar_wait_warp(&pv_done[buf], par, abort_flag, wlim);
            if (!ok) break;
            tc_fence_after();
            if constexpr (PG) {
                if (u.slot >= 0) {  // a piece
                    store_partial(u.slot);
                    base += 2 * nmax;
                    continue;
                }
            }
            const float inv = 1.f / l;  // (every row attends itself)
            // (whole lines: 16 heads over 1 of 256 in a window of 1024 68.0 -> 65.6 us with
            // the partial rows' below, 32 single tokens of 64 over 8 of 128 96.7 -> 95.8; at
            // D = 64, a line a row, prompts over states lose 33.1 -> 34.0)
            if constexpr (PG && D > 64) {
                const long long at = tok < end_tok ? (((long long)(u.row0 + tok) * p.Hq + u.h0 + r_head) * D) * 2 : -1;
                long long off[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) off[r] = __shfl_sync(0xffffffffu, at, (lane & ~3) + r);
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c) {
                    uint32_t w[32];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float o[32];
                        tmem_ld32(o_t + c * 64 + h * 32, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[h * 16 + i] = bf16x2_of(o[2 * i] * inv, o[2 * i + 1] * inv);
                    }
                    store_lines(p.out + c * 64, off, w);
                }
            } else {
            uint16_t *dst = p.out + ((size_t)(u.row0 + tok) * p.Hq + u.h0 + r_head) * D;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
                tmem_ld32(o_t + c * 32, o);
                tmem_ld_wait();
                if (tok < end_tok) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) w[i] = bf16x2_of(o[2 * i] * inv, o[2 * i + 1] * inv);
                    st_global_32b(dst + c * 32, w);
                    st_global_32b(dst + c * 32 + 16, w + 8);
                }
            }
            }
            tc_fence_before();
            __syncwarp();
        } else if constexpr (PG) {
            // (a piece behind this query tile's last key)
            store_nothing(u.slot);
        }
        base += 2 * nmax;
    }
    if (!ok) {
        pf_error(p.err, DEV_ERR_TIMEOUT);
        *abort_flag = 1;
    }
    tc_fence_before();
    named_bar_sync(kBarEndPf, C::THREADS);
}

template <int D, bool PG, bool FEW>
cudaError_t launch_pf(const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv,
                      const ParamsOf<PG> &p, int num_ctas, cudaStream_t stream, const QuarterMap<PG> &tmq4 = {}) {
    static int done_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!(dev >= 0 && dev < 64 && done_for_device[dev])) {
        e = cudaFuncSetAttribute(prefill_kernel<D, PG, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PfCfg<D, PG>::alloc);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) done_for_device[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_ctas);
    cfg.blockDim = dim3(PfCfg<D, PG>::THREADS);
    cfg.dynamicSmemBytes = PfCfg<D, PG>::alloc;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefill_kernel<D, PG, FEW>, tmq, tmk, tmv, p, tmq4);
}

// 3-D map over packed rows [N, H, D] with `stride` elements from token to
// token: dims (D, H, N), box (64, heads, tokens), 128-byte swizzle; tokens
// past N read as zeros.
int encode_rows_map(CUtensorMap *m, const void *base, int D, int H, int N, long long stride, int heads,
                    int tokens) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)N};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)tokens};
    return api_encode_bf16_3d(m, base, dims, strides, box);
}

}  // namespace

}  // namespace kvattn
