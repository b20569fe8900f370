// prefill.cu -- causal grouped-query attention over whole prompts, packed one
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
// output is bf16: the weights' rounding, at most 2^-9 each, averages out below
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
#include <cfloat>
#include <climits>
#include <cmath>
#include <cuda_bf16.h>
#include <type_traits>

#include "../../include/kvattn.h"
#include "internal.h"
#include "ptx.cuh"

namespace kvattn {

namespace {

constexpr int kRows = 128;      // query rows of a tile = keys of a tile
constexpr int kSlab = 16384;    // 128 rows x 64 columns of bf16
constexpr int kSmemMax = 232448;
constexpr float kTauPf = 8.f;   // log2 headroom before the running max must move
constexpr int kBuckets = 128;
constexpr int kDesc = 4;        // units in flight between the work list and its readers
constexpr int kBarEndPf = 1;

struct PrefillParams {
    const int32_t *cu;  // [B + 1] first rows of the sequences
    uint16_t *out;      // bf16 [N, Hq, D]
    unsigned int *err;
    int B, N, Hq, Hkv, G;
    int hpg, hpg_lg;    // query heads of a tile, a power of two
    int tpt;            // tokens of a tile, 128 / hpg
    int passes;         // G / hpg
    int window;         // keys one query attends at most (N: all)
    float sl;           // |scale| log2(e), at least the smallest normal number
    int neg;            // scale < 0: the MMA negates q
    unsigned int wait_limit;
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

template <int D>
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
    static constexpr int nbar = 2 * NS + 2 * 2 + 3 * 2 + 2 * kDesc + 1 + 2;
    static constexpr int off_misc = off_bar + nbar * 8;          // tmem base, abort flag
    static constexpr int off_unit = (off_misc + 32 + 15) / 16 * 16;
    static constexpr int off_cnt = off_unit + kDesc * (int)sizeof(Unit);
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

// Pairs of binary32 values in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rc, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\tmov.b64 rc, {%6, %7};\n\t"
        "fma.rn.f32x2 rd, ra, rb, rc;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
        "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 32 bytes, a whole sector, from one thread (dst 32-byte aligned).
__device__ __forceinline__ void st_global_32b(uint16_t *dst, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
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

// A published unit, the same in every lane.
__device__ __forceinline__ Unit read_unit(const Unit &from) {
    Unit u;
    const int *src = reinterpret_cast<const int *>(&from);
    int *dst = reinterpret_cast<int *>(&u);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(Unit) / 4); ++i) dst[i] = __shfl_sync(0xffffffffu, src[i], 0);
    return u;
}

// First of the unit's key tiles that query tile s attends: its window may start
// behind whole tiles that the first query tile needs (one of ten in a window of
// 1024 with 128 tokens a tile: three prompts of 16 heads of 64, 78.3 us with them
// computed, 74.1 without; full prompts lose 0.4 % to the test).
__device__ __forceinline__ int first_tile(const PrefillParams &p, const Unit &u, int s) {
    return max(0, u.t0 + s * p.tpt + 1 - p.window - u.kbeg) / kRows;
}

// Length of sequence b (0 where its bounds are not 0 <= cu[b] <= cu[b+1] <= N).
__device__ __forceinline__ int pf_len(const PrefillParams &p, int b, int *row0) {
    const int a = p.cu[b], e = p.cu[b + 1];
    *row0 = a;
    return (a < 0 || e < a || e > p.N) ? -1 : e - a;
}

template <int D>
__global__ void __launch_bounds__(PfCfg<D>::THREADS, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                   const __grid_constant__ CUtensorMap tmv, const PrefillParams p) {
    using C = PfCfg<D>;
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
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::off_misc);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::off_misc + 16);
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
    const long long total = (long long)*sum_pairs * heads;
    const int mnb = *max_nb;
    // one wave of units: any order does
    const int width = total <= gridDim.x ? max(mnb, 1) : (mnb + kBuckets - 1) / kBuckets;
    const int nbk = width > 0 ? (mnb + width - 1) / width : 0;
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
    int fills = 0;  // slots filled by this warp
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
    // (by one lane) the last fills of a ring of n slots from slot `off` have landed
    auto landed = [&](int n, int off) {
        volatile int never = 0;
        for (int i = fills > n ? fills - n : 0; i < fills; ++i)
            pf_wait(&slot_full[off + i % n], (uint32_t)((i / n) & 1), &never);
    };
    // A walk over the key tiles of all units (one query tile).
    struct Walk {
        Unit u;
        int k = -1, g = -1;  // unit, key tile of the CTA
        int j = 0;           // key tile of the unit
        bool done = false;
    };
    auto step = [&](Walk &w) -> bool {
        ++w.g;
        if (w.k >= 0 && ++w.j < w.u.n[0]) return true;
        w.j = 0;
        if (!next_unit(++w.k, &w.u)) return false;
        w.done = w.u.n[0] == 0;
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
        Unit u = {};
        int k = 0;
        bool more = true, done;  // the last unit published does not end the list
        find(0, &u);
        auto pump = [&](bool must) {  // publishes the next unit and finds the one after
            if (!more) return true;
            if (!publish(k, u, must, &done)) return false;
            if (done) {
                more = u.n[0] != 0;
                ++k;
                if (more) find(k, &u);
            }
            return true;
        };
        if (NQ == 2) {
            while (ok && more) ok = pump(true);
        } else {
            // this warp copies V, too, and publishes units as their places come free
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
        if (!ok && lane == 0) {
            pf_error(p.err, DEV_ERR_TIMEOUT);
            *abort_flag = 1;
        }
        __syncwarp();
        named_bar_sync(kBarEndPf, C::THREADS);
        if (NQ == 1 && *abort_flag && lane == 0) landed(C::VN, C::KN);
        return;
    }

    // ================================================================== TMA
    if (warp == 0) {
        bool ok = true;
        uint32_t qn[2] = {0, 0};     // query tiles issued
        typename C::KRing rc;
        auto load_q = [&](const Unit &u) -> bool {
            for (int s = 0; s < NQ; ++s) {
                if (u.n[s] == 0) continue;
                if (qn[s] && !mbar_wait_warp(&q_empty[s], (qn[s] - 1) & 1, abort_flag)) return false;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&q_full[s], C::QT);
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
        if (NQ == 2) {
            Unit u;
            for (int k = 0; ok; ++k) {
                ok = next_unit(k, &u);
                if (!ok || u.n[0] == 0) break;
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
        auto pv = [&](int buf, typename C::VRing r, int keys, bool first) {
            const uint32_t a = tmem + buf * 128, d = tmem + C::O0 + s * D;
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
            for (int k = 0; ok; ++k) {
                ok = next_unit(k, &u);
                if (!ok) break;
                if (u.n[0] == 0) {
                    if (owed) ok = turn_of(0, 0, 0, 0, 0);
                    break;
                }
                const int n = u.n[s], nmax = max(u.n[0], u.n[1]), j0 = first_tile(p, u, s);
                // keys of the unit's key tiles that the query tile attends at most
                const int end = min(u.t0 + (s + 1) * p.tpt, u.len) - u.kbeg;
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
                    const int keys = min(kRows, min(w.u.t0 + p.tpt, w.u.len) - w.u.kbeg - w.j * kRows);
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
    const int r_tok = row >> p.hpg_lg, r_head = row & (p.hpg - 1);
    long long g = 0;      // key tiles so far
    long long base = 0;   // ring slots of the units before this one
    bool ok = true;

    Unit u;
    for (int k = 0;; ++k) {
        ok = next_unit(k, &u);
        if (!ok || u.n[0] == 0) break;
        const int n = u.n[s], nmax = max(u.n[0], u.n[1]);
        const int first_tok = u.t0 + s * p.tpt;
        const int end_tok = min(first_tok + p.tpt, u.len);
        const int tok = first_tok + r_tok;
        const int tq = min(tok, u.len - 1);
        float m = -INFINITY, l = 0.f;

        const int j0 = first_tile(p, u, s);
        for (int j = j0; j < n; ++j, ++g) {
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
            float v[128];
            const int kb = u.kbeg + j * kRows;
            const int keys = min(kRows, end_tok - kb);
            const int hi = tq + 1 - kb, lo = tq + 1 - p.window - kb;
            const int sure_hi = first_tok + 1 - kb, sure_lo = end_tok - p.window - kb;
            // (a whole tile that hides nothing takes the straight path)
            const bool whole = keys == kRows && kRows <= sure_hi && sure_lo <= 0;
            float mn;
            if (whole) {
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
            const bool grow = (mn - m) * p.sl > kTauPf;  // (both -inf: no)
            if (__any_sync(0xffffffffu, grow)) {
                const float alpha = (grow && m != -INFINITY) ? fast_exp2((m - mn) * p.sl) : 1.f;
                if (grow) m = mn;
                l *= alpha;
                if (j > j0 && __any_sync(0xffffffffu, alpha != 1.f)) {
                    // O holds the tiles up to j - 1
                    const int pb = NQ == 2 ? s : buf ^ 1;
                    const uint32_t pp = (uint32_t)((NQ == 2 ? g - 1 : (g - 1) >> 1) & 1);
                    ok = mbar_wait_warp(&pv_done[pb], pp, abort_flag, wlim);
                    if (!ok) break;
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
            if (whole) {
#pragma unroll
                for (int c = 0; c < 4; ++c) weights(c);
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c * 32 < keys) weights(c);
            }
            ls[0] = add2(ls[0], ls[1]);
            l = ls[0].x + ls[0].y;
            // rows past the sequence's end that the last 16 keys of P V would
            // read belong to another sequence (or to none) and may hold
            // anything, which a weight of zero does not hide: they are zeroed
            const int stop = (keys + 15) / 16 * 16, past = u.len - kb;
            if (past < stop) {
                const long long iv = NQ == 2 ? base + 2 * j + 1 : g * CPT;  // (of the ring that V is in)
                // (one query tile: the scores may be two tiles ahead of P V, and
                // the slot's parity says something once the V tile before is done with)
                if (NQ == 1 && g > 0) ok = mbar_wait_warp(&pv_done[buf ^ 1], (uint32_t)(((g - 1) >> 1) & 1), abort_flag);
                for (int c = 0; c < CPT && ok; ++c) {
                    const int slot = (NQ == 2 ? 0 : C::KN) + (int)((iv + c) % C::VN);
                    ok = mbar_wait_warp(&slot_full[slot], (uint32_t)(((iv + c) / C::VN) & 1), abort_flag);
                    if (ok)
                        for (int i = row; i < (stop - past) * (C::KC / 64) * 8; i += 128) {
                            const int r = past + (i >> 3) / (C::KC / 64), sl = (i >> 3) % (C::KC / 64);
                            *reinterpret_cast<uint4 *>(ring + slot * C::SLOT + sl * kSlab + r * 128 +
                                                       (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                }
                if (!ok) break;
                fence_proxy_async_smem();
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[buf]);
        }
        if (!ok) break;
        if (n > 0) {
            const int buf = NQ == 2 ? s : (int)((g - 1) & 1);
            const uint32_t par = (uint32_t)((NQ == 2 ? g - 1 : (g - 1) >> 1) & 1);
            ok = mbar_wait_warp(&pv_done[buf], par, abort_flag, wlim);
            if (!ok) break;
            tc_fence_after();
            const float inv = 1.f / l;  // (every row attends itself)
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
            tc_fence_before();
            __syncwarp();
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

template <int D>
cudaError_t launch_pf(const CUtensorMap &tmq, const CUtensorMap &tmk, const CUtensorMap &tmv,
                      const PrefillParams &p, int num_ctas, cudaStream_t stream) {
    static int done_for_device[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (!(dev >= 0 && dev < 64 && done_for_device[dev])) {
        e = cudaFuncSetAttribute(prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 PfCfg<D>::alloc);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) done_for_device[dev] = 1;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_ctas);
    cfg.blockDim = dim3(PfCfg<D>::THREADS);
    cfg.dynamicSmemBytes = PfCfg<D>::alloc;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefill_kernel<D>, tmq, tmk, tmv, p);
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

using namespace kvattn;

extern "C" int gqa_prefill_attn(const void *q, const void *k, const void *v,
                                const int32_t *cu_seqlens, void *out, int B, int N, int Hq, int Hkv,
                                int D, long long q_stride, long long k_stride, long long v_stride,
                                float scale, int window, kvattn_stream_t stream) {
    const char *who = "gqa_prefill_attn";
    api_begin();
    if (!q || !k || !v || !cu_seqlens || !out) return api_failf(KVATTN_ERR_INVALID_ARG, "%s: null pointer", who);
    if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15u) ||
        (reinterpret_cast<uintptr_t>(out) & 31u) || (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u))
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: q, k and v must be 16-byte, out 32-byte aligned", who);
    if (!std::isfinite(scale)) return api_failf(KVATTN_ERR_INVALID_ARG, "%s: scale must be finite", who);
    if (window < 1) return api_failf(KVATTN_ERR_INVALID_ARG, "%s: window must be >= 1 (got %d)", who, window);
    int rc = api_check_sizes(B, Hq, Hkv, D, 1);
    if (rc) return rc;
    if (N < 1) return api_failf(KVATTN_ERR_INVALID_ARG, "%s: N must be positive (got %d)", who, N);
    if (N > (1 << 28)) return api_failf(KVATTN_ERR_UNSUPPORTED, "%s: N = %d rows beyond 2^28", who, N);
    if ((rc = api_check_row_stride(q_stride, Hq, D, who)) || (rc = api_check_row_stride(k_stride, Hkv, D, who)) ||
        (rc = api_check_row_stride(v_stride, Hkv, D, who)))
        return rc;
    int num_sms;
    PrefillParams p = {};
    if ((rc = api_device(&num_sms, &p.err, &p.wait_limit))) return rc;

    p.cu = cu_seqlens;
    p.out = static_cast<uint16_t *>(out);
    p.B = B; p.N = N; p.Hq = Hq; p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.hpg = 1;
    while (p.hpg < kRows && p.G % (2 * p.hpg) == 0) p.hpg *= 2, ++p.hpg_lg;
    p.tpt = kRows / p.hpg;
    p.passes = p.G / p.hpg;
    p.window = window < N ? window : N;
    const float sl = (float)(std::fabs((double)scale) * 1.4426950408889634);
    p.sl = std::isfinite(sl) ? std::fmax(sl, FLT_MIN) : FLT_MAX;  // (masked scores stay -inf at scale 0)
    p.neg = scale < 0.f;
    CUtensorMap tmq, tmk, tmv;
    if ((rc = encode_rows_map(&tmq, q, D, Hq, N, q_stride, p.hpg, p.tpt)) ||
        (rc = encode_rows_map(&tmk, k, D, Hkv, N, k_stride, 1, kRows)) ||
        (rc = encode_rows_map(&tmv, v, D, Hkv, N, v_stride, 1, kRows)))
        return rc;
    // at most one unit per NQ tiles of tokens and one more per sequence
    const int tpu = (D == 256 ? 1 : 2) * p.tpt;
    const long long most = ((long long)N / tpu + B) * Hkv * p.passes;
    const int ctas = (int)(most < num_sms ? most : num_sms);
    cudaError_t e;
    switch (D) {
        case 64: e = launch_pf<64>(tmq, tmk, tmv, p, ctas, reinterpret_cast<cudaStream_t>(stream)); break;
        case 128: e = launch_pf<128>(tmq, tmk, tmv, p, ctas, reinterpret_cast<cudaStream_t>(stream)); break;
        default: e = launch_pf<256>(tmq, tmk, tmv, p, ctas, reinterpret_cast<cudaStream_t>(stream)); break;
    }
    if (e != cudaSuccess) return api_cuda_fail(e, "prefill kernel launch");
    return KVATTN_OK;
}
