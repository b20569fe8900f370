// extend.cu -- gqa_extend_attn and gqa_cross_attn: packed tokens of ragged counts
// over K/V rows in a paged pool, causal behind what their request has cached, or
// over all rows of another sequence, such as an encoder's states.
//
// The kernel is that of prefill.cuh; what differs over a pool:
//  * K/V tiles come through the block table, a box of min(block size, 128) rows
//    a lane of the copy warp, whose ids are loaded 32 at a time; a tile is the
//    positions from a multiple of 128 on, so that boxes are whole blocks;
//  * token t attends [max(0, e - window), e) with e = cached + t + 1 (extend) or all
//    positions (cross); rows that attend nothing are zeroed beside the schedule;
//  * a step's requests bring one token each as often as thousands: the key tiles
//    of all units in a row are cut into equal ranges, a CTA each (units.cuh), so
//    that a single long request fills the chip as 64 ragged ones do.  A unit that
//    a range ends in leaves unnormalised rows O with their maximum and sum (m, l)
//    in the workspace, two pieces a CTA at most, which merge_kernel joins:
//        out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,  M = max m_i;
//  * where requests bring few tokens (extend_few.cu) a unit of up to 32 query rows
//    has them four times in its tile, a warp takes a quarter of a key tile's
//    columns for its copy, and even and odd key tiles go through the two query
//    tiles' buffers, so that a softmax of 32 columns a warp stands behind a key tile
//    and the chains of two overlap.
//
// What bounds it.  Many tokens: what bounds prompt attention, the tensor pipe
// between its turns (four prompts of 2048 tokens behind 6144, 64 heads over 8 of 128:
// 1377 us in a graph, 1397 TFLOP/s, 0.74 of the cuBLAS rate; called, 1412 to 1419), and
// the merge (7 to 10 us where all CTAs leave units of 128 or 256 rows).  Beside prompt
// attention of the same 8192 tokens: 764 us for 753 there (64 heads over 8 of 128; in a
// window of 1024 275 for 228), 421 for 334 (16 over 1 of 256; 178 for 116), 182 for 162
// (16 over 16 of 64; 85 for 67).  Short units: their starts and ends, some
// 4 us each (eight requests of up to 511 tokens in a window of 1024, 16 heads over 1
// of 256: 66 us, of which a CTA's first piece takes 13: instructions and the first
// rows are far away).  Single tokens: memory, 5.5 TB/s (0.81 of
// copy bandwidth) for 32 of up to 8192 positions, 64 heads over 8 of 128, in blocks of
// 16, 5.7 in larger ones; 3.9 for 64 of up to 2048 states, 16 heads of 64, whose units
// are 1 to 16 key tiles long and take 2.5 us to begin and end.  A kernel's local
// memory is L2 here (227 KB of shared memory leave little L1): a stack frame or a
// spill in a loop cost some 1000 cycles a turn under load.  (The form for few rows at
// D = 128 still has two registers spilled, with 720 bytes of loads; where is not known.)
#include <cfloat>
#include <cmath>

#include "../../include/kvattn.h"
#include "prefill.cuh"

namespace kvattn {

namespace {

struct MergeParams {
    const float *ws_o, *ws_ml;
    const int4 *split;  // per CTA: (packed row, tokens, first head, pieces) of the unit it leaves unfinished
    uint16_t *out;
    int Hq, hpg, tpt;
};

constexpr int kMergeThreads = 256;

// (by a warp) row `row` of a unit from its n partial results, the i-th in workspace
// slot at(i), where units have few rows.  The first AHEAD of them are loaded with
// their (m, l), before it is known what they weigh, the others MORE at a time.
template <int D, class At>
__device__ __forceinline__ void join_row(const float *ws_o, const float *ws_ml, int row, At at, int n,
                                         uint16_t *out) {
    constexpr int AHEAD = 8, MORE = 4;
    constexpr int V = D / 32;  // values of a lane
    const int lane = threadIdx.x & 31;
    auto load = [&](int i, float *x) {
        const float *src = ws_o + Partial<D, true>::row(at(i), row) + lane * V;
        if constexpr (V == 2) {
            const float2 f = __ldcg(reinterpret_cast<const float2 *>(src));
            x[0] = f.x;
            x[1] = f.y;
        } else {
            const float4 f = __ldcg(reinterpret_cast<const float4 *>(src));
            x[0] = f.x;
            x[1] = f.y;
            x[2] = f.z;
            x[3] = f.w;
        }
    };
    auto ml_of = [&](int i) {
        return i < n ? __ldcg(reinterpret_cast<const float2 *>(ws_ml + Partial<D, true>::ml(at(i), row)))
                     : make_float2(-INFINITY, 0.f);
    };
    float2 ml = ml_of(lane);
    float x[AHEAD][V];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (i < n) load(i, x[i]);
    float m = ml.x;
    for (int i = 32 + lane; i < n; i += 32) m = fmaxf(m, ml_of(i).x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float o[V], l = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = 0.f;
    for (int i0 = 0; i0 < n; i0 += 32) {
        if (i0 > 0) ml = ml_of(i0 + lane);
        const float w = ml.y > 0.f ? fast_exp2(ml.x - m) : 0.f;
        l += w * ml.y;
        // (a piece that held none of the row's keys weighs nothing, and may hold anything)
        if (i0 == 0) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const float wi = __shfl_sync(0xffffffffu, w, i);
                if (i < n && wi != 0.f) {
#pragma unroll
                    for (int k = 0; k < V; ++k) o[k] = fmaf(wi, x[i][k], o[k]);
                }
            }
        }
        const int e = min(32, n - i0);
        for (int i = i0 == 0 ? AHEAD : 0; i < e; i += MORE) {
            float y[MORE][V];
#pragma unroll
            for (int q = 0; q < MORE; ++q)
                if (i + q < e) load(i0 + i + q, y[q]);
#pragma unroll
            for (int q = 0; q < MORE; ++q) {
                const float wi = __shfl_sync(0xffffffffu, w, min(i + q, 31));
                if (i + q < e && wi != 0.f) {
#pragma unroll
                    for (int k = 0; k < V; ++k) o[k] = fmaf(wi, y[q][k], o[k]);
                }
            }
        }
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
    store_row<V>(out + lane * V, o, 1.f / l);  // (every row attends something)
}

// The same of units of many rows: up to 128 values from d0 on of four rows a warp, 8 of
// every 64 a lane, since the rows' pieces of eight values are side by side.
template <int D, class At>
__device__ __forceinline__ void join_rows(const float *ws_o, const float *ws_ml, int row, At at, int n,
                                          int d0, uint16_t *out, bool write) {
    using P = Partial<D, false>;
    constexpr int C = D > 64 ? 2 : 1;
    const int d = d0 + (threadIdx.x & 31) / 4 * 8;
    auto load = [&](int i, float (&x)[C][8]) {
#pragma unroll
        for (int c = 0; c < C; ++c) ld_global_32b(ws_o + P::row(at(i), row) + (d / 8 + c * 8) * P::STEP, x[c]);
    };
    auto ml_of = [&](int i) { return __ldcg(reinterpret_cast<const float2 *>(ws_ml + P::ml(at(i), row))); };
    float x[2][C][8];  // (two pieces at least; most have no more)
    load(0, x[0]);
    load(1, x[1]);
    const float2 ml0 = ml_of(0), ml1 = ml_of(1);
    float m = fmaxf(ml0.x, ml1.x);
#pragma unroll 4
    for (int i = 2; i < n; ++i) m = fmaxf(m, ml_of(i).x);
    float o[C][8] = {}, l = 0.f;
    auto add = [&](float2 ml, const float (&y)[C][8]) {
        const float w = ml.y > 0.f ? fast_exp2(ml.x - m) : 0.f;
        if (w == 0.f) return;  // (it held none of the row's keys, and may hold anything)
        l += w * ml.y;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int k = 0; k < 8; ++k) o[c][k] = fmaf(w, y[c][k], o[c][k]);
    };
    add(ml0, x[0]);
    add(ml1, x[1]);
#pragma unroll 1
    for (int i = 2; i < n; ++i) {
        load(i, x[0]);
        add(ml_of(i), x[0]);
    }
    const float inv = 1.f / l;  // (every row attends something)
    if (write) {
#pragma unroll
        for (int c = 0; c < C; ++c) store_row<8>(out + d + c * 64, o[c], inv);
    }
}

// Block (c, y): rows of the unit that CTA c leaves unfinished.  What bounds it is
// latency: of the record, then of (m, l) and the rows; with few tokens a request,
// whose keys may be in many pieces, a warp takes a row, else four.
template <int D, bool FEW>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const MergeParams p) {
    constexpr int AT_ONCE = FEW ? 1 : 4, COLS = FEW || D < 128 ? D : 128;
    pdl_launch_dependents();
    pdl_wait_prior();
    const int c = blockIdx.x;
    const int4 u = __ldcg(p.split + c);
    const int rows = u.w > 0 ? u.y * p.hpg : 0;
    auto slot = [&](int i) { return i == 0 ? 2 * c + 1 : 2 * (c + i); };
    const int warp = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5);
    for (int r0 = warp / (D / COLS) * AT_ONCE; r0 < rows; r0 += gridDim.y * (kMergeThreads / 32) / (D / COLS) * AT_ONCE) {
        const int r = FEW ? r0 : min(r0 + (int)(threadIdx.x & 3), rows - 1);
        const int t = r / p.hpg, h = r - t * p.hpg;
        const int row = t / p.tpt * kRows + t % p.tpt * p.hpg + h;
        uint16_t *out = p.out + ((size_t)(u.x + t) * p.Hq + u.z + h) * D;
        if constexpr (FEW)
            join_row<D>(p.ws_o, p.ws_ml, row, slot, u.w, out);
        else
            join_rows<D>(p.ws_o, p.ws_ml, row, slot, u.w, warp % (D / COLS) * COLS, out,
                         r0 + (int)(threadIdx.x & 3) < rows);
    }
}

template <int D>
cudaError_t launch_merge(const MergeParams &p, bool few, int ctas, int parts, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, parts);
    cfg.blockDim = dim3(kMergeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if constexpr (D < 256)
        if (few) return cudaLaunchKernelEx(&cfg, merge_kernel<D, true>, p);
    return cudaLaunchKernelEx(&cfg, merge_kernel<D, false>, p);
}

// 3-D map over a pool [num_blocks, Hkv, block_size, D]: dims (D, block_size,
// num_blocks * Hkv), box (64, min(block_size, 128), 1).
int encode_pool(CUtensorMap *m, const void *base, int D, int block_size, long long heads, int box_rows) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)block_size, (cuuint64_t)heads};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * 2 * (cuuint64_t)block_size};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, 1};
    return api_encode_bf16_3d(m, base, dims, strides, box);
}

int run_extend(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
               const int32_t *kv_lens, const int32_t *cu_seqlens, void *out, int B, int N, int Hq, int Hkv, int D,
               long long q_stride, int num_blocks, int block_size, int max_blocks, float scale, int causal,
               int window, kvattn_stream_t stream_, const char *who) {
    api_begin();
    if (!q || !k_pool || !v_pool || !block_table || !kv_lens || !cu_seqlens || !out)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: null pointer", who);
    if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k_pool) |
          reinterpret_cast<uintptr_t>(v_pool)) & 15u) ||
        (reinterpret_cast<uintptr_t>(out) & 31u) ||
        ((reinterpret_cast<uintptr_t>(cu_seqlens) | reinterpret_cast<uintptr_t>(kv_lens)) & 3u))
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: q and pools must be 16-byte, out 32-byte aligned", who);
    if (!std::isfinite(scale)) return api_failf(KVATTN_ERR_INVALID_ARG, "%s: scale must be finite", who);
    if (window < 1) return api_failf(KVATTN_ERR_INVALID_ARG, "%s: window must be >= 1 (got %d)", who, window);
    PagedPrefillParams p = {};
    int rc, lmax;
    if ((rc = api_check_sizes(B, Hq, Hkv, D, 1))) return rc;
    if ((rc = api_check_paged(block_table, Hkv, block_size, max_blocks, num_blocks, who, &p.lg, &lmax))) return rc;
    if (N < 1) return api_failf(KVATTN_ERR_INVALID_ARG, "%s: N must be positive (got %d)", who, N);
    if (N > (1 << 28)) return api_failf(KVATTN_ERR_UNSUPPORTED, "%s: N = %d rows beyond 2^28", who, N);
    if ((rc = api_check_row_stride(q_stride, Hq, D, who))) return rc;
    int ctas;
    if ((rc = api_device(&ctas, &p.err, &p.wait_limit))) return rc;

    p.cu = cu_seqlens;
    p.out = static_cast<uint16_t *>(out);
    p.B = B; p.N = N; p.Hq = Hq; p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.hpg = 1;
    while (p.hpg < kRows && p.G % (2 * p.hpg) == 0) p.hpg *= 2;
    p.tpt = kRows / p.hpg;
    // Groups of no power of two: with up to two units' tokens a request on average,
    // all heads of a group in one tile, by a power of two of tokens, so that a
    // request's keys are read once for the group; beyond, every row of the tile counts.
    // (The lengths are on the device; padding rows and requests without tokens count in
    // the averages, too, and can have a call take the other form.)
    // 16 requests of 4096 positions, one pass / as many as it takes: 20 heads over 4
    // of 128 with 1 token 37 / 81 us, 64 tokens 72 / 125, 128 126 / 133; 24 over 2 of
    // 128 with 32 tokens 48 / 54, 64 75 / 67; 48 over 1 of 256 with 4 38 / 38, 8 50 / 46.
    if (p.G <= kRows && p.hpg < p.G) {
        int tpt = 1;
        while (2 * tpt * p.G <= kRows) tpt *= 2;
        if ((long long)N <= 2LL * B * tpt * (D == 256 ? 1 : 2)) {
            p.hpg = p.G;
            p.tpt = tpt;
        }
    }
    p.passes = p.G / p.hpg;
    p.rows = p.hpg * p.tpt;
    p.q_bytes = p.rows * D * 2;
    p.tpu_lg = 0;
    while (1 << p.tpu_lg < (D == 256 ? 1 : 2) * p.tpt) ++p.tpu_lg;
    // Units of few rows in a form of their own where a request has few on average
    // (with it / without, 16 requests of 4096 positions: 16 heads of 64 56 / 91 us, 32
    // over 2 of 64 21 / 22, with 2 tokens 25 / 22; 64 over 8 of 128 56 / 59, with 2 60 /
    // 60, 32 over 2 of 128 30 / 26; at D = 256 it loses).  An average that idle requests
    // bring down is not borne out: 16 requests of 64 tokens behind 4032, 16 heads over 16
    // of 64, 80 us, beside 240 without tokens 103; 64 single tokens of 64 over 8 of 128
    // 100 us, with one row of padding 102.
    int few = 0;
    if (D < 256 && p.hpg <= 32 && (long long)N * p.hpg <= (D == 64 ? 16LL : 8LL) * B)
        for (few = 1; 2 * few * p.hpg <= 32;) few *= 2;  // tokens whose rows fit a quarter of the tile
    p.few_tok = few;
    p.few_bytes = few * p.hpg * D * 2;
    p.window = window < lmax ? window : lmax;
    const float sl = (float)(std::fabs((double)scale) * 1.4426950408889634);
    p.sl = std::isfinite(sl) ? std::fmax(sl, FLT_MIN) : FLT_MAX;  // (masked scores stay -inf at scale 0)
    p.neg = scale < 0.f;
    p.table = block_table;
    p.kv_lens = kv_lens;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.box_lg = p.lg < 7 ? p.lg : 7;
    p.box = 1 << p.box_lg;
    p.causal = causal;
    // Costs as measured, in fifths of a key tile of two query tiles (1.7 us at D =
    // 128; of one 1.35, of few rows the same for all).  A unit's start and end (its
    // copies' latency, the output's read-out, a join) is 2 tiles' work, at D = 64
    // with few rows 5: 64 requests of 16 heads of 64 over up to 2048 states 91 us
    // with 2, 75 with 5, 78 with 10; 8192 tokens of 64 heads over 8 of 128 770 with 2,
    // 755 with 1.6 (and the mixed calls the same), of 16 over 1 of 256 408 with 2.6, 412
    // with 2, 429 with 1.6.
    p.w2 = 5;
    p.w1 = p.few_tok || D == 256 ? 5 : 4;
    p.cost_piece = p.few_tok ? (D == 64 ? 25 : 10) : D == 256 ? 13 : 10;
    p.min_range = p.w2 + p.cost_piece;

    CUtensorMap tmq, tmq4, tmk, tmv;
    const long long heads = (long long)num_blocks * Hkv;
    if ((rc = encode_rows_map(&tmq, q, D, Hq, N, q_stride, p.hpg, p.tpt)) ||
        (rc = encode_rows_map(&tmq4, q, D, Hq, N, q_stride, few ? p.hpg : 1, few ? few : 1)) ||
        (rc = encode_pool(&tmk, k_pool, D, block_size, heads, p.box)) ||
        (rc = encode_pool(&tmv, v_pool, D, block_size, heads, p.box)))
        return rc;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const int slot_rows = (D == 256 ? 1 : 2) * kRows;
    const size_t rows = (size_t)2 * ctas * slot_rows;  // two pieces a CTA
    WorkspaceLease ws;  // (held until the merge is launched)
    if ((rc = api_call_workspace(stream, rows * (D + 2) * sizeof(float) + (size_t)ctas * sizeof(int4), &ws)))
        return rc;
    p.ws_o = static_cast<float *>(ws.ptr);
    p.ws_ml = p.ws_o + rows * D;
    p.split = reinterpret_cast<int4 *>(p.ws_ml + rows * 2);

    MergeParams m = {p.ws_o, p.ws_ml, p.split, p.out, Hq, p.hpg, p.tpt};
    const long long unit_rows = (long long)N * p.hpg < slot_rows ? (long long)N * p.hpg : slot_rows;
    const int share = few || D == 256 ? 16 : 32;  // rows of a block
    const int parts = (int)((unit_rows + share - 1) / share);
    cudaError_t e;
    switch (D) {
        case 64:
            e = p.few_tok ? launch_extend_few(D, tmq, tmk, tmv, &p, ctas, stream, tmq4)
                          : launch_pf<64, true, false>(tmq, tmk, tmv, p, ctas, stream, tmq4);
            if (e == cudaSuccess) e = launch_merge<64>(m, p.few_tok > 0, ctas, parts, stream);
            break;
        case 128:
            e = p.few_tok ? launch_extend_few(D, tmq, tmk, tmv, &p, ctas, stream, tmq4)
                          : launch_pf<128, true, false>(tmq, tmk, tmv, p, ctas, stream, tmq4);
            if (e == cudaSuccess) e = launch_merge<128>(m, p.few_tok > 0, ctas, parts, stream);
            break;
        default:
            e = launch_pf<256, true, false>(tmq, tmk, tmv, p, ctas, stream, tmq4);
            if (e == cudaSuccess) e = launch_merge<256>(m, p.few_tok > 0, ctas, parts, stream);
            break;
    }
    if (e != cudaSuccess) return api_cuda_fail(e, "paged prompt attention launch");
    return KVATTN_OK;
}

}  // namespace

}  // namespace kvattn

using namespace kvattn;

extern "C" {

int gqa_extend_attn(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
                    const int32_t *seq_lens, const int32_t *cu_seqlens, void *out, int B, int N, int Hq, int Hkv,
                    int D, long long q_stride, int num_blocks, int block_size, int max_blocks, float scale,
                    int window, kvattn_stream_t stream) {
    return run_extend(q, k_pool, v_pool, block_table, seq_lens, cu_seqlens, out, B, N, Hq, Hkv, D, q_stride,
                      num_blocks, block_size, max_blocks, scale, 1, window, stream, "gqa_extend_attn");
}

int gqa_cross_attn(const void *q, const void *k_pool, const void *v_pool, const int32_t *block_table,
                   const int32_t *kv_lens, const int32_t *cu_seqlens, void *out, int B, int N, int Hq, int Hkv,
                   int D, long long q_stride, int num_blocks, int block_size, int max_blocks, float scale,
                   kvattn_stream_t stream) {
    return run_extend(q, k_pool, v_pool, block_table, kv_lens, cu_seqlens, out, B, N, Hq, Hkv, D, q_stride,
                      num_blocks, block_size, max_blocks, scale, 0, 0x7fffffff, stream, "gqa_cross_attn");
}

}  // extern "C"
