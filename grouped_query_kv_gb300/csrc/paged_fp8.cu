// paged_fp8.cu -- writing packed K/V rows into a paged 8-bit pool: E4M3 codes
// with one power-of-two scale per (block, K/V head) ("The Basics of
// Transformer Inference", item "Quantization"; "Machine Learning Engineering
// and AI Systems at Scale", section "Quantization").
//
//     need  = smallest 2^e, e >= -100, with absmax(new rows) <= 448 * 2^e
//     scale = max(scale the block's earlier rows have, need)
//     code  = E4M3(x / scale);  earlier codes: E4M3(value * old / scale)
// Powers of two make the quotient exact, so the only rounding is E4M3's (and
// a code written before its scale grew is the code it would have had, unless
// its value fell below E4M3's normal range).
//
// A block of 128 threads writes (pool block, K/V head) pairs of K and of V one
// after the other: it owns their scales, so nothing is shared between blocks
// and no atomic decides an order.  `split` consecutive blocks of the grid share
// a candidate: x < B is request x's first touched pool block (the one that may
// hold earlier rows), x >= B the pool blocks that start inside the bs packed
// rows from (x - B) bs; each takes a run of its heads, K and V (long runs where
// there are many candidates: a search for the request then serves them all, and
// blocks that run together read neighbouring heads of the same rows; with the
// candidates consecutive instead some 2 % slower).
// What bounds it is the copy: 2 bytes read and 1 written per value.  Up to
// kHeld 16-byte vectors a thread the new rows stay in registers between the
// search for the largest and the rounding; longer blocks read them again.
// 32 prompts, 67 k rows of 8 x 128 into blocks of 64: 65.0 us, 0.96 of the
// measured copy rate; 64 single rows 4.3 us.
#include "../../include/kvattn.h"
#include "internal.h"
#include "ptx.cuh"
#include "fp8_codec.cuh"

namespace kvattn {

namespace {

constexpr int kThreads = 128;
constexpr int kMaxBlock = 1024;  // positions of a block at most

struct Append8Params {
    uint8_t *codes[2];           // K, V: [num_blocks, Hkv, bs, D]
    float *scales[2];            // [num_blocks, Hkv]
    const uint16_t *rows[2];     // packed new rows
    long long stride[2];         // elements from row to row
    const int32_t *table, *cached, *cu;
    unsigned int *err;
    int B, N, Hkv, lg, max_blocks, num_blocks;
    int split;                   // blocks of the grid per candidate
};

// Exponent of the smallest power of two s (>= 2^-100) with a <= 448 s,
// a >= 0: a = 1.f 2^x <= 1.75 2^(8 + e)  <=>  e = x - 8 if 1.f <= 1.75, else x - 7.
__device__ __forceinline__ int scale_exponent(float a) {
    const uint32_t bits = __float_as_uint(a);
    const int x = (int)(bits >> 23) - 127;
    const int e = x - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return max(e, -100);
}

// Eight bf16 values (four words, low half first) as binary32.
__device__ __forceinline__ void unpack8(uint4 raw, float (&x)[8]) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// Two codes times a power of two <= 1, as codes.
__device__ __forceinline__ uint32_t rescale2(uint32_t two, float f) {
    const float2 v = e4m3x2_value((uint16_t)two);
    return e4m3x2_from_f32(v.x * f, v.y * f);
}

constexpr int kHeld = 8;

__device__ __forceinline__ float absmax8(uint4 raw, float a) {
    float x[8];
    unpack8(raw, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) a = fmaxf(a, fabsf(x[j]));
    return a;
}
__device__ __forceinline__ uint2 codes8(uint4 raw, float inv) {
    float x[8];
    unpack8(raw, x);
    return make_uint2((uint32_t)e4m3x2_from_f32(x[0] * inv, x[1] * inv) |
                          ((uint32_t)e4m3x2_from_f32(x[2] * inv, x[3] * inv) << 16),
                      (uint32_t)e4m3x2_from_f32(x[4] * inv, x[5] * inv) |
                          ((uint32_t)e4m3x2_from_f32(x[6] * inv, x[7] * inv) << 16));
}

// Writes m packed rows from row t to positions pos.. (of one pool block) of
// request b, for head h of K (kv = 0) or V; called by the whole block, `turn`
// counting the blocks that it wrote.
template <int D>
__device__ __forceinline__ void write_block(const Append8Params &p, int kv, int h, int b, int pos, int t,
                                            int m, float (*red)[4], int &turn) {
    constexpr int VPR = D / 8;               // 16-byte vectors of a new row
    constexpr int RPP = kThreads / VPR;      // rows per pass
    const int tid = threadIdx.x;
    const int blk = p.table[(size_t)b * p.max_blocks + (pos >> p.lg)];
    if (blk < 0 || blk >= p.num_blocks) {
        if (tid == 0) atomicCAS(p.err, 0u, (unsigned int)DEV_ERR_BOUNDS);
        return;
    }
    const int r0 = pos & ((1 << p.lg) - 1);
    const size_t bh = (size_t)blk * p.Hkv + h;
    uint8_t *codes = p.codes[kv] + (bh << p.lg) * D;
    float *scale = p.scales[kv] + bh;
    const int row = tid / VPR;
    const long long stride = p.stride[kv];
    const uint16_t *src = p.rows[kv] + (t + row) * stride + (size_t)h * D + (tid % VPR) * 8;
    const float old = r0 > 0 ? *scale : 0.f;
    const bool held = m <= kHeld * RPP;

    uint4 raw[kHeld];
    float a = 0.f;
    if (held) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            raw[i] = row + i * RPP < m ? __ldcs(reinterpret_cast<const uint4 *>(src + i * RPP * stride))
                                       : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < kHeld; ++i) a = absmax8(raw[i], a);
    } else {
        for (int r = 0; row + r < m; r += kHeld * RPP) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                raw[i] = row + r + i * RPP < m ? *reinterpret_cast<const uint4 *>(src + (r + i * RPP) * stride)
                                               : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int i = 0; i < kHeld; ++i) a = absmax8(raw[i], a);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    // (two buffers in turn: the barrier of the next block written keeps the one
    // after it from this buffer until every thread has read it)
    float *mine = red[turn++ & 1];
    if ((tid & 31) == 0) mine[tid >> 5] = a;
    __syncthreads();              // (every thread has read the old scale, too)
    a = fmaxf(fmaxf(mine[0], mine[1]), fmaxf(mine[2], mine[3]));
    const float now = fmaxf(old, __uint_as_float((uint32_t)(127 + scale_exponent(a)) << 23));
    if (tid == 0) *scale = now;
    if (r0 > 0 && now > old) {
        // the earlier rows' codes for the larger scale
        const float f = old / now;
        uint4 *c = reinterpret_cast<uint4 *>(codes);
        for (int i = tid; i < r0 * (D / 16); i += kThreads) {
            const uint4 w = c[i];
            const uint32_t in[4] = {w.x, w.y, w.z, w.w};
            uint32_t o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[j] = rescale2(in[j] & 0xffffu, f) | (rescale2(in[j] >> 16, f) << 16);
            c[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
    const float inv = 1.f / now;  // exact: 2^-120 .. 2^100
    uint8_t *dst = codes + (size_t)(r0 + row) * D + (tid % VPR) * 8;
    if (held) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (row + i * RPP < m) __stcs(reinterpret_cast<uint2 *>(dst + i * RPP * D), codes8(raw[i], inv));
    } else {
        for (int r = 0; row + r < m; r += kHeld * RPP) {
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                if (row + r + i * RPP < m)
                    raw[i] = *reinterpret_cast<const uint4 *>(src + (r + i * RPP) * stride);
#pragma unroll
            for (int i = 0; i < kHeld; ++i)
                if (row + r + i * RPP < m)
                    *reinterpret_cast<uint2 *>(dst + (size_t)(r + i * RPP) * D) = codes8(raw[i], inv);
        }
    }
}

// A request's packed rows and positions; false if it writes nothing.
__device__ __forceinline__ bool request(const Append8Params &p, int b, int *first, int *n, int *c, bool *bad) {
    const int a = p.cu[b], e = p.cu[b + 1];
    *first = a;
    *n = e - a;
    *c = p.cached[b];
    *bad = a < 0 || e < a || e > p.N || *c < 0 ||
           (long long)*c + (e - a) > ((long long)p.max_blocks << p.lg);
    return !*bad && e > a;
}

// (p stays where the launch put it: indexed by K and V, a plain parameter is
// copied to each thread's stack, 71 us for 66 below; ten blocks an SM, 48
// registers: 65.0 us, eight 66.0, eleven 69.3)
template <int D>
__global__ void __launch_bounds__(kThreads, 10) append_paged8_kernel(const __grid_constant__ Append8Params p) {
    __shared__ float red[2][4];
    __shared__ int found;
    __shared__ int s_b[kMaxBlock], s_t[kMaxBlock];
    pdl_launch_dependents();
    pdl_wait_prior();
    const int bs = 1 << p.lg;
    const int x = (int)(blockIdx.x / (unsigned)p.split), part = (int)(blockIdx.x - (unsigned)x * p.split);
    const int hk0 = part * 2 * p.Hkv / p.split, hk1 = (part + 1) * 2 * p.Hkv / p.split;
    int first, n, c, turn = 0;
    bool bad;
    if (x < p.B) {
        const int b = x;
        const bool some = request(p, b, &first, &n, &c, &bad);
        if (bad && part == 0 && threadIdx.x == 0) atomicCAS(p.err, 0u, (unsigned int)DEV_ERR_BOUNDS);
        if (some)
            for (int hk = hk0; hk < hk1; ++hk)
                write_block<D>(p, hk & 1, hk >> 1, b, c, first, min(n, bs - (c & (bs - 1))), red, turn);
        return;
    }
    // pool blocks that start at packed rows [t0, t1), the requests' first
    // touched ones aside: of bs consecutive rows of a request one starts a block
    const int t0 = (x - p.B) << p.lg, t1 = min(t0 + bs, p.N);
    // the last request that starts at or before t0, 32 probes at a time
    int lo = 0, span = p.B;  // it is in [lo, lo + span)
    while (span > 1) {
        const int each = (span + 31) / 32, at = lo + (int)(threadIdx.x & 31) * each;
        const bool before = (threadIdx.x & 31) * each < span && p.cu[at] <= t0;
        const int past = __popc(__ballot_sync(0xffffffffu, before));  // (cu does not decrease)
        const int step = max(past - 1, 0) * each;
        lo += step;
        span = min(each, span - step);
    }
    if (threadIdx.x == 0) found = 0;
    __syncthreads();
    for (int b = lo + threadIdx.x; b < p.B && p.cu[b] < t1; b += kThreads) {
        if (!request(p, b, &first, &n, &c, &bad)) continue;
        const int t = max(t0, first + 1);
        const int start = t + ((bs - ((c + t - first) & (bs - 1))) & (bs - 1));
        if (start < min(t1, first + n)) {
            const int i = atomicAdd(&found, 1);
            if (i < kMaxBlock) {
                s_b[i] = b;
                s_t[i] = start;
            }
        }
    }
    __syncthreads();
    const int blocks = min(found, kMaxBlock);
    for (int i = 0; i < blocks; ++i) {
        const int b = s_b[i], t = s_t[i];
        request(p, b, &first, &n, &c, &bad);
        for (int hk = hk0; hk < hk1; ++hk)
            write_block<D>(p, hk & 1, hk >> 1, b, c + t - first, t, min(bs, first + n - t), red, turn);
    }
}

}  // namespace

}  // namespace kvattn

using namespace kvattn;

extern "C" int kv_append_paged_fp8(void *k_codes, void *v_codes, float *k_scale, float *v_scale,
                                   const void *k_new, const void *v_new, const int32_t *block_table,
                                   const int32_t *cached_lens, const int32_t *cu_seqlens, int B, int N,
                                   int Hkv, int D, long long k_stride, long long v_stride,
                                   int num_blocks, int block_size, int max_blocks,
                                   kvattn_stream_t stream) {
    const char *who = "kv_append_paged_fp8";
    api_begin();
    if (!k_codes || !v_codes || !k_scale || !v_scale || !k_new || !v_new || !block_table || !cached_lens ||
        !cu_seqlens)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: null pointer", who);
    if (((reinterpret_cast<uintptr_t>(k_codes) | reinterpret_cast<uintptr_t>(v_codes) |
          reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15u) ||
        ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale) |
          reinterpret_cast<uintptr_t>(cached_lens) | reinterpret_cast<uintptr_t>(cu_seqlens)) & 3u))
        return api_failf(KVATTN_ERR_INVALID_ARG,
                         "%s: pointers must be 16-byte aligned (scales and int32 arrays 4)", who);
    int rc, lg, lmax;
    if ((rc = api_check_sizes(B, Hkv, Hkv, D, 1))) return rc;
    if ((rc = api_check_paged(block_table, Hkv, block_size, max_blocks, num_blocks, who, &lg, &lmax))) return rc;
    if (block_size > kMaxBlock)
        return api_failf(KVATTN_ERR_UNSUPPORTED, "%s: an 8-bit block holds at most %d positions (got %d)", who,
                         kMaxBlock, block_size);
    if (N < 1) return api_failf(KVATTN_ERR_INVALID_ARG, "%s: N must be positive (got %d)", who, N);
    if (N > (1 << 28)) return api_failf(KVATTN_ERR_UNSUPPORTED, "%s: N = %d rows beyond 2^28", who, N);
    if ((rc = api_check_row_stride(k_stride, Hkv, D, who)) ||
        (rc = api_check_row_stride(v_stride, Hkv, D, who)))
        return rc;
    Append8Params p = {};
    int ctas;
    unsigned int wait_limit;
    if ((rc = api_device(&ctas, &p.err, &wait_limit))) return rc;
    p.codes[0] = static_cast<uint8_t *>(k_codes);
    p.codes[1] = static_cast<uint8_t *>(v_codes);
    p.scales[0] = k_scale;
    p.scales[1] = v_scale;
    p.rows[0] = static_cast<const uint16_t *>(k_new);
    p.rows[1] = static_cast<const uint16_t *>(v_new);
    p.stride[0] = k_stride;
    p.stride[1] = v_stride;
    p.table = block_table;
    p.cached = cached_lens;
    p.cu = cu_seqlens;
    p.B = B;
    p.N = N;
    p.Hkv = Hkv;
    p.lg = lg;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    cudaLaunchConfig_t cfg = {};
    // candidates, and enough splits of the heads to give every SM 64 blocks (65 thousand
    // rows of 8 heads of 128: 24 blocks 67.2 us, 64 65.1, 128 64.8)
    const long long cand = (long long)B + ((long long)N + block_size - 1) / block_size;
    const long long split = (64LL * ctas + cand - 1) / cand;
    p.split = (int)(split < 2 * Hkv ? split : 2 * Hkv);
    cfg.gridDim = dim3((unsigned)(cand * p.split));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = D == 64    ? cudaLaunchKernelEx(&cfg, append_paged8_kernel<64>, p)
                    : D == 128 ? cudaLaunchKernelEx(&cfg, append_paged8_kernel<128>, p)
                               : cudaLaunchKernelEx(&cfg, append_paged8_kernel<256>, p);
    if (e != cudaSuccess) return api_cuda_fail(e, "paged 8-bit append launch");
    return KVATTN_OK;
}
