// rope.cu -- queries and keys on their way into attention: the norm of each
// head, the rotation by its token's position, and the rows' write, in one pass.
//
// Mathematics, per token i and head h (x: the head's D values, fp32 from bf16):
//     y_d = x_d / sqrt(mean_d x_d^2 + eps) * w_d       (where weights are given)
//     (a, b) -> (a c_j - b s_j, a s_j + b c_j)          j < rope_dim / 2
// with c, s row positions[i] of the tables and (a, b) the values j and
// j + rope_dim / 2, or 2 j and 2 j + 1; dims from rope_dim on pass through.  One
// rounding to bf16, at the end: norm and rotation in bf16 one after the other
// would round three times.
//
// Layout.  A head's row is D / 8 lanes, four values of each half of its rotated
// dims (or 16 bytes of neighbours) a lane, so that a lane has both partners of its
// rotations.  A warp takes up to 8 x 32 / (D / 8) heads of one token, with all their
// loads in flight (fewer where tokens are few); a lane's cosines and sines, times the weights, serve all of
// them.  The heads are the token's queries, then its keys, then its values, which
// are copied.
//
// What bounds it: HBM, every value read once and written once: 16 384 tokens of 64
// heads over 8 of 128 with norms 115 us (5.9 TB/s, 0.87 of the measured copy rate;
// 107 without norms; 197 with 16 bytes of a row a lane, partners met by shuffles and
// rows of any kind in a warp: instructions).  64 such tokens 2.4 us: a launch and the
// chain of position, table and rows.
#include <cmath>
#include <cuda_bf16.h>

#include "../../include/kvattn.h"
#include "internal.h"
#include "ptx.cuh"

namespace kvattn {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 8;  // head rows per lane at most

struct RopeParams {
    const uint2 *q, *k, *v;
    const int32_t *pos;
    const float *cos, *sin;
    const float *qw, *kw;      // [D], or null: no norm
    const long long *slots;    // null: no pool
    uint2 *q_out, *k_out;      // k_out null: the pool takes the keys
    uint2 *k_pool, *v_pool;
    unsigned int *err;
    long long q_stride, k_stride, v_stride, qo_stride, ko_stride;  // of four values, from row to row
    long long num_slots;
    int N, Hq, Hkv;
    int chunks, q_chunks, k_chunks;  // warps per token: of all, of q, of k (and of v)
    int q_per, k_per;                // head rows of their lanes
    int half;                  // rope_dim / 2
    int max_pos;
    int lg;                    // log2(block_size)
    float eps;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf_pair(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Four values in two pairs.
struct Four {
    float2 x, y;
};
// (Plain loads: a kernel that starts before the one in front of it ends may not take
// what that one writes, or the one before it wrote, through the read-only path.)
__device__ __forceinline__ Four load4(const float *src) {
    const float4 f = *reinterpret_cast<const float4 *>(src);
    return {make_float2(f.x, f.y), make_float2(f.z, f.w)};
}
__device__ __forceinline__ Four times(Four a, Four b) { return {mul2(a.x, b.x), mul2(a.y, b.y)}; }
__device__ __forceinline__ Four times(Four a, float f) {
    return {mul2(a.x, make_float2(f, f)), mul2(a.y, make_float2(f, f))};
}

// D head dims; NEXT: neighbours rotate together, else values rope_dim / 2 apart.
template <int D, bool NEXT>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    constexpr int LP = D / 8;      // lanes of a head's row
    constexpr int VPW = 32 / LP;   // head rows of a warp at once
    constexpr int HV = D / 4;      // vectors of four values of a head
    pdl_launch_dependents();
    pdl_wait_prior();
    const int lane = threadIdx.x & 31, l = lane % LP;
    // a block has one chunk of eight tokens' heads, the next block the next chunk
    const unsigned group = blockIdx.x / (unsigned)p.chunks;
    const int chunk = (int)(blockIdx.x - group * (unsigned)p.chunks);
    const long long row = (long long)group * (kRopeThreads / 32) + (threadIdx.x >> 5);
    if (row >= p.N) return;
    const int pos = p.pos[row];

    // what the chunk's heads are (the same in the whole block), and which the lane's
    const int kind = chunk < p.q_chunks ? 0 : chunk < p.q_chunks + p.k_chunks ? 1 : 2;
    const int nth = chunk - (kind == 0 ? 0 : kind == 1 ? p.q_chunks : p.q_chunks + p.k_chunks);
    const int per = (kind == 0 ? p.q_per : p.k_per) * VPW;
    const int h0 = nth * per + lane / LP, h1 = min(nth * per + per, kind == 0 ? p.Hq : p.Hkv);
    const uint2 *src = (kind == 0 ? p.q + row * p.q_stride : kind == 1 ? p.k + row * p.k_stride : p.v + row * p.v_stride) +
                       h0 * HV;
    // the lane's vectors of a head: of the first and the second partners, or of two
    // that pass through
    const bool turns = l < p.half / 4;
    const int va = NEXT ? 2 * l : turns ? l : p.half / 2 + 2 * (l - p.half / 4);
    const int vb = NEXT || !turns ? va + 1 : l + p.half / 4;
    uint2 a[kRopeRows], b[kRopeRows];
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) {
        a[u] = b[u] = make_uint2(0u, 0u);
        if (h0 + u * VPW < h1) {
            if constexpr (NEXT) {
                const uint4 x = __ldcs(reinterpret_cast<const uint4 *>(src + u * (VPW * HV)) + l);
                a[u] = make_uint2(x.x, x.y);
                b[u] = make_uint2(x.z, x.w);
            } else {
                a[u] = __ldcs(src + u * (VPW * HV) + va);
                b[u] = __ldcs(src + u * (VPW * HV) + vb);
            }
        }
    }
    const bool there = pos >= 0 && pos < p.max_pos;
    if (pos >= p.max_pos && chunk == 0 && lane == 0) atomicCAS(p.err, 0u, (unsigned int)DEV_ERR_BOUNDS);
    // where the rows go: a head's, and the elements from one of the lane's to the next
    uint2 *dst;
    long long step = VPW * HV;
    bool keep = true;
    if (kind == 0) {
        dst = p.q_out + row * p.qo_stride + h0 * HV;
    } else if (!p.slots) {
        dst = p.k_out + row * p.ko_stride + h0 * HV;
    } else {
        const long long slot = there ? p.slots[row] : -1;
        keep = slot >= 0 && slot < p.num_slots;
        if (slot >= p.num_slots && kind == 1 && nth == 0 && lane == 0)
            atomicCAS(p.err, 0u, (unsigned int)DEV_ERR_BOUNDS);
        dst = (kind == 1 ? p.k_pool : p.v_pool) +
              ((((keep ? slot >> p.lg : 0) * p.Hkv + h0) << p.lg) + (slot & ((1 << p.lg) - 1))) * HV;
        step <<= p.lg;
    }
    auto put = [&](int u, uint2 f, uint2 g) {
        if (!keep || h0 + u * VPW >= h1) return;
        uint2 *to = dst + u * step;
        if constexpr (NEXT) {
            *reinterpret_cast<uint4 *>(to + va) = make_uint4(f.x, f.y, g.x, g.y);
        } else {
            to[va] = f;
            to[vb] = g;
        }
    };
    if (kind == 2) {
#pragma unroll
        for (int u = 0; u < kRopeRows; ++u) put(u, a[u], b[u]);
        return;
    }
    if (!there) {
#pragma unroll
        for (int u = 0; u < kRopeRows; ++u) put(u, make_uint2(0u, 0u), make_uint2(0u, 0u));
        return;
    }
    Four c = {make_float2(1.f, 1.f), make_float2(1.f, 1.f)}, s = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    if (turns) {
        const long long at = (long long)pos * p.half + 4 * l;
        c = load4(p.cos + at);
        s = load4(p.sin + at);
    }
    // with weights wa, wb of the two vectors: a' = a wa c - b wb s, b' = a wa s + b wb c
    Four ac = c, as = s, bc = c, bs = times(s, -1.f);
    const float *wp = kind == 0 ? p.qw : p.kw;
    if (wp) {
        Four wa, wb;
        if constexpr (NEXT) {
            const Four e = load4(wp + 8 * l), f = load4(wp + 8 * l + 4);
            wa = {make_float2(e.x.x, e.y.x), make_float2(f.x.x, f.y.x)};
            wb = {make_float2(e.x.y, e.y.y), make_float2(f.x.y, f.y.y)};
        } else {
            wa = load4(wp + 4 * va);
            wb = load4(wp + 4 * vb);
        }
        ac = times(ac, wa);
        as = times(as, wa);
        bc = times(bc, wb);
        bs = times(bs, wb);
    }
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) {
        if (u * VPW >= per) break;  // (the same in every lane)
        Four x, y;
        if constexpr (NEXT) {
            x = {make_float2(bf_lo(a[u].x), bf_lo(a[u].y)), make_float2(bf_lo(b[u].x), bf_lo(b[u].y))};
            y = {make_float2(bf_hi(a[u].x), bf_hi(a[u].y)), make_float2(bf_hi(b[u].x), bf_hi(b[u].y))};
        } else {
            x = {make_float2(bf_lo(a[u].x), bf_hi(a[u].x)), make_float2(bf_lo(a[u].y), bf_hi(a[u].y))};
            y = {make_float2(bf_lo(b[u].x), bf_hi(b[u].x)), make_float2(bf_lo(b[u].y), bf_hi(b[u].y))};
        }
        Four xt = times(x, ac), yt = times(y, bc);
        if (turns) {  // (elsewhere 0 times an infinity is none of its business)
            xt = {fma2(y.x, bs.x, xt.x), fma2(y.y, bs.y, xt.y)};
            yt = {fma2(x.x, as.x, yt.x), fma2(x.y, as.y, yt.y)};
        }
        if (wp) {
            const float2 q = fma2(x.x, x.x, fma2(x.y, x.y, fma2(y.x, y.x, mul2(y.y, y.y))));
            float ss = q.x + q.y;
#pragma unroll
            for (int o = LP / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float r = rsqrtf(ss * (1.f / D) + p.eps);
            xt = times(xt, r);
            yt = times(yt, r);
        }
        if constexpr (NEXT)
            put(u, make_uint2(bf_pair(xt.x.x, yt.x.x), bf_pair(xt.x.y, yt.x.y)),
                make_uint2(bf_pair(xt.y.x, yt.y.x), bf_pair(xt.y.y, yt.y.y)));
        else
            put(u, make_uint2(bf_pair(xt.x.x, xt.x.y), bf_pair(xt.y.x, xt.y.y)),
                make_uint2(bf_pair(yt.x.x, yt.x.y), bf_pair(yt.y.x, yt.y.y)));
    }
}

template <int D>
cudaError_t launch_rope(const RopeParams &p, bool next, unsigned grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return next ? cudaLaunchKernelEx(&cfg, rope_kernel<D, true>, p) : cudaLaunchKernelEx(&cfg, rope_kernel<D, false>, p);
}

bool off(const void *p, unsigned mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; }

// What both calls check, and the launch.
int run_rope(RopeParams p, int D, int rope_dim, long long q_stride, long long k_stride, long long v_stride,
             long long qo_stride, long long ko_stride, int interleaved, kvattn_stream_t stream, const char *who) {
    if (off(p.q, 15) || off(p.k, 15) || off(p.v, 15) || off(p.cos, 15) || off(p.sin, 15) || off(p.qw, 15) ||
        off(p.kw, 15) || off(p.q_out, 15) || off(p.k_out, 15) || off(p.k_pool, 15) || off(p.v_pool, 15) ||
        off(p.pos, 3) || off(p.slots, 7))
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned (positions 4, slots 8)", who);
    int rc;
    if ((rc = api_check_sizes(1, p.Hq, p.Hkv, D, 1))) return rc;
    if (p.N < 1) return api_failf(KVATTN_ERR_INVALID_ARG, "%s: N must be positive (got %d)", who, p.N);
    if (p.N > (1 << 28)) return api_failf(KVATTN_ERR_UNSUPPORTED, "%s: N = %d rows beyond 2^28", who, p.N);
    if (rope_dim < 16 || rope_dim > D || rope_dim % 16)
        return api_failf(KVATTN_ERR_UNSUPPORTED, "%s: rope_dim must be a multiple of 16 in [16, D] (got %d)", who,
                         rope_dim);
    if (p.max_pos < 1)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: max_pos must be positive (got %d)", who, p.max_pos);
    if (!std::isfinite(p.eps) || p.eps < 0.f)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: eps must be finite and not negative", who);
    if ((rc = api_check_row_stride(q_stride, p.Hq, D, who)) || (rc = api_check_row_stride(k_stride, p.Hkv, D, who)) ||
        (rc = api_check_row_stride(v_stride, p.Hkv, D, who)) || (rc = api_check_row_stride(qo_stride, p.Hq, D, who)) ||
        (rc = api_check_row_stride(ko_stride, p.Hkv, D, who)))
        return rc;
    int ctas;
    unsigned int wait_limit;
    if ((rc = api_device(&ctas, &p.err, &wait_limit))) return rc;
    p.q_stride = q_stride / 4;
    p.k_stride = k_stride / 4;
    p.v_stride = v_stride / 4;
    p.qo_stride = qo_stride / 4;
    p.ko_stride = ko_stride / 4;
    p.half = rope_dim / 2;
    const int at_once = 32 / (D / 8);  // head rows of a warp
    const unsigned long long groups = ((unsigned long long)p.N + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    // head rows a lane: as many as leave two blocks an SM, else one at least (64 heads over
    // 8 of 128: a token 2.1 us for 2.6, 64 2.4 for 3.2, 256 3.3 for 4.1 with eight; with
    // three blocks an SM 256 take 4.1, too, and 512 5.3 for 4.7)
    for (int rows = kRopeRows;; rows /= 2) {
        p.q_chunks = (p.Hq + rows * at_once - 1) / (rows * at_once);
        p.k_chunks = (p.Hkv + rows * at_once - 1) / (rows * at_once);
        p.q_per = (p.Hq + p.q_chunks * at_once - 1) / (p.q_chunks * at_once);
        p.k_per = (p.Hkv + p.k_chunks * at_once - 1) / (p.k_chunks * at_once);
        p.chunks = p.q_chunks + (p.slots ? 2 : 1) * p.k_chunks;
        if (rows == 1 || groups * p.chunks >= 2ULL * ctas) break;
    }
    const unsigned long long grid = groups * p.chunks;
    if (grid > 0x7fffffffULL) return api_failf(KVATTN_ERR_UNSUPPORTED, "%s: too many rows for one launch", who);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (D) {
        case 64: e = launch_rope<64>(p, interleaved != 0, (unsigned)grid, st); break;
        case 128: e = launch_rope<128>(p, interleaved != 0, (unsigned)grid, st); break;
        default: e = launch_rope<256>(p, interleaved != 0, (unsigned)grid, st); break;
    }
    if (e != cudaSuccess) return api_cuda_fail(e, "rotation launch");
    return KVATTN_OK;
}

}  // namespace

}  // namespace kvattn

using namespace kvattn;

extern "C" {

int qk_norm_rope(const void *q, const void *k, const int32_t *positions, const float *cos_table,
                 const float *sin_table, const float *q_weight, const float *k_weight, void *q_out, void *k_out,
                 int N, int Hq, int Hkv, int D, int rope_dim, int max_pos, long long q_stride, long long k_stride,
                 long long q_out_stride, long long k_out_stride, float eps, int interleaved,
                 kvattn_stream_t stream) {
    const char *who = "qk_norm_rope";
    api_begin();
    if (!q || !k || !positions || !cos_table || !sin_table || !q_out || !k_out)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: null pointer", who);
    RopeParams p = {};
    p.q = static_cast<const uint2 *>(q);
    p.k = static_cast<const uint2 *>(k);
    p.pos = positions;
    p.cos = cos_table;
    p.sin = sin_table;
    p.qw = q_weight;
    p.kw = k_weight;
    p.q_out = static_cast<uint2 *>(q_out);
    p.k_out = static_cast<uint2 *>(k_out);
    p.N = N; p.Hq = Hq; p.Hkv = Hkv;
    p.max_pos = max_pos;
    p.eps = eps;
    return run_rope(p, D, rope_dim, q_stride, k_stride, k_stride, q_out_stride, k_out_stride, interleaved, stream,
                    who);
}

int kv_append_rope(const void *q, const void *k, const void *v, const int32_t *positions, const float *cos_table,
                   const float *sin_table, const float *q_weight, const float *k_weight, const int64_t *slots,
                   void *q_out, void *k_pool, void *v_pool, int N, int Hq, int Hkv, int D, int rope_dim,
                   int max_pos, long long q_stride, long long k_stride, long long v_stride,
                   long long q_out_stride, float eps, int interleaved, int num_blocks, int block_size,
                   kvattn_stream_t stream) {
    const char *who = "kv_append_rope";
    api_begin();
    if (!q || !k || !v || !positions || !cos_table || !sin_table || !slots || !q_out || !k_pool || !v_pool)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: null pointer", who);
    RopeParams p = {};
    int rc, lmax;
    static const int32_t no_table = 0;  // (the sizes' check wants a table)
    if ((rc = api_check_sizes(1, Hq, Hkv, D, 1))) return rc;
    if ((rc = api_check_paged(&no_table, Hkv, block_size, 1, num_blocks, who, &p.lg, &lmax))) return rc;
    p.q = static_cast<const uint2 *>(q);
    p.k = static_cast<const uint2 *>(k);
    p.v = static_cast<const uint2 *>(v);
    p.pos = positions;
    p.cos = cos_table;
    p.sin = sin_table;
    p.qw = q_weight;
    p.kw = k_weight;
    p.slots = reinterpret_cast<const long long *>(slots);
    p.q_out = static_cast<uint2 *>(q_out);
    p.k_pool = static_cast<uint2 *>(k_pool);
    p.v_pool = static_cast<uint2 *>(v_pool);
    p.num_slots = (long long)num_blocks << p.lg;
    p.N = N; p.Hq = Hq; p.Hkv = Hkv;
    p.max_pos = max_pos;
    p.eps = eps;
    return run_rope(p, D, rope_dim, q_stride, k_stride, v_stride, q_out_stride, k_stride, interleaved, stream, who);
}

}  // extern "C"
