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
// Layout.  A head's row is D / 8 lanes of 16 bytes; a warp takes 4 x 32 / (D /
// 8) heads of one token, four loads a lane in flight, so that a lane's cosines,
// sines and weights (the same for all heads) are loaded once for four rows.
// Partners of a rotation D / 16 lanes apart meet by a shuffle.  The heads are
// the token's queries, then its keys, then its values, which are copied.
//
// What bounds it: HBM, every value read once and written once.
#include <cmath>
#include <cuda_bf16.h>

#include "../../include/kvattn.h"
#include "internal.h"
#include "ptx.cuh"

namespace kvattn {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = 4;  // head rows per lane

struct RopeParams {
    const uint4 *q, *k, *v;
    const int32_t *pos;
    const float *cos, *sin;
    const float *qw, *kw;      // [D], or null: no norm
    const long long *slots;    // null: no pool
    uint4 *q_out, *k_out;      // k_out null: the pool takes the keys
    uint4 *k_pool, *v_pool;
    unsigned int *err;
    long long q_stride, k_stride, v_stride, qo_stride, ko_stride;  // vectors from row to row
    long long num_slots;
    int N, Hq, Hkv, heads;     // heads: of q, k and (with a pool) v together
    int chunks;                // warps per token
    int half;                  // rope_dim / 2
    int max_pos;
    int lg;                    // log2(block_size)
    float eps;
};

__device__ __forceinline__ void unpack8(const uint4 &u, float *x) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void load4(const float *src, float *x) {
    const float4 f = __ldg(reinterpret_cast<const float4 *>(src));
    x[0] = f.x;
    x[1] = f.y;
    x[2] = f.z;
    x[3] = f.w;
}

// D head dims; NEXT: neighbours rotate together, else values rope_dim / 2 apart.
template <int D, bool NEXT>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p) {
    constexpr int LP = D / 8;        // lanes of a head's row
    constexpr int VPW = 32 / LP;     // head rows of a warp at once
    constexpr int NC = NEXT ? 4 : 8;  // cosines of a lane
    pdl_launch_dependents();
    pdl_wait_prior();
    const int lane = threadIdx.x & 31, l = lane % LP;
    const unsigned long long w = (unsigned long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
    const long long row = (long long)(w / (unsigned)p.chunks);
    if (row >= p.N) return;
    const int h0 = (int)(w - (unsigned long long)row * (unsigned)p.chunks) * (VPW * kRopeRows) + lane / LP;

    const int pos = p.pos[row];
    uint4 raw[kRopeRows];
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) {
        const int h = h0 + u * VPW;
        raw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (h < p.Hq)
            raw[u] = __ldcs(p.q + row * p.q_stride + (long long)h * LP + l);
        else if (h < p.Hq + p.Hkv)
            raw[u] = __ldcs(p.k + row * p.k_stride + (long long)(h - p.Hq) * LP + l);
        else if (h < p.heads)
            raw[u] = __ldcs(p.v + row * p.v_stride + (long long)(h - p.Hq - p.Hkv) * LP + l);
    }
    const bool there = pos >= 0 && pos < p.max_pos;
    if (pos >= p.max_pos && h0 == 0 && l == 0) atomicCAS(p.err, 0u, (unsigned int)DEV_ERR_BOUNDS);
    // where the row's keys and values go in the pool
    long long to = -1;  // vectors to row 0's head
    if (p.slots && there) {
        const long long slot = p.slots[row];
        if (slot >= p.num_slots) {
            if (h0 == 0 && l == 0) atomicCAS(p.err, 0u, (unsigned int)DEV_ERR_BOUNDS);
        } else if (slot >= 0) {
            to = ((((slot >> p.lg) * p.Hkv) << p.lg) + (slot & ((1 << p.lg) - 1))) * LP;
        }
    }

    // the lane's rotation: none, of the first of its pairs, or of the second
    const int d0 = 8 * l;
    const bool turns = d0 < 2 * p.half;
    const bool second = !NEXT && d0 >= p.half;
    float c[NC], s[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) c[i] = 1.f, s[i] = 0.f;
    if (there && turns) {
        const int j0 = NEXT ? d0 / 2 : second ? d0 - p.half : d0;
        const long long at = (long long)pos * p.half + j0;
#pragma unroll
        for (int i = 0; i < NC; i += 4) {
            load4(p.cos + at + i, c + i);
            load4(p.sin + at + i, s + i);
        }
    }
    if (!NEXT && !second) {
#pragma unroll
        for (int i = 0; i < NC; ++i) s[i] = -s[i];  // a c - b s; b c + a s
    }
    // the lane that holds the partners
    const int mate = !turns ? lane : second ? lane - p.half / 8 : lane + p.half / 8;

    const float *w_of = nullptr;
    float wt[8];
#pragma unroll
    for (int u = 0; u < kRopeRows; ++u) {
        const int h = h0 + u * VPW;
        const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;  // q, k, v (or none)
        float x[8];
        unpack8(raw[u], x);
        const float *wp = kind == 0 ? p.qw : kind == 1 ? p.kw : nullptr;
        if (p.qw || p.kw) {  // (the same in every lane)
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = LP / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (wp) {
                const float r = rsqrtf(ss * (1.f / D) + p.eps);
                if (wp != w_of) {
                    w_of = wp;
                    load4(wp + d0, wt);
                    load4(wp + d0 + 4, wt + 4);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= r * wt[i];
            }
        }
        float y[8];
        if constexpr (NEXT) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[2 * i] = x[2 * i] * c[i] - x[2 * i + 1] * s[i];
                y[2 * i + 1] = x[2 * i] * s[i] + x[2 * i + 1] * c[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float b = __shfl_sync(0xffffffffu, x[i], mate);
                y[i] = x[i] * c[i] + b * s[i];
            }
        }
        if (!turns) {  // (0 times an infinity is none of its business)
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[i];
        }
        uint4 out = pack8(y);
        if (!there) out = make_uint4(0u, 0u, 0u, 0u);
        if (kind == 0) {
            p.q_out[row * p.qo_stride + (long long)h * LP + l] = out;
        } else if (kind == 1) {
            const int kh = h - p.Hq;
            if (p.k_out) p.k_out[row * p.ko_stride + (long long)kh * LP + l] = out;
            if (to >= 0) p.k_pool[to + (((long long)kh << p.lg) * LP) + l] = out;
        } else if (h < p.heads && to >= 0) {
            const int vh = h - p.Hq - p.Hkv;
            p.v_pool[to + (((long long)vh << p.lg) * LP) + l] = raw[u];
        }
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
    p.q_stride = q_stride / 8;
    p.k_stride = k_stride / 8;
    p.v_stride = v_stride / 8;
    p.qo_stride = qo_stride / 8;
    p.ko_stride = ko_stride / 8;
    p.half = rope_dim / 2;
    p.heads = p.Hq + (p.slots ? 2 : 1) * p.Hkv;
    const int per_warp = kRopeRows * 32 / (D / 8);
    p.chunks = (p.heads + per_warp - 1) / per_warp;
    const unsigned long long warps = (unsigned long long)p.N * p.chunks;
    const unsigned long long grid = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
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
    p.q = static_cast<const uint4 *>(q);
    p.k = static_cast<const uint4 *>(k);
    p.pos = positions;
    p.cos = cos_table;
    p.sin = sin_table;
    p.qw = q_weight;
    p.kw = k_weight;
    p.q_out = static_cast<uint4 *>(q_out);
    p.k_out = static_cast<uint4 *>(k_out);
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
    p.q = static_cast<const uint4 *>(q);
    p.k = static_cast<const uint4 *>(k);
    p.v = static_cast<const uint4 *>(v);
    p.pos = positions;
    p.cos = cos_table;
    p.sin = sin_table;
    p.qw = q_weight;
    p.kw = k_weight;
    p.slots = reinterpret_cast<const long long *>(slots);
    p.q_out = static_cast<uint4 *>(q_out);
    p.k_pool = static_cast<uint4 *>(k_pool);
    p.v_pool = static_cast<uint4 *>(v_pool);
    p.num_slots = (long long)num_blocks << p.lg;
    p.N = N; p.Hq = Hq; p.Hkv = Hkv;
    p.max_pos = max_pos;
    p.eps = eps;
    return run_rope(p, D, rope_dim, q_stride, k_stride, v_stride, q_out_stride, k_stride, interleaved, stream, who);
}

}  // extern "C"
