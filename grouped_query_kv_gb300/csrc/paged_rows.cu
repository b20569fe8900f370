// paged_rows.cu -- blocks and slots for packed new tokens, and the write of
// their K/V rows into a paged bf16 pool ("Machine Learning Engineering and AI
// Systems at Scale", section "The key and value cache", on PagedAttention:
// blocks are handed out as sequences grow, a table maps positions to blocks).
//
// Block tables.  With c_b tokens cached and n_b new ones, request b has
// have_b = ceil(c_b / bs) blocks and needs up to upto_b = ceil((c_b + n_b) /
// bs); before_b = sum of (upto - have) over the requests before it places it
// in the free stack.  The bytes are few (8 per token), so what bounds a call
// is the chain of launch, length loads, two prefix sums over the requests and
// one dependent load per token.  Every block of the grid does the prefix sums
// itself (B lengths from L2, no workspace, nothing to wait for), then takes
// tiles of 4096 packed rows, a row's thread also writing the table entry of
// the block that starts at it; up to one tile the call is one block.  On the
// device 64 requests of one token take 4.3 us, 1024 requests of 1.0 M rows
// 8.6 to 9.8 (their 8.4 MB of slots are 1.3).
//
// Row write.  A copy of 16-byte vectors, four K and four V vectors of a
// thread in flight; both sides are contiguous per (token, head), so it runs
// at the copy's bandwidth: 65 536 rows of 8 x 128 (537 MB read and written)
// 80.4 us, 0.98 of the measured copy rate; 64 rows 2.5 us, a launch.
#include "../../include/kvattn.h"
#include "internal.h"
#include "ptx.cuh"

namespace kvattn {

namespace {

constexpr int kTblThreads = 1024;
constexpr int kTblRows = 4;                        // consecutive rows per thread
constexpr int kTblTile = kTblThreads * kTblRows;

struct TableParams {
    const int32_t *cached, *fresh;
    int32_t *table;
    const int32_t *free_ids, *free_count;
    int32_t *free_out, *cu;
    long long *slots;
    unsigned int *err;
    int B, max_blocks, lg, num_free, num_slots;
    int rows, count;  // write the slots and tables; write the count
};

// One request: its new rows and the blocks it lacks for them.
struct Request {
    int c, n, have, need;
    bool ok;  // lengths that are not negative and fit its table row
};

__device__ __forceinline__ Request get_request(const TableParams &p, int b) {
    Request r;
    r.c = p.cached[b];
    r.n = p.fresh[b];
    r.ok = r.c >= 0 && r.n >= 0 && (long long)r.c + r.n <= ((long long)p.max_blocks << p.lg);
    const int bs1 = (1 << p.lg) - 1;
    r.have = r.ok ? (r.c + bs1) >> p.lg : 0;
    r.need = r.ok ? ((r.c + r.n + bs1) >> p.lg) - r.have : 0;
    r.n = max(r.n, 0);
    return r;
}

__device__ __forceinline__ int cap32(long long x) { return (int)min(x, 0x7fffffffLL); }

__global__ void __launch_bounds__(kTblThreads) block_table_kernel(const TableParams p) {
    __shared__ longlong2 warps[32];
    __shared__ int s_rows[kTblThreads], s_blocks[kTblThreads];  // before each thread's requests
    __shared__ int s_taken;
    pdl_launch_dependents();
    pdl_wait_prior();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int count = p.free_count[0];
    bool bad = count < 0 || count > p.num_free;
    if (bad) count = 0;
    if (tid == 0) s_taken = 0;

    // prefix sums of rows and blocks: `per` consecutive requests per thread
    const int per = (p.B + kTblThreads - 1) / kTblThreads;
    const int b0 = tid * per, b1 = min(p.B, b0 + per);
    long long rows = 0, blocks = 0;
    for (int b = b0; b < b1; ++b) {
        const Request r = get_request(p, b);
        rows += r.n;
        blocks += r.need;
        bad |= !r.ok;
    }
    long long ir = rows, ib = blocks;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long vr = __shfl_up_sync(0xffffffffu, ir, o), vb = __shfl_up_sync(0xffffffffu, ib, o);
        if (lane >= o) {
            ir += vr;
            ib += vb;
        }
    }
    if (lane == 31) warps[warp] = make_longlong2(ir, ib);
    __syncthreads();
    if (warp == 0) {
        longlong2 w = warps[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long vr = __shfl_up_sync(0xffffffffu, w.x, o), vb = __shfl_up_sync(0xffffffffu, w.y, o);
            if (lane >= o) {
                w.x += vr;
                w.y += vb;
            }
        }
        warps[lane] = w;
    }
    __syncthreads();
    if (warp > 0) {
        ir += warps[warp - 1].x;
        ib += warps[warp - 1].y;
    }
    long long at_row = ir - rows, at_block = ib - blocks;
    s_rows[tid] = cap32(at_row);
    s_blocks[tid] = cap32(at_block);
    const long long all_rows = warps[31].x;

    if (blockIdx.x == 0) {
        // cu_seqlens, and the blocks taken: by the requests up to the last that
        // is served
        int taken = 0;
        for (int b = b0; b < b1; ++b) {
            const Request r = get_request(p, b);
            if (p.rows) {
                p.cu[b] = cap32(at_row);
                if (b == p.B - 1) p.cu[p.B] = cap32(at_row + r.n);
            }
            at_row += r.n;
            at_block += r.need;
            if (r.need > 0) {
                if (at_block <= count && at_row <= p.num_slots)
                    taken = (int)at_block;
                else
                    bad = true;
            }
        }
        if (taken) atomicMax(&s_taken, taken);
        if (all_rows > p.num_slots) bad = true;
        if (bad) atomicCAS(p.err, 0u, (unsigned int)DEV_ERR_BOUNDS);
    }
    __syncthreads();
    if (blockIdx.x == 0 && p.count && tid == 0) p.free_out[0] = count - s_taken;
    if (!p.rows) return;

    for (long long tile = (long long)blockIdx.x * kTblTile; tile < p.num_slots; tile += (long long)gridDim.x * kTblTile) {
        const int t0 = (int)tile + tid * kTblRows;
        if (t0 >= p.num_slots) continue;
        long long slot[kTblRows];
        int b = 0, first = 0, before = 0, blk = -1, blk_of = -1;
        Request r = {};
        bool served = false;
        // the request after `b` starts at first + r.n
        auto enter = [&](int nb) {
            b = nb;
            r = get_request(p, b);
            served = r.ok && (long long)first + r.n <= p.num_slots &&
                     (r.need == 0 || (long long)before + r.need <= count);
            blk_of = -1;
        };
        if (t0 < all_rows) {
            int lo = 0, hi = (p.B - 1) / per;  // the last thread whose requests start at or before t0
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_rows[mid] <= t0) lo = mid;
                else hi = mid - 1;
            }
            first = s_rows[lo];
            before = s_blocks[lo];
            enter(lo * per);
        }
#pragma unroll
        for (int i = 0; i < kTblRows; ++i) {
            const int t = t0 + i;
            slot[i] = -1;
            if (t < all_rows && t < p.num_slots) {
                // (ends: t is before the last request's end; first + n may pass 32 bits)
                while (t - first >= r.n) {
                    first += r.n;
                    before = cap32((long long)before + r.need);
                    enter(b + 1);
                }
                if (r.ok) {
                    const int pos = r.c + (t - first), e = pos >> p.lg;
                    int32_t *entry = p.table + (size_t)b * p.max_blocks + e;
                    if (e != blk_of) {
                        blk_of = e;
                        blk = !served ? -1 : e < r.have ? *entry : p.free_ids[count - 1 - (before + e - r.have)];
                    }
                    // the block's first row writes its entry (-1: none was left)
                    if (e >= r.have && (pos & ((1 << p.lg) - 1)) == 0) *entry = blk;
                    if (blk >= 0) slot[i] = ((long long)blk << p.lg) + (pos & ((1 << p.lg) - 1));
                }
            }
        }
        if ((reinterpret_cast<uintptr_t>(p.slots) & 15u) == 0 && t0 + kTblRows <= p.num_slots) {
#pragma unroll
            for (int i = 0; i < kTblRows; i += 2)
                *reinterpret_cast<longlong2 *>(p.slots + t0 + i) = make_longlong2(slot[i], slot[i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < kTblRows; ++i)
                if (t0 + i < p.num_slots) p.slots[t0 + i] = slot[i];
        }
    }
}

constexpr int kRowThreads = 256;
constexpr int kRowVecs = 4;  // vectors of K, and of V, per thread

struct RowParams {
    uint4 *k_pool, *v_pool;
    const uint4 *k_new, *v_new;
    const long long *slots;
    unsigned int *err;
    int N, Hkv, lg, vlg;          // vlg: log2 of 16-byte vectors per (row, head)
    long long k_stride, v_stride;  // vectors from row to row
    long long num_slots;           // num_blocks << lg
};

__global__ void __launch_bounds__(kRowThreads) append_slots_kernel(const RowParams p) {
    pdl_launch_dependents();
    pdl_wait_prior();
    const unsigned per_row = (unsigned)p.Hkv << p.vlg;  // vectors of a row
    // 256 x 4 consecutive vectors of the packed rows, from a row of its own in 64 bits
    const unsigned long long v0 = (unsigned long long)blockIdx.x * (kRowThreads * kRowVecs);
    const long long row0 = (long long)(v0 / per_row);
    const unsigned off0 = (unsigned)(v0 - (unsigned long long)row0 * per_row);
    uint4 k[kRowVecs], v[kRowVecs];
    long long dst[kRowVecs];
#pragma unroll
    for (int i = 0; i < kRowVecs; ++i) {
        const unsigned x = off0 + i * kRowThreads + threadIdx.x;
        const unsigned r = x / per_row, c = x - r * per_row;
        const long long row = row0 + r;
        dst[i] = -1;
        if (row < p.N) {
            const long long slot = p.slots[row];
            if (slot >= p.num_slots) {
                atomicCAS(p.err, 0u, (unsigned int)DEV_ERR_BOUNDS);
            } else if (slot >= 0) {
                const long long blk = slot >> p.lg;
                const int pos = (int)(slot & ((1 << p.lg) - 1));
                const unsigned h = c >> p.vlg, e = c & ((1u << p.vlg) - 1);
                dst[i] = ((((blk * p.Hkv + h) << p.lg) + pos) << p.vlg) + e;
                k[i] = __ldcs(p.k_new + row * p.k_stride + c);
                v[i] = __ldcs(p.v_new + row * p.v_stride + c);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRowVecs; ++i)
        if (dst[i] >= 0) {
            p.k_pool[dst[i]] = k[i];
            p.v_pool[dst[i]] = v[i];
        }
}

template <class Kernel, class Params>
cudaError_t launch_pdl(Kernel kernel, unsigned grid, unsigned block, cudaStream_t stream, const Params &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = 0;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

}  // namespace kvattn

using namespace kvattn;

extern "C" {

int kv_block_tables(const int32_t *cached_lens, const int32_t *new_lens, int32_t *block_table,
                    const int32_t *free_blocks, const int32_t *free_count, int32_t *free_count_out,
                    int32_t *cu_seqlens, int64_t *slots, int B, int max_blocks, int block_size,
                    int num_free, int num_slots, kvattn_stream_t stream) {
    const char *who = "kv_block_tables";
    api_begin();
    if (!cached_lens || !new_lens || !block_table || !free_blocks || !free_count || !free_count_out ||
        !cu_seqlens || !slots)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: null pointer", who);
    if (((reinterpret_cast<uintptr_t>(cached_lens) | reinterpret_cast<uintptr_t>(new_lens) |
          reinterpret_cast<uintptr_t>(free_blocks) | reinterpret_cast<uintptr_t>(free_count) |
          reinterpret_cast<uintptr_t>(free_count_out) | reinterpret_cast<uintptr_t>(cu_seqlens)) & 3u) ||
        (reinterpret_cast<uintptr_t>(slots) & 7u))
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: int32 arrays must be 4-byte, slots 8-byte aligned", who);
    if (B <= 0 || num_free <= 0 || num_slots <= 0)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: B, num_free and num_slots must be positive (%d, %d, %d)",
                         who, B, num_free, num_slots);
    if (B > 65535 || num_slots > (1 << 28))
        return api_failf(KVATTN_ERR_UNSUPPORTED, "%s: sizes beyond limits (B <= 65535, num_slots <= 2^28)", who);
    int lg, lmax, rc;
    if ((rc = api_check_paged(block_table, 1, block_size, max_blocks, 1, who, &lg, &lmax))) return rc;
    TableParams p = {};
    int ctas;
    unsigned int wait_limit;
    if ((rc = api_device(&ctas, &p.err, &wait_limit))) return rc;
    p.cached = cached_lens;
    p.fresh = new_lens;
    p.table = block_table;
    p.free_ids = free_blocks;
    p.free_count = free_count;
    p.free_out = free_count_out;
    p.cu = cu_seqlens;
    p.slots = reinterpret_cast<long long *>(slots);
    p.B = B;
    p.max_blocks = max_blocks;
    p.lg = lg;
    p.num_free = num_free;
    p.num_slots = num_slots;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // one block per tile of rows, two to an SM; the count, where it goes back
    // into the word that every block reads, is written by a launch of its own
    const int tiles = (num_slots + kTblTile - 1) / kTblTile;
    const int grid = tiles < 2 * ctas ? tiles : 2 * ctas;
    const bool apart = grid > 1 && free_count == free_count_out;
    p.rows = 1;
    p.count = apart ? 0 : 1;
    cudaError_t e = launch_pdl(block_table_kernel, grid, kTblThreads, st, p);
    if (e == cudaSuccess && apart) {
        p.rows = 0;
        p.count = 1;
        e = launch_pdl(block_table_kernel, 1, kTblThreads, st, p);
    }
    if (e != cudaSuccess) return api_cuda_fail(e, "block table launch");
    return KVATTN_OK;
}

int kv_append_slots(void *k_pool, void *v_pool, const void *k_new, const void *v_new,
                    const int64_t *slots, int N, int Hkv, int D, long long k_stride,
                    long long v_stride, int num_blocks, int block_size, kvattn_stream_t stream) {
    const char *who = "kv_append_slots";
    api_begin();
    if (!k_pool || !v_pool || !k_new || !v_new || !slots)
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: null pointer", who);
    if (((reinterpret_cast<uintptr_t>(k_pool) | reinterpret_cast<uintptr_t>(v_pool) |
          reinterpret_cast<uintptr_t>(k_new) | reinterpret_cast<uintptr_t>(v_new)) & 15u) ||
        (reinterpret_cast<uintptr_t>(slots) & 7u))
        return api_failf(KVATTN_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned (slots 8)", who);
    int rc, lg, lmax;
    static const int32_t no_table = 0;  // (the sizes' check wants a table)
    if ((rc = api_check_sizes(1, Hkv, Hkv, D, 1))) return rc;
    if ((rc = api_check_paged(&no_table, Hkv, block_size, 1, num_blocks, who, &lg, &lmax))) return rc;
    if (N < 1) return api_failf(KVATTN_ERR_INVALID_ARG, "%s: N must be positive (got %d)", who, N);
    if (N > (1 << 28)) return api_failf(KVATTN_ERR_UNSUPPORTED, "%s: N = %d rows beyond 2^28", who, N);
    if ((rc = api_check_row_stride(k_stride, Hkv, D, who)) ||
        (rc = api_check_row_stride(v_stride, Hkv, D, who)))
        return rc;
    RowParams p = {};
    int ctas;
    unsigned int wait_limit;
    if ((rc = api_device(&ctas, &p.err, &wait_limit))) return rc;
    p.k_pool = static_cast<uint4 *>(k_pool);
    p.v_pool = static_cast<uint4 *>(v_pool);
    p.k_new = static_cast<const uint4 *>(k_new);
    p.v_new = static_cast<const uint4 *>(v_new);
    p.slots = reinterpret_cast<const long long *>(slots);
    p.N = N;
    p.Hkv = Hkv;
    p.lg = lg;
    p.vlg = D == 64 ? 3 : D == 128 ? 4 : 5;
    p.k_stride = k_stride / 8;
    p.v_stride = v_stride / 8;
    p.num_slots = (long long)num_blocks << lg;
    const unsigned long long vecs = (unsigned long long)N * ((unsigned)Hkv << p.vlg);
    const unsigned long long grid = (vecs + kRowThreads * kRowVecs - 1) / (kRowThreads * kRowVecs);
    if (grid > 0x7fffffffULL) return api_failf(KVATTN_ERR_UNSUPPORTED, "%s: too many rows for one launch", who);
    cudaError_t e = launch_pdl(append_slots_kernel, (unsigned)grid, kRowThreads,
                               reinterpret_cast<cudaStream_t>(stream), p);
    if (e != cudaSuccess) return api_cuda_fail(e, "slot append launch");
    return KVATTN_OK;
}

}  // extern "C"
