// paged_rows.cu -- blocks and slots for packed new tokens, and the write of
// their K/V rows into a paged bf16 pool ("Machine Learning Engineering and AI
// Systems at Scale", section "The key and value cache", on PagedAttention:
// blocks are handed out as sequences grow, a table maps positions to blocks).
//
// Block tables.  With c_b tokens cached and n_b new ones, request b has
// have_b = ceil(c_b / bs) blocks and needs up to upto_b = ceil((c_b + n_b) /
// bs); before_b = sum of (upto - have) over the requests before it places it
// in the free stack.  Two prefix sums over B lengths and one write per new
// block and per token: the bytes are few (8 per token), so what bounds a
// call is the chain of launch, length loads, scans and dependent loads.  One
// block of 1024 threads does the sums, the tables and (up to
// kOneBlockSlots slots) the slot map; larger maps get a second launch of
// many blocks, which starts its prologue under the first.
//
// Row write.  A copy of 16-byte vectors, four K and four V vectors of a
// thread in flight; both sides are contiguous per (token, head), so it runs
// at the copy's bandwidth.
#include "../../include/kvattn.h"
#include "internal.h"
#include "ptx.cuh"

namespace kvattn {

namespace {

constexpr int kTblThreads = 1024;
constexpr int kOneBlockSlots = 4096;  // slots that the table kernel writes itself
constexpr int kSlotThreads = 256;
constexpr int kSlotsPerThread = 4;

struct TableParams {
    const int32_t *cached, *fresh;
    int32_t *table;
    const int32_t *free_ids, *free_count;
    int32_t *free_out, *cu;
    long long *slots;
    unsigned int *err;
    int B, max_blocks, lg, num_free, num_slots;
};

// Lengths of one request; false if they are negative or do not fit its table row.
__device__ __forceinline__ bool request_ok(int c, int n, int max_blocks, int lg) {
    return c >= 0 && n >= 0 && (long long)c + n <= ((long long)max_blocks << lg);
}

// Slot of packed row t of request b (-1: none).  A request whose first
// missing block is -1 got no blocks.
__device__ __forceinline__ long long slot_of(const TableParams &p, int b, int c, int n, long long i) {
    if (!request_ok(c, n, p.max_blocks, p.lg)) return -1;
    const int bs1 = (1 << p.lg) - 1;
    const int have = (c + bs1) >> p.lg, upto = (c + n + bs1) >> p.lg;
    const int32_t *row = p.table + (size_t)b * p.max_blocks;
    if (upto > have && row[have] < 0) return -1;
    const int pos = c + (int)i;
    const int blk = row[pos >> p.lg];
    return blk < 0 ? -1 : ((long long)blk << p.lg) + (pos & bs1);
}

// Exclusive prefix sums of two values over the block; *ta, *tb the totals.
__device__ __forceinline__ void block_scan2(long long a, long long b, long long *ea, long long *eb,
                                            long long *ta, long long *tb, longlong2 *warps) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long va = __shfl_up_sync(0xffffffffu, ia, o), vb = __shfl_up_sync(0xffffffffu, ib, o);
        if (lane >= o) {
            ia += va;
            ib += vb;
        }
    }
    if (lane == 31) warps[warp] = make_longlong2(ia, ib);
    __syncthreads();
    if (warp == 0) {
        longlong2 w = warps[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long va = __shfl_up_sync(0xffffffffu, w.x, o), vb = __shfl_up_sync(0xffffffffu, w.y, o);
            if (lane >= o) {
                w.x += va;
                w.y += vb;
            }
        }
        warps[lane] = w;
    }
    __syncthreads();
    const longlong2 before = warp ? warps[warp - 1] : make_longlong2(0, 0);
    *ea = before.x + ia - a;
    *eb = before.y + ib - b;
    *ta = warps[31].x;
    *tb = warps[31].y;
    __syncthreads();
}

__global__ void __launch_bounds__(kTblThreads) block_table_kernel(const TableParams p) {
    __shared__ longlong2 warps[32];
    __shared__ int s_first[kTblThreads + 1];  // first new block of each request of a chunk
    __shared__ int s_have[kTblThreads];
    __shared__ int s_cut;                     // requests from here on are not served
    pdl_launch_dependents();
    pdl_wait_prior();
    const int tid = threadIdx.x;
    int count = p.free_count[0];
    bool bad = false;
    if (count < 0 || count > p.num_free) {
        count = 0;
        bad = true;
    }
    long long rows = 0, taken = 0;  // of the requests before this chunk
    long long wanted = 0;
    bool out = false;  // the free list has run out
    for (int b0 = 0; b0 < p.B; b0 += kTblThreads) {
        const int b = b0 + tid;
        int c = 0, n = 0, have = 0, need = 0;
        if (b < p.B) {
            c = p.cached[b];
            n = p.fresh[b];
            if (request_ok(c, n, p.max_blocks, p.lg)) {
                const int bs1 = (1 << p.lg) - 1;
                have = (c + bs1) >> p.lg;
                need = ((c + n + bs1) >> p.lg) - have;
            } else {
                bad = true;
                n = max(n, 0);
            }
        }
        long long er, eb, tr, tb;
        block_scan2(n, need, &er, &eb, &tr, &tb, warps);
        if (b < p.B) {
            const long long at = rows + er;
            p.cu[b] = (int)min(at, 0x7fffffffLL);
            if (b == p.B - 1) p.cu[p.B] = (int)min(at + n, 0x7fffffffLL);
        }
        rows += tr;
        // served: every request whose blocks end within the list (a prefix of those that need any)
        const bool fits = !out && wanted + eb + need <= count;
        const int chunk = min(kTblThreads, p.B - b0);
        if (tid == 0) s_cut = chunk;
        s_first[tid] = (int)min(eb, 0x7fffffffLL);
        s_have[tid] = have;
        if (tid == 0) s_first[chunk] = (int)min(tb, 0x7fffffffLL);
        __syncthreads();
        if (b < p.B && need > 0 && !fits) atomicMin(&s_cut, tid);
        __syncthreads();
        const int cut = s_cut;
        const int blocks = s_first[chunk], good = s_first[cut];
        // one new block per thread: its request by bisection over s_first
        for (int e = tid; e < blocks; e += kTblThreads) {
            int lo = 0, hi = chunk - 1;  // the last request whose first block is <= e
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_first[mid] <= e) lo = mid;
                else hi = mid - 1;
            }
            const int id = e < good ? p.free_ids[count - 1 - (int)(taken + e)] : -1;
            p.table[(size_t)(b0 + lo) * p.max_blocks + s_have[lo] + (e - s_first[lo])] = id;
        }
        if (cut < chunk) {
            out = true;
            bad = true;
        }
        taken += good;
        wanted += tb;
        __syncthreads();
    }
    if (rows > p.num_slots) bad = true;
    if (tid == 0) p.free_out[0] = count - (int)taken;
    if (bad) atomicCAS(p.err, 0u, (unsigned int)DEV_ERR_BOUNDS);
    if (p.num_slots > kOneBlockSlots) return;
    // (this block wrote the table and cu_seqlens: visible after the barrier above)
    for (int t = tid; t < p.num_slots; t += kTblThreads) {
        long long s = -1;
        if (t < rows) {
            int lo = 0, hi = p.B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (p.cu[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            s = slot_of(p, lo, p.cached[lo], p.fresh[lo], t - p.cu[lo]);
        }
        p.slots[t] = s;
    }
}

// Slots of many rows: kSlotsPerThread consecutive ones per thread.
__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const TableParams p) {
    pdl_launch_dependents();
    pdl_wait_prior();
    const int t0 = (blockIdx.x * kSlotThreads + threadIdx.x) * kSlotsPerThread;
    if (t0 >= p.num_slots) return;
    const int rows = p.cu[p.B];
    int b = 0, next = 0, c = 0, n = 0, first = 0;
    if (t0 < rows) {
        int lo = 0, hi = p.B - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (p.cu[mid] <= t0) lo = mid;
            else hi = mid - 1;
        }
        b = lo;
        first = p.cu[b];
        next = p.cu[b + 1];
        c = p.cached[b];
        n = p.fresh[b];
    }
    long long s[kSlotsPerThread];
#pragma unroll
    for (int i = 0; i < kSlotsPerThread; ++i) {
        const int t = t0 + i;
        s[i] = -1;
        if (t < rows) {
            while (t >= next) {  // (ends: t < cu[B])
                ++b;
                first = next;
                next = p.cu[b + 1];
                c = p.cached[b];
                n = p.fresh[b];
            }
            s[i] = slot_of(p, b, c, n, t - first);
        }
    }
#pragma unroll
    for (int i = 0; i < kSlotsPerThread; ++i)
        if (t0 + i < p.num_slots) p.slots[t0 + i] = s[i];
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
    cudaError_t e = launch_pdl(block_table_kernel, 1, kTblThreads, st, p);
    if (e != cudaSuccess) return api_cuda_fail(e, "block table launch");
    if (num_slots > kOneBlockSlots) {
        const unsigned per = kSlotThreads * kSlotsPerThread;
        e = launch_pdl(slot_map_kernel, (num_slots + per - 1) / per, kSlotThreads, st, p);
        if (e != cudaSuccess) return api_cuda_fail(e, "slot map launch");
    }
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
