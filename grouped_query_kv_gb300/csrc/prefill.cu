// prefill.cu -- gqa_prefill_attn: the prompt attention of prefill.cuh over packed
// K/V rows.
#include <cfloat>
#include <cmath>

#include "../../include/kvattn.h"
#include "prefill.cuh"

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
        case 64: e = launch_pf<64, false, false>(tmq, tmk, tmv, p, ctas, reinterpret_cast<cudaStream_t>(stream)); break;
        case 128: e = launch_pf<128, false, false>(tmq, tmk, tmv, p, ctas, reinterpret_cast<cudaStream_t>(stream)); break;
        default: e = launch_pf<256, false, false>(tmq, tmk, tmv, p, ctas, reinterpret_cast<cudaStream_t>(stream)); break;
    }
    if (e != cudaSuccess) return api_cuda_fail(e, "prefill kernel launch");
    return KVATTN_OK;
}
