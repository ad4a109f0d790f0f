// Verification of drafted tokens and the draw of the next one (dl_verify_draft).
#include "dl_host.h"
#include "dl_device.cuh"

namespace dl {

struct VerifyParams {
    const int* draft_tokens;
    const void *draft_probs, *target_probs;
    const float *u_accept, *u_next;
    const int* draft_lens;
    int *tokens, *count;
    int drafts, vocab;
};

constexpr int kVerifyThreads = 1024;
constexpr int kWeightBits = 44;

__device__ __forceinline__ float prob(const float* p, size_t i) { return p[i]; }
__device__ __forceinline__ float prob(const uint16_t* p, size_t i) { return bf16_bits_to_f32(p[i]); }

// A probability as a whole multiple of 2^-44 (NaN: 0).  The product is exact.
__device__ __forceinline__ long long whole(float x) {
    x = fminf(fmaxf(x, 0.f), 1.f);
    return __float2ll_rn(x * (float)(1ll << kWeightBits));
}

// One CTA for each sequence.
template <class T>
__global__ void __launch_bounds__(kVerifyThreads) verify_draft_kernel(const __grid_constant__ VerifyParams p) {
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = p.vocab;
    const T* target = static_cast<const T*>(p.target_probs) + (size_t)b * (p.drafts + 1) * V;
    const T* guess = p.draft_probs ? static_cast<const T*>(p.draft_probs) + (size_t)b * p.drafts * V : nullptr;
    __shared__ int s_count, s_next;
    __shared__ long long s_warp[kVerifyThreads / 32], s_run;
    const int n = p.draft_lens ? min(max(p.draft_lens[b], 0), p.drafts) : p.drafts;
    if (tid == 0) {
        int c = 0;
        for (; c < n; ++c) {
            const int x = p.draft_tokens[(size_t)b * p.drafts + c];
            if (x < 0 || x >= V) break;
            const float g = guess ? prob(guess, (size_t)c * V + x) : 1.f;
            if (!((double)p.u_accept[(size_t)b * p.drafts + c] * (double)g < (double)prob(target, (size_t)c * V + x))) break;
        }
        s_count = c;
        s_next = -1;
    }
    __syncthreads();
    const int c = s_count;
    const T* pr = target + (size_t)c * V;
    const T* gr = guess && c < n ? guess + (size_t)c * V : nullptr;
    const int x = c < n ? p.draft_tokens[(size_t)b * p.drafts + c] : -1;
    bool plain = false;
    auto weight = [&](int v) {
        long long w = whole(prob(pr, v));
        if (plain || c == n) return w;
        w -= gr ? whole(prob(gr, v)) : (v == x ? 1ll << kWeightBits : 0ll);
        return w > 0 ? w : 0ll;
    };
    auto block_sum = [&](long long w) {
        for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(~0u, w, o);
        if (lane == 0) s_warp[warp] = w;
        __syncthreads();
        long long sum = 0;
        for (int i = 0; i < kVerifyThreads / 32; ++i) sum += s_warp[i];
        __syncthreads();
        return sum;
    };
    long long total = 0;
    for (int pass = 0; pass < 2 && total == 0; ++pass) {
        plain = pass == 1;
        long long w = 0;
        for (int v = tid; v < V; v += kVerifyThreads) w += weight(v);
        total = block_sum(w);
    }
    if (total > 0) {
        const float u = fminf(fmaxf(p.u_next[b], 0.f), 1.f);
        long long r = (long long)floorf(u * 16777216.f);
        if (r > (1ll << 24) - 1) r = (1ll << 24) - 1;
        const long long mark = (total >> 24) * r + (((total & ((1ll << 24) - 1)) * r) >> 24);
        if (tid == 0) s_run = 0;
        __syncthreads();
        for (int v0 = 0; v0 < V; v0 += kVerifyThreads) {
            const int v = v0 + tid;
            const long long w = v < V ? weight(v) : 0;
            long long inc = w;
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(~0u, inc, o);
                if (lane >= o) inc += y;
            }
            if (lane == 31) s_warp[warp] = inc;
            __syncthreads();
            long long before = s_run;
            for (int i = 0; i < warp; ++i) before += s_warp[i];
            if (w > 0 && before + inc > mark && before + inc - w <= mark) s_next = v;
            __syncthreads();
            if (tid == kVerifyThreads - 1) s_run = before + inc;
            __syncthreads();
            if (s_next >= 0) break;
        }
    }
    for (int i = tid; i <= p.drafts; i += kVerifyThreads)
        p.tokens[(size_t)b * (p.drafts + 1) + i] =
            i < c ? p.draft_tokens[(size_t)b * p.drafts + i] : i == c ? s_next : -1;
    if (tid == 0) p.count[b] = c;
}

}  // namespace dl

extern "C" dl_status dl_verify_draft(const int* draft_tokens, const void* draft_probs,
                                     const void* target_probs, int probs_dtype, const float* u_accept,
                                     const float* u_next, const int* draft_lens, int* tokens,
                                     int* count, int batch, int drafts, int vocab, void* stream) {
    using namespace dl;
    if (probs_dtype != DL_PROBS_F32 && probs_dtype != DL_PROBS_BF16)
        return host_fail(DL_ERR_INVALID_ARG, "unknown probs_dtype %d", probs_dtype);
    if (batch < 0) return host_fail(DL_ERR_INVALID_ARG, "batch=%d must be >= 0", batch);
    if (drafts < 0 || drafts > 63)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "drafts=%d is outside [0, 63]", drafts);
    if (vocab < 1 || vocab > (1 << 18))
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "vocab=%d is outside [1, 262144]", vocab);
    if (batch == 0) return host_ok();
    if (!target_probs || !u_next || !tokens || !count || (drafts && (!draft_tokens || !u_accept)))
        return host_fail(DL_ERR_INVALID_ARG, "a required pointer is NULL");
    const uintptr_t el = probs_dtype == DL_PROBS_F32 ? 3 : 1;
    if (((uintptr_t)target_probs | (uintptr_t)draft_probs) & el)
        return host_fail(DL_ERR_MISALIGNED, "probabilities must be aligned to their type");
    if (((uintptr_t)draft_tokens | (uintptr_t)u_accept | (uintptr_t)u_next | (uintptr_t)draft_lens |
         (uintptr_t)tokens | (uintptr_t)count) & 3)
        return host_fail(DL_ERR_MISALIGNED, "an int32 or fp32 array is not 4-byte aligned");
    const VerifyParams p = {draft_tokens, drafts ? draft_probs : nullptr, target_probs, u_accept, u_next,
                            draft_lens, tokens, count, drafts, vocab};
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (probs_dtype == DL_PROBS_F32)
        verify_draft_kernel<float><<<batch, kVerifyThreads, 0, st>>>(p);
    else
        verify_draft_kernel<uint16_t><<<batch, kVerifyThreads, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "verify_draft launch: %s", cudaGetErrorString(e));
    return host_ok();
}
