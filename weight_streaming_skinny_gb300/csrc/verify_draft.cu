// Verification of drafted tokens and the draw of the next one (dl_verify_draft).
#include <cooperative_groups.h>

#include <atomic>
#include <type_traits>

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

// A cluster of CTAs takes one sequence, each warp a contiguous run of its vocabulary.
// What bounds it: for many sequences the one read of p (and g) and the arithmetic on
// it, for few the chain of dependent loads (draft token, its probabilities, the
// row) and the cluster's two barriers: 6.6 us for one sequence of 152064 entries, 15 us
// for 48 (45 MB: 3.0 TB/s).  The first pass keeps the sums by CTA and warp, so that the drawn token is
// found by reading one warp's run again, not the row.
constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 16;

// Four consecutive probabilities from entry i on, entries at or past `end` as
// zeros; `wide`: the row's groups of four are aligned to their size; ALL: they are, and
// end at or before `end`.
template <bool ALL>
__device__ __forceinline__ void four(const float* row, int i, int end, bool wide, float (&f)[4]) {
    if (ALL || (wide && i + 4 <= end)) {
        const uint4 v = ldg128(row + i);
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = i + k < end ? row[i + k] : 0.f;
    }
}
template <bool ALL>
__device__ __forceinline__ void four(const uint16_t* row, int i, int end, bool wide, float (&f)[4]) {
    if (ALL || (wide && i + 4 <= end)) {
        const uint2 v = ldg64(row + i);
        f[0] = __uint_as_float(v.x << 16); f[1] = __uint_as_float(v.x & 0xffff0000u);
        f[2] = __uint_as_float(v.y << 16); f[3] = __uint_as_float(v.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = i + k < end ? bf16_bits_to_f32(row[i + k]) : 0.f;
    }
}
__device__ __forceinline__ float prob(const float* p, size_t i) { return p[i]; }
__device__ __forceinline__ float prob(const uint16_t* p, size_t i) { return bf16_bits_to_f32(p[i]); }

// Two probabilities x of [0, 1], as the whole numbers nearest to x 2^44: hi 2^22 + lo each, both
// offset by kOffset.  Adding 1.5 * 2^23 leaves a rounded integer in an fp32's low
// bits; hi's rounding error is exact in fp32, so lo rounds the whole value once, to
// even at ties (hi 2^22 is even).
constexpr float kMagic = 12582912.f, kStep = 4194304.f;       // 1.5 * 2^23, 2^22
constexpr int kOffset = 0x4B400000;                           // the bits of kMagic
__device__ __forceinline__ void whole2(float x0, float x1, int& hi0, int& hi1, int& lo0, int& lo1) {
    const F2 x = f2(x0, x1), step = f2(kStep, kStep), magic = f2(kMagic, kMagic);
    const F2 a = fma2(x, step, magic);
    const F2 rest = fma2(x, step, fma2(a, f2(-1.f, -1.f), magic));
    float h0, h1, l0, l1;
    unpack(a, h0, h1);
    unpack(fma2(rest, step, magic), l0, l1);
    hi0 = __float_as_int(h0); hi1 = __float_as_int(h1);
    lo0 = __float_as_int(l0); lo1 = __float_as_int(l1);
}

// The weights max(P - G, 0) of four entries, as hi 2^22 + lo each: P is never below G where
// p is not, so max(p, g) in p's place leaves 0.  Probabilities are taken inside [0, 1] (NaN: 0).
template <bool G>
__device__ __forceinline__ void weights(const float (&f)[4], const float (&g)[4], int (&hi)[4], int (&lo)[4]) {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
        float x[2] = {__saturatef(f[k]), __saturatef(f[k + 1])};
        int gh[2] = {kOffset, kOffset}, gl[2] = {kOffset, kOffset};
        if (G) {
            const float z[2] = {__saturatef(g[k]), __saturatef(g[k + 1])};
            whole2(z[0], z[1], gh[0], gh[1], gl[0], gl[1]);
            x[0] = fmaxf(x[0], z[0]);
            x[1] = fmaxf(x[1], z[1]);
        }
        whole2(x[0], x[1], hi[k], hi[k + 1], lo[k], lo[k + 1]);
        hi[k] -= gh[0]; hi[k + 1] -= gh[1];
        lo[k] -= gl[0]; lo[k + 1] -= gl[1];
    }
}
__device__ __forceinline__ long long joined(int hi, int lo) { return (long long)hi * (1 << 22) + lo; }

__device__ __forceinline__ long long warp_sum(long long w) {
    for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(~0u, w, o);
    return w;
}

__device__ __forceinline__ long long warp_scan(long long w, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(~0u, w, o);
        if (lane >= o) w += y;
    }
    return w;
}

// Groups of 128 entries that a warp has in flight: two, with registers for three CTAs on an SM, whose
// other warps hide the rest.  (Four with registers for one CTA gain 1 to 5 % up to 7 sequences
// of 32768 to 262144 entries, and lose a third from 8 on, where not all clusters find SMs of their own.)
constexpr int kGroups = 2;

template <class T>
__global__ void __launch_bounds__(kVerifyThreads, 3) verify_draft_kernel(const __grid_constant__ VerifyParams p) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / size, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, V = p.vocab;
    griddep_wait();
    griddep_launch_dependents();
    const T* target = static_cast<const T*>(p.target_probs) + (size_t)b * (p.drafts + 1) * V;
    const T* guess = p.draft_probs ? static_cast<const T*>(p.draft_probs) + (size_t)b * p.drafts * V : nullptr;
    const int* drafts = p.draft_tokens + (size_t)b * p.drafts;
    const int n = p.draft_lens ? min(max(p.draft_lens[b], 0), p.drafts) : p.drafts;
    __shared__ long long s_sum[kVerifyWarps], s_total;
    __shared__ int s_no[2];

    // every CTA accepts for itself: one draft position each thread of two warps
    if (warp < 2) {
        bool no = false;
        if (tid < n) {
            const int x = drafts[tid];
            no = true;
            if (x >= 0 && x < V) {
                const float g = guess ? prob(guess, (size_t)tid * V + x) : 1.f;
                // products of two fp32 numbers are exact in fp64
                no = !((double)p.u_accept[(size_t)b * p.drafts + tid] * (double)g < (double)prob(target, (size_t)tid * V + x));
            }
        }
        const unsigned m = __ballot_sync(~0u, no);
        if (lane == 0) s_no[warp] = m ? 32 * warp + __ffs(m) - 1 : 64;
    }
    __syncthreads();
    const int c = min(min(s_no[0], s_no[1]), n);
    const T* pr = target + (size_t)c * V;
    const T* gr = guess && c < n ? guess + (size_t)c * V : nullptr;
    // without probabilities of its own the draft has all weight at its token: nothing is left there
    const int skip = c < n && !guess ? drafts[c] : -1;
    const bool wide = !(((uintptr_t)pr | (uintptr_t)gr) & (4 * sizeof(T) - 1));
    // this warp's run of entries, a multiple of 128, and the CTA's
    const int run = ((V + size * kVerifyWarps - 1) / (size * kVerifyWarps) + 127) / 128 * 128;
    const int cta_begin = min(rank * kVerifyWarps * run, V);
    auto run_begin = [&](int w) { return min(cta_begin + w * run, V); };
    auto load = [&](auto whole, int i, int end, bool plain, float (&f)[4], float (&g)[4]) {
        constexpr bool all = decltype(whole)::value;
        four<all>(pr, i, end, wide, f);
        if (gr && !plain) four<all>(gr, i, end, wide, g);
        if (!plain && (unsigned)(skip - i) < 4u) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (i + k == skip) f[k] = 0.f;
        }
    };
    auto weigh = [&](bool plain, const float (&f)[4], const float (&g)[4], int (&hi)[4], int (&lo)[4]) {
        if (gr && !plain)
            weights<true>(f, g, hi, lo);
        else
            weights<false>(f, g, hi, lo);
    };
    long long total = 0, before = 0;
    bool plain = false;
    for (int pass = 0; pass < 2; ++pass) {
        plain = pass == 1;              // nothing left of p - g: draw from p
        long long sum = 0;
        const int end = run_begin(warp + 1);
        for (int i0 = run_begin(warp); i0 < end; i0 += 128 * kGroups) {
            float f[kGroups][4] = {}, g[kGroups][4] = {};
            if (wide && i0 + 128 * kGroups <= end) {
#pragma unroll
                for (int t = 0; t < kGroups; ++t) load(std::true_type(), i0 + 128 * t + lane * 4, end, plain, f[t], g[t]);
            } else {
#pragma unroll
                for (int t = 0; t < kGroups; ++t) {
                    const int i = i0 + 128 * t + lane * 4;
                    if (i < end) load(std::false_type(), i, end, plain, f[t], g[t]);
                }
            }
            int hi_sum = 0, lo_sum = 0;     // of 4 kGroups entries
#pragma unroll
            for (int t = 0; t < kGroups; ++t) {
                int hi[4], lo[4];
                weigh(plain, f[t], g[t], hi, lo);
                hi_sum += (hi[0] + hi[1]) + (hi[2] + hi[3]);
                lo_sum += (lo[0] + lo[1]) + (lo[2] + lo[3]);
            }
            sum += joined(hi_sum, lo_sum);
        }
        sum = warp_sum(sum);
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            const long long all = warp_sum(lane < kVerifyWarps ? s_sum[lane] : 0);
            if (lane == 0) s_total = all;
        }
        cluster.sync();
        // every rank's total, a lane each
        const long long theirs = lane < size ? *cluster.map_shared_rank(&s_total, lane) : 0;
        total = warp_sum(theirs);
        before = warp_sum(lane < rank ? theirs : 0);
        // no CTA leaves, or writes its total again, before all have read it
        cluster.barrier_arrive();
        if (total > 0 || pass == 1) break;
        cluster.barrier_wait();
    }
    if (total > 0) {
        long long r = (long long)floorf(fminf(fmaxf(p.u_next[b], 0.f), 1.f) * 16777216.f);
        if (r > (1ll << 24) - 1) r = (1ll << 24) - 1;
        // floor(total r / 2^24)
        const long long mark = (total >> 24) * r + (((total & ((1ll << 24) - 1)) * r) >> 24);
        // the warp whose run passes the mark, in the CTA whose part does
        long long at = before;
        int found = -1;
#pragma unroll
        for (int w = 0; w < kVerifyWarps; ++w) {
            const long long s = s_sum[w];
            if (found < 0 && at + s > mark) found = w;
            if (found < 0) at += s;
        }
        if (before <= mark && found >= 0) {
            const int end = run_begin(found + 1);
            for (int i0 = run_begin(found); i0 < end; i0 += kVerifyThreads * 4) {
                const int i = i0 + tid * 4;
                float f[4] = {}, g[4] = {};
                int hi[4], lo[4];
                if (i < end) load(std::false_type(), i, end, plain, f, g);
                weigh(plain, f, g, hi, lo);
                const long long own = joined((hi[0] + hi[1]) + (hi[2] + hi[3]), (lo[0] + lo[1]) + (lo[2] + lo[3]));
                const long long inc = warp_scan(own, lane);
                __syncthreads();
                if (lane == 31) s_sum[warp] = inc;
                __syncthreads();
                long long first = at + inc - own;
#pragma unroll
                for (int w = 0; w < kVerifyWarps; ++w) {
                    const long long s = s_sum[w];
                    if (w < warp) first += s;
                    at += s;
                }
                if (first <= mark && first + own > mark) {
                    int k = 0;
                    while (k < 3 && first + joined(hi[k], lo[k]) <= mark) {
                        first += joined(hi[k], lo[k]);
                        ++k;
                    }
                    p.tokens[(size_t)b * (p.drafts + 1) + c] = i + k;
                }
                if (at > mark) break;
            }
        }
    }
    if (rank == 0) {
        if (tid <= p.drafts && (tid != c || total == 0))
            p.tokens[(size_t)b * (p.drafts + 1) + tid] = tid < c ? drafts[tid] : -1;
        if (tid == 0) p.count[b] = c;
    }
    cluster.barrier_wait();
}

template <class T>
cudaError_t launch_verify(const VerifyParams& p, int batch, int sm_count, cudaStream_t stream) {
    // CTAs of a sequence: a power of two, as many as leave three to each SM (48 sequences of
    // 152064 entries: 15 us; two to each SM 17 us, one 22 us), at most 16, a cluster (one sequence:
    // 6.6 us; 8 take 7.1), each warp with 128 entries at least
    int size = 1;
    while (size < kMaxCluster && (long long)batch * size * 2 <= 3LL * sm_count &&
           size * kVerifyWarps * 128 < p.vocab)
        size *= 2;
    static std::atomic<bool> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev].load()) {
        e = cudaFuncSetAttribute(verify_draft_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        ready[dev].store(true);
    }
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)batch * size);
    cfg.blockDim = dim3(kVerifyThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_draft_kernel<T>, p);
}

}  // namespace dl

extern "C" dl_status dl_verify_draft(const int* draft_tokens, const void* draft_probs,
                                     const void* target_probs, int probs_dtype, const float* u_accept,
                                     const float* u_next, const int* draft_lens, int* tokens,
                                     int* count, int batch, int drafts, int vocab, void* stream) {
    using namespace dl;
    if (probs_dtype != DL_PROBS_F32 && probs_dtype != DL_PROBS_BF16)
        return host_fail(DL_ERR_INVALID_ARG, "unknown probs_dtype %d", probs_dtype);
    if (batch < 0 || batch > (1 << 24))
        return host_fail(DL_ERR_INVALID_ARG, "batch=%d is outside [0, 2^24]", batch);
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
    HostDevice device;
    const dl_status s = host_device(device);
    if (s != DL_OK) return s;
    const cudaError_t e = probs_dtype == DL_PROBS_F32 ? launch_verify<float>(p, batch, device.sm_count, st)
                                                      : launch_verify<uint16_t>(p, batch, device.sm_count, st);
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "verify_draft launch: %s", cudaGetErrorString(e));
    return host_ok();
}
