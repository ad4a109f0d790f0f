// Verification of drafted tokens and the draw of the next one (dl_verify_draft).
#include <cooperative_groups.h>

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

// A cluster of CTAs takes one sequence, each a contiguous part of its vocabulary.
// What bounds it: for many sequences the one read of p (and g), for few the
// chain of dependent loads (draft token, its probabilities, the row).  The sums
// of the first pass are kept by CTA, tile and warp, so that the drawn token is
// found by reading 128 entries again, not the row.
constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kVerifyTile = kVerifyThreads * 4;             // entries of a tile
constexpr int kMaxCluster = 8;
constexpr int kMaxTiles = (1 << 18) / kMaxCluster / kVerifyTile;
constexpr int kWeightBits = 44;

// Four consecutive probabilities from entry i on, entries at or past `end` as
// zeros; `wide`: the row's groups of four are aligned to their size.
__device__ __forceinline__ void four(const float* row, int i, int end, bool wide, float (&f)[4]) {
    if (wide && i + 4 <= end) {
        const uint4 v = ldg128(row + i);
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = i + k < end ? row[i + k] : 0.f;
    }
}
__device__ __forceinline__ void four(const uint16_t* row, int i, int end, bool wide, float (&f)[4]) {
    if (wide && i + 4 <= end) {
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

// A probability, taken inside [0, 1] (NaN: 0), as the whole number nearest to x 2^44: hi 2^22 + lo.
// Adding 1.5 * 2^23 leaves a rounded integer in an fp32's low bits; hi's rounding error is
// exact in fp32, so lo rounds the whole value once, to even at ties (hi 2^22 is even).
__device__ __forceinline__ void whole(float x, int& hi, int& lo) {
    constexpr float kMagic = 12582912.f, kStep = 4194304.f;   // 1.5 * 2^23, 2^22
    x = fminf(fmaxf(x, 0.f), 1.f);
    const float y = __fmul_rn(x, kStep);
    const float a = __fadd_rn(y, kMagic);
    hi = __float_as_int(a) - __float_as_int(kMagic);
    const float rest = __fsub_rn(y, __fsub_rn(a, kMagic));
    lo = __float_as_int(__fadd_rn(__fmul_rn(rest, kStep), kMagic)) - __float_as_int(kMagic);
}

__device__ __forceinline__ long long warp_sum(long long w) {
    for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(~0u, w, o);
    return w;
}

template <class T>
__global__ void __launch_bounds__(kVerifyThreads) verify_draft_kernel(const __grid_constant__ VerifyParams p) {
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
    __shared__ long long s_sum[kMaxTiles * kVerifyWarps], s_total;
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
    const int x = c < n && !guess ? drafts[c] : -1;
    const bool wide = !(((uintptr_t)pr | (uintptr_t)gr) & (4 * sizeof(T) - 1));
    // this CTA's part, a whole number of tiles from its begin on
    const int tiles = ((V + kVerifyTile - 1) / kVerifyTile + size - 1) / size;
    const int begin = min(rank * tiles * kVerifyTile, V), end = min(begin + tiles * kVerifyTile, V);
    auto weights = [&](int i, bool plain, long long (&w)[4]) {
        float f[4], g[4] = {0.f, 0.f, 0.f, 0.f};
        four(pr, i, end, wide, f);
        if (gr && !plain) four(gr, i, end, wide, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            int ph, pl, gh, gl;
            whole(f[k], ph, pl);
            whole(g[k], gh, gl);
            if (i + k == x && !plain) gh = 1 << (kWeightBits - 22);
            const long long d = (long long)(ph - gh) * (1 << 22) + (pl - gl);
            w[k] = d > 0 ? d : 0;
        }
    };
    long long total = 0, before = 0;
    bool plain = false;
    for (int pass = 0; pass < 2; ++pass) {
        plain = pass == 1;              // nothing left of p - g: draw from p
        long long mine = 0;
#pragma unroll 2
        for (int t = 0; t < tiles; ++t) {
            const int i = begin + t * kVerifyTile + tid * 4;
            long long w[4] = {0, 0, 0, 0};
            if (i < end) weights(i, plain, w);
            const long long s = warp_sum((w[0] + w[1]) + (w[2] + w[3]));
            if (lane == 0) s_sum[t * kVerifyWarps + warp] = s;
        }
        __syncthreads();
        if (warp == 0) {
            for (int i = lane; i < tiles * kVerifyWarps; i += 32) mine += s_sum[i];
            mine = warp_sum(mine);
            if (lane == 0) s_total = mine;
        }
        cluster.sync();
        total = before = 0;
        for (int r = 0; r < size; ++r) {
            const long long s = *cluster.map_shared_rank(&s_total, r);
            if (r < rank) before += s;
            total += s;
        }
        cluster.sync();
        if (total > 0) break;
    }
    if (total > 0 && warp == 0) {
        long long r = (long long)floorf(fminf(fmaxf(p.u_next[b], 0.f), 1.f) * 16777216.f);
        if (r > (1ll << 24) - 1) r = (1ll << 24) - 1;
        // floor(total r / 2^24)
        const long long mark = (total >> 24) * r + (((total & ((1ll << 24) - 1)) * r) >> 24);
        // the warp's run of 128 entries whose sums pass the mark, then the entry
        long long run = before;
        int found = -1;
        for (int i0 = 0; i0 < tiles * kVerifyWarps && found < 0; i0 += 32) {
            const long long s = i0 + lane < tiles * kVerifyWarps ? s_sum[i0 + lane] : 0;
            long long inc = s;
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(~0u, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned hit = __ballot_sync(~0u, run + inc > mark);
            if (hit) {
                const int src = __ffs(hit) - 1;
                found = i0 + src;
                run += __shfl_sync(~0u, inc - s, src);
            } else {
                run += __shfl_sync(~0u, inc, 31);
            }
        }
        if (found >= 0 && before <= mark) {
            const int i = begin + found / kVerifyWarps * kVerifyTile + found % kVerifyWarps * 128 + lane * 4;
            long long w[4] = {0, 0, 0, 0};
            if (i < end) weights(i, plain, w);
            long long inc = (w[0] + w[1]) + (w[2] + w[3]);
            const long long own = inc;
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(~0u, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned hit = __ballot_sync(~0u, run + inc > mark);
            if (lane == __ffs(hit) - 1) {
                long long at = run + inc - own;
                int k = 0;
                while (k < 3 && at + w[k] <= mark) at += w[k++];
                p.tokens[(size_t)b * (p.drafts + 1) + c] = i + k;
            }
        }
    }
    if (rank == 0) {
        if (tid <= p.drafts && (tid != c || total == 0))
            p.tokens[(size_t)b * (p.drafts + 1) + tid] = tid < c ? drafts[tid] : -1;
        if (tid == 0) p.count[b] = c;
    }
}

template <class T>
cudaError_t launch_verify(const VerifyParams& p, int batch, cudaStream_t stream) {
    // CTAs of a sequence: one for each two tiles of its vocabulary, up to the portable 8
    int size = 1;
    while (size < kMaxCluster && size * 2 * kVerifyTile < p.vocab) size *= 2;
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
    const cudaError_t e = probs_dtype == DL_PROBS_F32 ? launch_verify<float>(p, batch, st)
                                                      : launch_verify<uint16_t>(p, batch, st);
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "verify_draft launch: %s", cudaGetErrorString(e));
    return host_ok();
}
