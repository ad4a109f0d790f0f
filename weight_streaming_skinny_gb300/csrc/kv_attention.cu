// Attention over the paged 8-bit cache (dl_attention_paged).
#include "dl_host.h"
#include "kv_cache.cuh"

namespace dl {

struct AttnParams {
    dl_kv_cache c;
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    long long q_stride;
    int q_heads, group;
    int page_shift, block_shift;
    float scale_log2;            // scale * log2(e)
    Sequences s;
};

// One warp for each (token, query head): lanes take tokens for the scores and
// dims for the sum.
__global__ void __launch_bounds__(128) attention_simple_kernel(const __grid_constant__ AttnParams p) {
    const int D = p.c.head_dim, lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (unit >= (long long)p.s.tokens * p.q_heads) return;
    const int t = (int)(unit / p.q_heads), h = (int)(unit % p.q_heads), hk = h / p.group;
    int b = 0;
    while (b < p.s.batch && p.s.q_start[b + 1] <= t) ++b;
    if (b >= p.s.batch) return;
    const SequenceView sv = sequence_view(p.s, b, p.c.page_size);
    const int i = t - sv.row0;
    if (i < 0 || i >= sv.n_work) return;
    const int seen = max(sv.len - sv.n + i + 1, 0);
    const uint16_t* q = p.q + (size_t)t * p.q_stride + (size_t)h * D;
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < seen; j0 += 32) {
        const int j = j0 + lane;
        int page = -1;
        if (j < seen) page = p.s.block_table[(size_t)b * p.s.table_cols + (j >> p.page_shift)];
        const bool in = page >= 0 && page < p.c.num_pages;
        const int in_page = j & (p.c.page_size - 1);
        const long long at = page * p.c.page_stride + hk * p.c.head_stride + (long long)in_page * D;
        const long long sc = page * p.c.scale_page_stride + hk * p.c.scale_head_stride + (in_page >> p.block_shift);
        float s = -INFINITY;
        if (in) {
            s = 0.f;
            const uint8_t* k = static_cast<const uint8_t*>(p.c.k) + at;
            for (int d = 0; d < D; d += 2) {
                const uint32_t kk = e4m3x2_to_bf16x2(k[d] | (uint32_t)k[d + 1] << 8);
                s = fma2_bf16(kk, q[d] | (uint32_t)q[d + 1] << 16, s);
            }
            s *= p.c.k_scale[sc] * p.scale_log2;
        }
        float top = s;
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
        const float m1 = fmaxf(m, top);
        const float base = m1 == -INFINITY ? 0.f : m1;
        const float fix = exp2f(m - base);
        const float w = in ? exp2f(s - base) : 0.f;
        l = l * fix + w;
        for (float& a : acc) a *= fix;
        m = m1;
        for (int r = 0; r < 32 && j0 + r < seen; ++r) {
            const float wr = __shfl_sync(~0u, w, r);
            const long long ar = __shfl_sync(~0u, at, r), sr = __shfl_sync(~0u, sc, r);
            if (!__shfl_sync(~0u, (int)in, r)) continue;
            const uint8_t* v = static_cast<const uint8_t*>(p.c.v) + ar;
            const float ws = wr * p.c.v_scale[sr];
            for (int c = 0; c < D / 32; ++c)
                acc[c] = fmaf(ws, __uint_as_float(e4m3x2_to_bf16x2(v[32 * c + lane]) << 16), acc[c]);
        }
    }
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
    for (int c = 0; c < D / 32; ++c)
        p.out[((size_t)t * p.q_heads + h) * D + 32 * c + lane] =
            f32_to_bf16_rne(l == 0.f ? 0.f : acc[c] / l);
    if (p.lse && lane == 0)
        p.lse[(size_t)t * p.q_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718056f;
}

}  // namespace dl

extern "C" size_t dl_attention_workspace_bytes(int batch, int tokens, int q_heads, int kv_heads,
                                               int head_dim, int max_q) {
    if (batch < 0 || tokens < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads ||
        q_heads / kv_heads > 128 || (head_dim != 64 && head_dim != 128) || max_q < 0) {
        dl::host_fail(DL_ERR_UNSUPPORTED_SHAPE, "attention sizes are out of range");
        return 0;
    }
    return DL_WORKSPACE_ZERO_BYTES;
}

extern "C" dl_status dl_attention_paged(const dl_kv_cache* cache, const void* q, long long q_stride,
                                        void* out, float* lse, const int* block_table, int table_cols,
                                        const int* seq_lens, const int* q_start, int batch, int tokens,
                                        int q_heads, int max_q, float scale, void* workspace,
                                        size_t ws_bytes, void* stream) {
    using namespace dl;
    dl_status s = check_cache(cache);
    if (s != DL_OK) return s;
    if ((s = check_sequences(block_table, table_cols, seq_lens, q_start, batch, tokens, max_q)) != DL_OK)
        return s;
    if (q_heads < 1 || q_heads % cache->num_heads || q_heads / cache->num_heads > 128)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "q_heads=%d is not 1 to 128 times num_heads=%d", q_heads,
                         cache->num_heads);
    if (batch == 0 || tokens == 0 || max_q == 0) return host_ok();
    if (!q || !out) return host_fail(DL_ERR_INVALID_ARG, "q or out is NULL");
    if (q_stride < (long long)q_heads * cache->head_dim || q_stride % 8)
        return host_fail(DL_ERR_INVALID_ARG, "q_stride=%lld must be a multiple of 8 that holds %d heads",
                         q_stride, q_heads);
    if (((uintptr_t)q | (uintptr_t)out) & 15)
        return host_fail(DL_ERR_MISALIGNED, "q and out must be 16-byte aligned");
    if ((uintptr_t)lse & 3) return host_fail(DL_ERR_MISALIGNED, "lse must be 4-byte aligned");
    const size_t need = dl_attention_workspace_bytes(batch, tokens, q_heads, cache->num_heads,
                                                     cache->head_dim, max_q);
    if (!workspace) return host_fail(DL_ERR_WORKSPACE, "workspace is NULL");
    if (ws_bytes < need)
        return host_fail(DL_ERR_WORKSPACE, "workspace holds %zu bytes, %zu are needed", ws_bytes, need);
    AttnParams p = {};
    p.c = *cache;
    p.q = static_cast<const uint16_t*>(q);
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.q_stride = q_stride;
    p.q_heads = q_heads;
    p.group = q_heads / cache->num_heads;
    while ((1 << p.page_shift) < cache->page_size) ++p.page_shift;
    while ((1 << p.block_shift) < cache->block) ++p.block_shift;
    p.scale_log2 = scale * 1.44269504089f;
    p.s = Sequences{block_table, seq_lens, q_start, table_cols, batch, tokens, max_q};
    const long long units = ((long long)tokens * q_heads + 3) / 4;
    if (units > 0x7fffffffLL) return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "too many tokens for one launch");
    attention_simple_kernel<<<(unsigned)units, 128, 0, static_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
    return host_ok();
}
