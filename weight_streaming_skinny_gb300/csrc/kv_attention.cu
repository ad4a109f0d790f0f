// Attention over the paged 8-bit cache (dl_attention_paged): arguments, the
// shape of a row tile, the workspace and the launch.
#include "dl_host.h"
#include "kv_attention.cuh"

namespace {

// Row tiles of at most kMaxRows rows, as even as the new tokens allow.  A group
// of more heads is cut into equal parts that each read the cache.
struct RowTiles {
    int parts, tokens, count, padded;
};

RowTiles row_tiles(int tokens, int max_q, int group) {
    RowTiles r;
    r.parts = 1;
    while (group / r.parts > dl::kMaxRows || group % r.parts) ++r.parts;
    const int heads = group / r.parts, most = dl::kMaxRows / heads, n = max_q < tokens ? max_q : tokens;
    r.count = (n + most - 1) / most;
    r.tokens = (n + r.count - 1) / r.count;
    r.padded = dl::attn_rows_padded(r.tokens * heads);
    return r;
}

size_t split_bytes(int grid) { return ((size_t)grid * sizeof(dl::AttnSplit) + 255) / 256 * 256; }

size_t workspace_bytes(int grid, int rp, int dim) {
    return DL_WORKSPACE_ZERO_BYTES + split_bytes(grid) + (size_t)grid * 2 * rp * (dim + 2) * sizeof(float);
}

// The codes as a tensor (dim, token, head, page); a box is a page's tokens, at
// most a tile's.
dl_status encode_codes(const dl_kv_cache& c, void* codes, CUtensorMap& map) {
    dl::EncodeTiled enc;
    const dl_status s = dl::host_encode(enc);
    if (s != DL_OK) return s;
    const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size, (cuuint64_t)c.num_heads,
                                (cuuint64_t)c.num_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.head_stride, (cuuint64_t)c.page_stride};
    const cuuint32_t box[4] = {(cuuint32_t)c.head_dim,
                               (cuuint32_t)(c.page_size < dl::kTile ? c.page_size : dl::kTile), 1, 1};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    const CUresult r = enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, codes, dims, strides, box, ones,
                           CU_TENSOR_MAP_INTERLEAVE_NONE,
                           c.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return dl::host_fail(DL_ERR_CUDA, "cuTensorMapEncodeTiled(cache): %d", (int)r);
    return DL_OK;
}

}  // namespace

extern "C" size_t dl_attention_workspace_bytes(int batch, int tokens, int q_heads, int kv_heads,
                                               int head_dim, int max_q) {
    if (batch < 0 || tokens < 0 || q_heads < 1 || kv_heads < 1 || q_heads % kv_heads ||
        q_heads / kv_heads > 128 || (head_dim != 64 && head_dim != 128) || max_q < 0) {
        dl::host_fail(DL_ERR_UNSUPPORTED_SHAPE, "attention sizes are out of range");
        return 0;
    }
    if (batch == 0 || tokens == 0 || max_q == 0) return DL_WORKSPACE_ZERO_BYTES;
    dl::HostDevice dev;
    if (dl::host_device(dev) != DL_OK) return 0;
    // a step of fewer tokens may need more (its instance has more CTAs or rows): the largest need of
    // all up to max_q.  Steps of more than one row tile have the tiles of some step of one.
    size_t most = 0;
    for (int n = 1; n <= dl::kMaxRows && n <= tokens && n <= max_q; ++n) {
        const int rp = row_tiles(tokens, n, q_heads / kv_heads).padded;
        const size_t need = workspace_bytes(dev.sm_count * dl::attn_ctas_per_sm(rp, head_dim), rp, head_dim);
        most = need > most ? need : most;
    }
    return most;
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
    if (!workspace) return host_fail(DL_ERR_WORKSPACE, "workspace is NULL");
    if ((uintptr_t)workspace & 255) return host_fail(DL_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    HostDevice dev;
    if ((s = host_device(dev)) != DL_OK) return s;
    const int group = q_heads / cache->num_heads;
    const RowTiles rt = row_tiles(tokens, max_q, group);
    if ((long long)batch * rt.count > 0x7fffffffLL)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "batch=%d times %d row tiles exceed one launch", batch, rt.count);
    AttnLaunch a = {};
    a.grid = dev.sm_count * attn_ctas_per_sm(rt.padded, cache->head_dim);
    a.stream = static_cast<cudaStream_t>(stream);
    const size_t need = workspace_bytes(a.grid, rt.padded, cache->head_dim);
    if (ws_bytes < need)
        return host_fail(DL_ERR_WORKSPACE, "workspace holds %zu bytes, %zu are needed", ws_bytes, need);
    if ((s = encode_codes(*cache, cache->k, a.tk)) != DL_OK) return s;
    if ((s = encode_codes(*cache, cache->v, a.tv)) != DL_OK) return s;
    AttnParams& p = a.p;
    p.q = static_cast<const uint16_t*>(q);
    p.out = static_cast<uint16_t*>(out);
    p.lse = lse;
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.q_stride = q_stride;
    p.scale_page_stride = cache->scale_page_stride;
    p.scale_head_stride = cache->scale_head_stride;
    p.num_pages = cache->num_pages;
    p.head_parts = rt.parts;
    p.kv_heads = cache->num_heads * rt.parts;
    p.q_heads = q_heads;
    p.group = group / rt.parts;
    p.page_size = cache->page_size;
    while ((1 << p.page_shift) < cache->page_size) ++p.page_shift;
    while ((1 << p.block_shift) < cache->block) ++p.block_shift;
    p.tile_tokens = rt.tokens;
    p.row_tiles = rt.count;
    p.scale_log2 = scale * 1.44269504088896341f;
    p.s = Sequences{block_table, seq_lens, q_start, table_cols, batch, tokens, max_q};
    unsigned char* ws = static_cast<unsigned char*>(workspace) + DL_WORKSPACE_ZERO_BYTES;
    p.split = reinterpret_cast<AttnSplit*>(ws);
    p.partial = reinterpret_cast<float*>(ws + split_bytes(a.grid));
    p.err_word = dev.err_word;
    p.wait_limit_ns = dev.wait_limit_ns;
    p.withhold = dev.withhold_stage;
    const cudaError_t e = cache->head_dim == 128 ? launch_attention_d128(rt.padded, a)
                                                 : launch_attention_d64(rt.padded, a);
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "attention launch: %s", cudaGetErrorString(e));
    return host_ok();
}
