// Rotation of the new tokens' queries and keys, and their keys' and values'
// way into the paged 8-bit cache (dl_kv_append).
#include "dl_host.h"
#include "kv_cache.cuh"

namespace dl {

struct AppendParams {
    dl_kv_cache c;
    const uint16_t *q, *k, *v;
    uint16_t* q_out;
    long long q_stride, k_stride, v_stride;
    const float *cos, *sin;
    const int* positions;
    int rotary_dim, max_pos, q_heads;
    int page_shift, block_shift;
    int blocks_per_seq;          // most blocks a sequence's new tokens touch
    Sequences s;
};

constexpr int kAppendThreads = 128;

// The new value of dim d of one row (a token's head), rotated at `pos`.
__device__ __forceinline__ float rotated(const AppendParams& p, const uint16_t* row, int d, int pos) {
    const float x = bf16_bits_to_f32(row[d]);
    if (!p.cos || d >= p.rotary_dim) return x;
    const int h = p.rotary_dim / 2;
    const int i = d < h ? d : d - h;
    const float c = p.cos[(size_t)pos * h + i], s = p.sin[(size_t)pos * h + i];
    const float y = bf16_bits_to_f32(row[d < h ? d + h : d - h]);
    return d < h ? __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s))
                 : __fadd_rn(__fmul_rn(x, c), __fmul_rn(y, s));
}

__device__ __forceinline__ int position_of(const AppendParams& p, int t, int index) {
    const int at = p.positions ? p.positions[t] : index;
    return min(max(at, 0), p.max_pos - 1);
}

__device__ __forceinline__ float e4m3_value(uint8_t code) {
    uint32_t lo, hi;
    e4m3x4_to_f16x2x2(code, lo, hi);
    float f;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(lo));
    return f;
}

// The smallest power of two s >= 2^-40 with 448 s >= amax (448 = 1.75 * 2^8).
__device__ __forceinline__ float block_scale(float amax) {
    const unsigned bits = __float_as_uint(amax);
    int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(e, -40);
    return __uint_as_float((unsigned)(e + 127) << 23);
}

// grid.x: first one CTA for each token's queries, then one for each (sequence,
// touched block, head, key or value).
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
    const int D = p.c.head_dim;
    const int tid = threadIdx.x;
    int unit = blockIdx.x;
    if (p.q) {
        if (unit < p.s.tokens) {
            const int t = unit;
            int before = 0;
            for (int b = 0; b < p.s.batch; ++b) before += p.s.q_start[b + 1] <= t;
            if (before >= p.s.batch) return;
            const SequenceView sv = sequence_view(p.s, before, p.c.page_size);
            const int i = t - sv.row0;
            if (i < 0 || i >= sv.n_work) return;
            const int pos = position_of(p, t, sv.len - sv.n + i);
            // both dims of a rotation by one thread, so that q_out may be q
            const int half = D / 2, hr = p.cos ? p.rotary_dim / 2 : 0;
            for (int e = tid; e < p.q_heads * half; e += kAppendThreads) {
                const int h = e / half, i2 = e % half;
                const int d0 = i2 < hr ? i2 : 2 * i2, d1 = i2 < hr ? i2 + hr : 2 * i2 + 1;
                const uint16_t* row = p.q + (size_t)t * p.q_stride + (size_t)h * D;
                const float a = rotated(p, row, d0, pos), c = rotated(p, row, d1, pos);
                uint16_t* to = p.q_out + ((size_t)t * p.q_heads + h) * D;
                to[d0] = f32_to_bf16_rne(a);
                to[d1] = f32_to_bf16_rne(c);
            }
            return;
        }
        unit -= p.s.tokens;
    }
    const bool is_v = unit & 1;
    unit >>= 1;
    const int h = unit % p.c.num_heads;
    unit /= p.c.num_heads;
    const int j = unit % p.blocks_per_seq, b = unit / p.blocks_per_seq;
    const SequenceView sv = sequence_view(p.s, b, p.c.page_size);
    const int first = sv.len - sv.n;                        // cache index of the first new token
    const int last = first + sv.n_work;                     // past the last one worked on
    const int begin = max(first, 0);
    const int blk = ((begin >> p.block_shift) + j) << p.block_shift;
    if (blk >= last) return;
    const int page = p.s.block_table[(size_t)b * p.s.table_cols + (blk >> p.page_shift)];
    if (page < 0 || page >= p.c.num_pages) return;
    const int t0 = blk & (p.c.page_size - 1);
    uint8_t* codes = static_cast<uint8_t*>(is_v ? p.c.v : p.c.k) + page * p.c.page_stride +
                     h * p.c.head_stride + (size_t)t0 * D;
    float* scale = (is_v ? p.c.v_scale : p.c.k_scale) + page * p.c.scale_page_stride +
                   h * p.c.scale_head_stride + (t0 >> p.block_shift);
    const uint16_t* src = is_v ? p.v : p.k;
    const long long stride = is_v ? p.v_stride : p.k_stride;
    const int lo = max(blk, begin), hi = min(blk + p.c.block, last);

    auto value = [&](int index, int d) {
        const int t = sv.row0 + index - first;
        const uint16_t* row = src + (size_t)t * stride + (size_t)h * D;
        return is_v ? bf16_bits_to_f32(row[d]) : rotated(p, row, d, position_of(p, t, index));
    };
    float amax = 0.f;
    for (int e = tid; e < (hi - lo) * D; e += kAppendThreads) {
        const float a = fabsf(value(lo + e / D, e % D));
        if (a <= 3.402823466e38f) amax = fmaxf(amax, a);
    }
    __shared__ float part[kAppendThreads / 32];
    amax = __uint_as_float(warp_max_u32(__float_as_uint(amax)));
    if ((tid & 31) == 0) part[tid >> 5] = amax;
    __syncthreads();
    for (int w = 0; w < kAppendThreads / 32; ++w) amax = fmaxf(amax, part[w]);
    float s1 = block_scale(amax);
    const float s0 = *scale;
    const bool had = lo > blk;
    if (had && !(s0 < s1)) s1 = s0;
    const float inv = __frcp_rn(s1);
    __syncthreads();
    if (had && s1 != s0)
        for (int e = tid; e < (lo - blk) * D; e += kAppendThreads)
            codes[e] = (uint8_t)f32x2_to_e4m3x2(__fmul_rn(__fmul_rn(e4m3_value(codes[e]), s0), inv), 0.f);
    for (int e = tid; e < (hi - lo) * D; e += kAppendThreads)
        codes[(lo - blk) * D + e] =
            (uint8_t)f32x2_to_e4m3x2(__fmul_rn(value(lo + e / D, e % D), inv), 0.f);
    if (tid == 0) *scale = s1;
}

namespace {
bool pow2(int v) { return v > 0 && (v & (v - 1)) == 0; }
int log2i(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}
}  // namespace

dl_status check_cache(const dl_kv_cache* c) {
    if (!c) return host_fail(DL_ERR_INVALID_ARG, "cache is NULL");
    if (!c->k || !c->v || !c->k_scale || !c->v_scale)
        return host_fail(DL_ERR_INVALID_ARG, "a cache pointer is NULL");
    if (c->num_pages < 1 || c->num_heads < 1)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "num_pages=%d and num_heads=%d must be >= 1",
                         c->num_pages, c->num_heads);
    if (c->head_dim != 64 && c->head_dim != 128)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "head_dim=%d is neither 64 nor 128", c->head_dim);
    if (!pow2(c->page_size) || c->page_size < 8 || c->page_size > 1024)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "page_size=%d is not a power of two in [8, 1024]",
                         c->page_size);
    if (!pow2(c->block) || c->block > c->page_size)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "block=%d is not a power of two in [1, page_size]",
                         c->block);
    const long long dense = (long long)c->page_size * c->head_dim;
    if (c->page_stride % 16 || c->head_stride % 16 || c->head_stride < dense || c->page_stride < dense ||
        c->scale_head_stride < c->page_size / c->block || c->scale_page_stride < c->page_size / c->block)
        return host_fail(DL_ERR_INVALID_ARG,
                         "cache strides: codes need multiples of 16 bytes >= %lld, scales >= %d", dense,
                         c->page_size / c->block);
    if (((uintptr_t)c->k | (uintptr_t)c->v) & 15)
        return host_fail(DL_ERR_MISALIGNED, "cache codes must be 16-byte aligned");
    if (((uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 3)
        return host_fail(DL_ERR_MISALIGNED, "cache scales must be 4-byte aligned");
    return DL_OK;
}

dl_status check_sequences(const int* block_table, int table_cols, const int* seq_lens,
                          const int* q_start, int batch, int tokens, int max_q) {
    if (batch < 0 || tokens < 0 || max_q < 0)
        return host_fail(DL_ERR_INVALID_ARG, "batch=%d, tokens=%d and max_q=%d must be >= 0", batch,
                         tokens, max_q);
    if (batch == 0 || tokens == 0 || max_q == 0) return DL_OK;      // nothing to do
    if (!block_table || !seq_lens || !q_start)
        return host_fail(DL_ERR_INVALID_ARG, "block_table, seq_lens or q_start is NULL");
    if (table_cols < 1) return host_fail(DL_ERR_INVALID_ARG, "table_cols=%d must be >= 1", table_cols);
    if (((uintptr_t)block_table | (uintptr_t)seq_lens | (uintptr_t)q_start) & 3)
        return host_fail(DL_ERR_MISALIGNED, "block_table, seq_lens and q_start must be 4-byte aligned");
    return DL_OK;
}

}  // namespace dl

extern "C" dl_status dl_kv_append(const dl_kv_cache* cache, const void* q, const void* k, const void* v,
                                  long long q_stride, long long k_stride, long long v_stride,
                                  void* q_out, const float* cos, const float* sin, int rotary_dim,
                                  int max_pos, const int* positions, const int* block_table,
                                  int table_cols, const int* seq_lens, const int* q_start, int batch,
                                  int tokens, int q_heads, int max_q, void* stream) {
    using namespace dl;
    dl_status s = check_cache(cache);
    if (s != DL_OK) return s;
    if ((s = check_sequences(block_table, table_cols, seq_lens, q_start, batch, tokens, max_q)) != DL_OK)
        return s;
    const int D = cache->head_dim;
    if (!cos != !sin) return host_fail(DL_ERR_INVALID_ARG, "cos and sin go together");
    if (cos && (rotary_dim < 16 || rotary_dim > D || rotary_dim % 16 || max_pos < 1))
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE,
                         "rotary_dim=%d is not a multiple of 16 in [16, %d], or max_pos=%d < 1",
                         rotary_dim, D, max_pos);
    if (!q != !q_out) return host_fail(DL_ERR_INVALID_ARG, "q and q_out go together");
    if (q && q_heads < 1) return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "q_heads=%d must be >= 1", q_heads);
    if (batch == 0 || tokens == 0 || max_q == 0) return host_ok();
    if (!k || !v) return host_fail(DL_ERR_INVALID_ARG, "k or v is NULL");
    if ((q && (q_stride < (long long)q_heads * D || q_stride % 8)) ||
        k_stride < (long long)cache->num_heads * D || v_stride < (long long)cache->num_heads * D ||
        k_stride % 8 || v_stride % 8)
        return host_fail(DL_ERR_INVALID_ARG,
                         "q, k and v strides must be multiples of 8 elements that hold a token's heads");
    if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)q_out | (uintptr_t)cos | (uintptr_t)sin) & 15)
        return host_fail(DL_ERR_MISALIGNED, "q, k, v, q_out, cos and sin must be 16-byte aligned");
    if ((uintptr_t)positions & 3) return host_fail(DL_ERR_MISALIGNED, "positions must be 4-byte aligned");
    AppendParams p = {};
    p.c = *cache;
    p.q = static_cast<const uint16_t*>(q);
    p.k = static_cast<const uint16_t*>(k);
    p.v = static_cast<const uint16_t*>(v);
    p.q_out = static_cast<uint16_t*>(q_out);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.cos = cos;
    p.sin = sin;
    p.positions = positions;
    p.rotary_dim = rotary_dim;
    p.max_pos = cos ? max_pos : 1;
    p.q_heads = q_heads;
    p.page_shift = log2i(cache->page_size);
    p.block_shift = log2i(cache->block);
    p.s = Sequences{block_table, seq_lens, q_start, table_cols, batch, tokens, max_q};
    const long long most = max_q < tokens ? max_q : tokens;
    p.blocks_per_seq = (int)((most + cache->block - 2) / cache->block + 1);
    const long long units = (q ? tokens : 0) + 2LL * batch * p.blocks_per_seq * cache->num_heads;
    if (units > 0x7fffffffLL)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "%lld blocks to write exceed one launch", units);
    kv_append_kernel<<<(unsigned)units, kAppendThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "kv_append launch: %s", cudaGetErrorString(e));
    return host_ok();
}
