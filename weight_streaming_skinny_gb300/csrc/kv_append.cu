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
    int team, per;               // threads of a block; tokens whose queries a CTA takes
    int kv_ctas, q_ctas, period; // CTAs that take blocks, and queries
    long long kv_units;          // blocks that get new tokens, at most
    Sequences s;
};

// What bounds it: memory.  A token's queries are read and written once, keys and
// values read once and written as codes.  A thread takes 16 dims at a time, the
// two groups of 8 that rotate into one another (or 16 dims that pass through):
// 16-byte loads and stores, and cos and sin stay in its registers while it goes
// through a token's heads.  4 prompts of 4096 tokens (64 query and 8 key/value heads of
// 128, 487 MB): 78 us, 6.2 TB/s; 48 x 6 tokens: 4.9 us, one token: 3.4 us, both the chain
// launch, sequence, page, scale, codes.
constexpr int kAppendThreads = 256;

__device__ __forceinline__ int position_of(const AppendParams& p, int t, int index) {
    const int at = p.positions ? p.positions[t] : index;
    return min(max(at, 0), p.max_pos - 1);
}

// Unit u of a row's D / 16: its two groups of 8 dims start at `a` and `b`.
struct RowUnit {
    int a, b, angle;            // angle: index of the first cos / sin, or -1
};
__device__ __forceinline__ RowUnit row_unit(int u, int rotary_dim) {
    const int pairs = rotary_dim / 16;
    if (u < pairs) return {8 * u, 8 * u + rotary_dim / 2, 8 * u};
    return {16 * u, 16 * u + 8, -1};
}

__device__ __forceinline__ void load_angles(const AppendParams& p, int pos, int angle, float (&c)[8], float (&s)[8]) {
    const size_t at = (size_t)pos * (p.rotary_dim / 2) + angle;
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
        const uint4 x = ldg128(p.cos + at + k), y = ldg128(p.sin + at + k);
        c[k] = __uint_as_float(x.x); c[k + 1] = __uint_as_float(x.y);
        c[k + 2] = __uint_as_float(x.z); c[k + 3] = __uint_as_float(x.w);
        s[k] = __uint_as_float(y.x); s[k + 1] = __uint_as_float(y.y);
        s[k + 2] = __uint_as_float(y.z); s[k + 3] = __uint_as_float(y.w);
    }
}

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}

// f[0..8) and f[8..16) rotated into one another; each product and sum rounded
// on its own, so that the codes do not depend on how it is compiled.
__device__ __forceinline__ void rotate(float (&f)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float x = f[k], y = f[k + 8];
        f[k] = __fsub_rn(__fmul_rn(x, c[k]), __fmul_rn(y, s[k]));
        f[k + 8] = __fadd_rn(__fmul_rn(y, c[k]), __fmul_rn(x, s[k]));
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
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

// One CTA: the queries of `per` (1 or 4) tokens, every head, a share of the threads for each
// token.  The first heads are read before the token's sequence and position are
// known, so that the latencies of the two overlap.
template <int D>
__device__ __forceinline__ void append_queries(const AppendParams& p, int t0) {
    constexpr int kUnits = D / 16, kAhead = 2;
    const int threads = kAppendThreads / p.per, step = threads / kUnits;
    const int tid = threadIdx.x % threads, h0 = tid / kUnits, t = t0 + threadIdx.x / threads;
    const RowUnit u = row_unit(tid % kUnits, p.rotary_dim);
    const uint16_t* src = p.q + (size_t)min(t, p.s.tokens - 1) * p.q_stride;
    uint4 x[kAhead], y[kAhead];
    auto read = [&](int h) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (h + i * step < p.q_heads) {
                x[i] = ldg128(src + (size_t)(h + i * step) * D + u.a);
                y[i] = ldg128(src + (size_t)(h + i * step) * D + u.b);
            }
    };
    read(h0);
    int b = 0;                          // sequences that end at or before t
    for (int i = 0; i < p.s.batch; i += kAppendThreads)
        b += __syncthreads_count(i + (int)threadIdx.x < p.s.batch && p.s.q_start[i + threadIdx.x + 1] <= t0);
    if (t >= p.s.tokens) return;
    while (b < p.s.batch && p.s.q_start[b + 1] <= t) ++b;
    if (b >= p.s.batch) return;
    const SequenceView sv = sequence_view(p.s, b, p.c.page_size);
    const int i = t - sv.row0;
    if (i < 0 || i >= sv.n_work) return;
    float c[8], s[8];
    if (u.angle >= 0) load_angles(p, position_of(p, t, sv.len - sv.n + i), u.angle, c, s);
    uint16_t* dst = p.q_out + (size_t)t * p.q_heads * D;
    for (int h = h0;;) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (h + k * step >= p.q_heads) continue;
            float f[16];
            unpack8(x[k], f);
            unpack8(y[k], f + 8);
            if (u.angle >= 0) rotate(f, c, s);
            uint16_t* to = dst + (size_t)(h + k * step) * D;
            *reinterpret_cast<uint4*>(to + u.a) =
                make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
            *reinterpret_cast<uint4*>(to + u.b) =
                make_uint4(pack_bf16(f[8], f[9]), pack_bf16(f[10], f[11]), pack_bf16(f[12], f[13]), pack_bf16(f[14], f[15]));
        }
        h += kAhead * step;
        if (h >= p.q_heads) break;
        read(h);
    }
}

// `team` threads (a power of two, a multiple of D / 16) take one block of one
// head, its keys and its values together: what leads to them (the sequence, then its
// page) is a chain of loads that costs more than the block.  The block's largest
// values come first, then its codes; where the block is more than one pass long its
// rows are read again (from L1 or L2) rather than held.
template <int D>
__device__ __forceinline__ void append_block(const AppendParams& p, long long unit, int at, int team) {
    constexpr int kUnits = D / 16;
    const bool live = unit < p.kv_units;
    const int h = live ? (int)(unit % p.c.num_heads) : 0;
    const long long rest = live ? unit / p.c.num_heads : 0;
    const int j = (int)(rest % p.blocks_per_seq), b = (int)(rest / p.blocks_per_seq);
    int lo = 0, hi = 0, blk = 0, first = 0, row0 = 0;
    if (live) {
        const SequenceView sv = sequence_view(p.s, b, p.c.page_size);
        first = sv.len - sv.n;                              // cache index of the first new token
        const int last = first + sv.n_work;                 // past the last one worked on
        const int begin = max(first, 0);
        row0 = sv.row0;
        blk = ((begin >> p.block_shift) + j) << p.block_shift;
        if (blk < last) {
            lo = max(blk, begin);
            hi = min(blk + p.c.block, last);
        }
    }
    int page = -1;
    if (hi > lo) page = p.s.block_table[(size_t)b * p.s.table_cols + (blk >> p.page_shift)];
    const RowUnit uk = row_unit(at % kUnits, p.rotary_dim), uv = row_unit(at % kUnits, 0);
    // a row's 16 keys of this thread, rotated, and its 16 values as they come (held in half the registers)
    auto load = [&](int index, float (&f)[16], uint4 (&raw)[2]) {
        const int t = row0 + index - first;
        const uint16_t* k = p.k + (size_t)t * p.k_stride + (size_t)h * D;
        const uint16_t* v = p.v + (size_t)t * p.v_stride + (size_t)h * D;
        const uint4 x0 = ldg128(k + uk.a), x1 = ldg128(k + uk.b);
        raw[0] = ldg128(v + uv.a);
        raw[1] = ldg128(v + uv.b);
        float c[8], s[8];
        if (uk.angle >= 0) load_angles(p, position_of(p, t, index), uk.angle, c, s);
        unpack8(x0, f);
        unpack8(x1, f + 8);
        if (uk.angle >= 0) rotate(f, c, s);
    };
    auto largest = [](const float* f, int n, float m) {       // of the finite ones
        for (int k = 0; k < n; ++k) {
            const float a = fabsf(f[k]);
            if (a <= 3.402823466e38f) m = fmaxf(m, a);
        }
        return m;
    };
    const int step = team / kUnits;
    float f[16], amax[2] = {0.f, 0.f};
    uint4 raw[2];
    for (int index = lo + at / kUnits; index < hi; index += step) {
        load(index, f, raw);
        amax[0] = largest(f, 16, amax[0]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float g[8];
            unpack8(raw[i], g);
            amax[1] = largest(g, 8, amax[1]);
        }
    }
    __shared__ float part[2][kAppendThreads / 32];
#pragma unroll
    for (int w = 0; w < 2; ++w)
        for (int o = min(team, 32) / 2; o; o >>= 1) amax[w] = fmaxf(amax[w], __shfl_xor_sync(~0u, amax[w], o));
    const bool found = (unsigned)page < (unsigned)p.c.num_pages;
    const int t0 = blk & (p.c.page_size - 1);
    const long long scale_at = found ? page * p.c.scale_page_stride + h * p.c.scale_head_stride + (t0 >> p.block_shift) : 0;
    const long long codes_at = found ? page * p.c.page_stride + h * p.c.head_stride + (long long)t0 * D : 0;
    const bool had = lo > blk;
    float s0[2] = {1.f, 1.f};
    if (found && had) {
        s0[0] = p.c.k_scale[scale_at];
        s0[1] = p.c.v_scale[scale_at];
    }
    if (team > 32) {
        const int warp = threadIdx.x >> 5, w0 = warp & ~(team / 32 - 1);
        if ((threadIdx.x & 31) == 0) {
            part[0][warp] = amax[0];
            part[1][warp] = amax[1];
        }
        __syncthreads();                    // and the old scales have been read by all
        for (int i = 0; i < team / 32; ++i) {
            amax[0] = fmaxf(amax[0], part[0][w0 + i]);
            amax[1] = fmaxf(amax[1], part[1][w0 + i]);
        }
    } else {
        __syncwarp();
    }
    if (hi <= lo || !found) return;
    const bool once = hi - lo <= step;          // the values of the first pass are still held
    float inv[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float s1 = block_scale(amax[w]);
        if (had && !(s0[w] < s1)) s1 = s0[w];
        inv[w] = __frcp_rn(s1);
        if (had && s1 != s0[w]) {
            uint8_t* codes = static_cast<uint8_t*>(w ? p.c.v : p.c.k) + codes_at;
            for (int e = at; e < (lo - blk) * D; e += team)
                codes[e] = (uint8_t)f32x2_to_e4m3x2(__fmul_rn(__fmul_rn(e4m3_value(codes[e]), s0[w]), inv[w]), 0.f);
        }
        if (at == 0) (w ? p.c.v_scale : p.c.k_scale)[scale_at] = s1;
    }
    for (int index = lo + at / kUnits; index < hi; index += step) {
        if (!once) load(index, f, raw);
        const size_t row = codes_at + (size_t)(index - blk) * D;
        auto code = [](const float* x, float inv) {           // four values
            return f32x2_to_e4m3x2(__fmul_rn(x[0], inv), __fmul_rn(x[1], inv)) |
                   f32x2_to_e4m3x2(__fmul_rn(x[2], inv), __fmul_rn(x[3], inv)) << 16;
        };
        uint8_t* k = static_cast<uint8_t*>(p.c.k) + row;
        *reinterpret_cast<uint2*>(k + uk.a) = make_uint2(code(f, inv[0]), code(f + 4, inv[0]));
        *reinterpret_cast<uint2*>(k + uk.b) = make_uint2(code(f + 8, inv[0]), code(f + 12, inv[0]));
        float g[8];
        unpack8(raw[0], g);
        const uint2 v0 = make_uint2(code(g, inv[1]), code(g + 4, inv[1]));
        unpack8(raw[1], g);
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.c.v) + row + uv.a) =
            make_uint4(v0.x, v0.y, code(g, inv[1]), code(g + 4, inv[1]));
    }
}

// grid.x: the CTAs of the blocks and those of the queries in turn, `period` apart
// the fewer ones: the blocks wait for their chains of loads while the queries stream.
template <int D>
__global__ void __launch_bounds__(kAppendThreads, 4) kv_append_kernel(const __grid_constant__ AppendParams p) {
    griddep_wait();
    griddep_launch_dependents();
    const int i = blockIdx.x, turn = i / p.period, fewer = min(p.kv_ctas, p.q_ctas);
    const bool of_fewer = i - turn * p.period == 0 && turn < fewer, kv_fewer = p.kv_ctas < p.q_ctas;
    const int index = of_fewer ? turn : i - min(turn + 1, fewer);
    if (of_fewer != kv_fewer) {
        append_queries<D>(p, index * p.per);
    } else {
        const int team = p.team, per = kAppendThreads / team;
        append_block<D>(p, (long long)index * per + threadIdx.x / team, threadIdx.x % team, team);
    }
}

template <int D>
cudaError_t launch_append(const AppendParams& p, unsigned grid, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kAppendThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_append_kernel<D>, p);
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
    p.rotary_dim = cos ? rotary_dim : 0;
    p.max_pos = cos ? max_pos : 1;
    p.q_heads = q_heads;
    p.page_shift = log2i(cache->page_size);
    p.block_shift = log2i(cache->block);
    p.s = Sequences{block_table, seq_lens, q_start, table_cols, batch, tokens, max_q};
    const long long most = max_q < tokens ? max_q : tokens;
    p.blocks_per_seq = (int)((most + cache->block - 2) / cache->block + 1);
    // threads of a block: one for each 16 of its values, as far as a CTA goes
    p.team = cache->block * D / 16 < kAppendThreads ? cache->block * D / 16 : kAppendThreads;
    p.kv_units = (long long)batch * p.blocks_per_seq * cache->num_heads;
    const int blocks = kAppendThreads / p.team;
    HostDevice dev;
    if ((s = host_device(dev)) != DL_OK) return s;
    // a CTA's search and position are shared by four tokens once that leaves several CTAs to each
    // SM (4 x 4096 tokens: 85 -> 78 us; at 48 x 6 tokens one is better: 6.1 -> 4.9 us)
    p.per = tokens >= 16 * dev.sm_count ? 4 : 1;
    const long long kv_ctas = (p.kv_units + blocks - 1) / blocks, q_ctas = q ? (tokens + p.per - 1) / p.per : 0;
    const long long grid = kv_ctas + q_ctas, fewer = kv_ctas < q_ctas ? kv_ctas : q_ctas;
    if (grid > 0x7fffffffLL)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "%lld blocks to write exceed one launch", p.kv_units);
    p.kv_ctas = (int)kv_ctas;
    p.q_ctas = (int)q_ctas;
    p.period = fewer ? (int)(grid / fewer) : 1;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = D == 128 ? launch_append<128>(p, (unsigned)grid, st) : launch_append<64>(p, (unsigned)grid, st);
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "kv_append launch: %s", cudaGetErrorString(e));
    return host_ok();
}
