// Low-rank adapters of many requests beside a shared projection (dl_linear_adapters).
#include <cooperative_groups.h>

#include "dl_device.cuh"
#include "dl_host.h"
#include "rows.cuh"

namespace dl {

constexpr int kMaxParts = 8, kMaxRank = 256;
constexpr int kTile = 16;                // tokens of a tile: all of one adapter
constexpr int kFewTokens = 256;          // up to here every CTA makes the list of tiles for itself
constexpr int kMaxAdapters = 16384;

struct AdapterParams {
    const uint16_t *a, *b;
    const float* scale;
    const int* ranks;
    int num, rank, K, N, parts;
    int part_end[kMaxParts];
    Rows x, base, y, y32;
    const int* index;
    int tokens;
    float* low;              // [tokens][parts * rank] scaled first products
    int* tiles;              // more than kFewTokens tokens: the list of tiles (else made by each CTA)
    bool in_place, in_place32;   // base is y, y32: rows without an adapter stay as they are
    bool wide;               // four consecutive columns of base, y and y32 are aligned to their size
};

// Tokens of one adapter, up to kTile of them; the others -1.
struct Tile {
    int adapter;             // -1: tokens without one
    int token[kTile];
};

// The tiles of at most kFewTokens tokens, made by the whole CTA from the tokens' adapters: a token's
// place among those of its adapter is the number of earlier ones, and every kTile-th opens a tile.
// Comparing all pairs takes 256 broadcast reads of shared memory a thread, less than the launch of a
// kernel that sorts.
struct FewTiles {
    int adapter[kFewTokens];
    int n;
    Tile tile[kFewTokens];
};

__device__ __forceinline__ int adapter_of(const AdapterParams& p, int t) {
    const int a = p.index[t];
    return a >= 0 && a < p.num ? a : -1;
}

__device__ __forceinline__ void make_tiles(const AdapterParams& p, FewTiles& s) {
    const int T = p.tokens;
    for (int t = threadIdx.x; t < T; t += blockDim.x) s.adapter[t] = adapter_of(p, t);
    __syncthreads();
    if (threadIdx.x < 32) {
        // tiles in the order of the tokens that open them, 32 tokens at a time
        int before = 0;
        for (int t0 = 0; t0 < T; t0 += 32) {
            const int t = t0 + threadIdx.x, mine = t < T ? s.adapter[t] : -2;
            int at = 0;
            if (t < T)
                for (int i = 0; i < t; ++i) at += s.adapter[i] == mine;
            const bool opens = t < T && at % kTile == 0;
            const unsigned m = __ballot_sync(~0u, opens);
            if (opens) {
                Tile& tile = s.tile[before + __popc(m & ((1u << threadIdx.x) - 1))];
                tile.adapter = mine;
                int k = 0;
                for (int i = t; i < T && k < kTile; ++i)
                    if (s.adapter[i] == mine) tile.token[k++] = i;
                for (; k < kTile; ++k) tile.token[k] = -1;
            }
            before += __popc(m);
        }
        if (threadIdx.x == 0) s.n = before;
    }
    __syncthreads();
}

// The list of tiles of many tokens, by one CTA: a counting sort by adapter.  Which tokens share a
// tile, and their order in it, do not change any result.
__global__ void __launch_bounds__(1024) sort_tokens_kernel(const __grid_constant__ AdapterParams p) {
    extern __shared__ int count[];       // of each adapter, then its first slot; the last: without one
    __shared__ int warp_sum[32], total;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    griddep_wait();
    griddep_launch_dependents();
    for (int i = tid; i <= p.num; i += 1024) count[i] = 0;
    if (tid == 0) total = 0;
    __syncthreads();
    for (int t0 = 0; t0 < p.tokens; t0 += 1024) {
        const int t = t0 + tid, a = t < p.tokens ? adapter_of(p, t) : -2, at = a == -1 ? p.num : a;
        const unsigned same = __match_any_sync(~0u, a);
        if (a != -2 && lane == __ffs(same) - 1) atomicAdd(&count[at], __popc(same));
    }
    __syncthreads();
    Tile* tiles = reinterpret_cast<Tile*>(p.tiles + 4);
    // slots of an adapter: its tokens, up to a whole number of tiles
    for (int i0 = 0; i0 <= p.num; i0 += 1024) {
        const int i = i0 + tid, n = i <= p.num ? count[i] : 0, mine = (n + kTile - 1) / kTile;
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(~0u, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        int first = total + inc - mine;
        for (int w = 0; w < warp; ++w) first += warp_sum[w];
        for (int j = 0; j < mine; ++j) {
            tiles[first + j].adapter = i < p.num ? i : -1;
            if (j == mine - 1)
                for (int k = n - j * kTile; k < kTile; ++k) tiles[first + j].token[k] = -1;
        }
        if (i <= p.num) count[i] = first * kTile;
        __syncthreads();
        if (tid == 1023) total = first + mine;
        __syncthreads();
    }
    for (int t0 = 0; t0 < p.tokens; t0 += 1024) {
        const int t = t0 + tid, a = t < p.tokens ? adapter_of(p, t) : -2, at = a == -1 ? p.num : a;
        const unsigned same = __match_any_sync(~0u, a);
        const int leader = __ffs(same) - 1;
        int slot = 0;
        if (a != -2 && lane == leader) slot = atomicAdd(&count[at], __popc(same));
        slot = __shfl_sync(~0u, slot, leader) + __popc(same & ((1u << lane) - 1));
        if (a != -2) tiles[slot / kTile].token[slot % kTile] = t;
    }
    if (tid == 0) p.tiles[0] = total;
}

// ---------------------------------------------------------------- first product

// low[t][j] = scale * sum_k A[j][k] x[t][k]: a cluster of CTAs shares K, a warp takes 16 rows of A and
// a tile's 16 tokens over its part of K.  A (and x) go from global memory straight into
// the operands of mma.m16n8k16: the sum over k may take its terms in any order, so a lane's
// 16-byte load of 8 consecutive k is the k-slots that it holds in two products.
constexpr int kLowThreads = 256, kLowWarps = kLowThreads / 32;
constexpr int kLowCluster = 8;

__global__ void __launch_bounds__(kLowThreads) adapters_low_kernel(const __grid_constant__ AdapterParams p) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float sum[kLowWarps][256];
    __shared__ float part[256];
    const int size = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    griddep_wait();
    griddep_launch_dependents();
    const Tile* tiles;
    int n_tiles;
    if (p.tokens <= kFewTokens) {
        FewTiles& s = *reinterpret_cast<FewTiles*>(smem);
        make_tiles(p, s);
        tiles = s.tile;
        n_tiles = s.n;
    } else {
        tiles = reinterpret_cast<const Tile*>(p.tiles + 4);
        n_tiles = p.tiles[0];
    }
    const int R = p.rank, groups = (R + 15) / 16, K = p.K;
    // this warp's part of K: whole runs of 32
    const int runs = (K + 31) / 32, workers = size * kLowWarps, worker = rank * kLowWarps + warp;
    const int k0 = (int)((long long)runs * worker / workers) * 32;
    const int k1 = (int)((long long)runs * (worker + 1) / workers) * 32;
    const long long items = (long long)n_tiles * p.parts * groups;
    for (long long item = blockIdx.x / size; item < items; item += gridDim.x / size) {
        const int j0 = (int)(item % groups) * 16, pt = (int)(item / groups) % p.parts;
        const Tile& tile = tiles[item / groups / p.parts];
        const int ad = tile.adapter;
        if (ad < 0) continue;
        const int r = p.ranks ? min(max(p.ranks[ad], 0), R) : R;
        if (j0 >= r) continue;
        const uint16_t* a = p.a + ((size_t)ad * p.parts + pt) * R * K + (size_t)j0 * K;
        const int t0 = tile.token[g], t1 = tile.token[g + 8];
        const bool two = tile.token[8] >= 0, row0 = j0 + g < r, row1 = j0 + g + 8 < r;
        const uint16_t* a0 = a + (size_t)g * K;
        const uint16_t* a1 = a0 + (size_t)8 * K;
        const char *x0 = row_ptr(p.x, max(t0, 0)), *x1 = row_ptr(p.x, max(t1, 0));
        float d0[4] = {}, d1[4] = {};
        const uint4 none = {0, 0, 0, 0};
#pragma unroll 4
        for (int run = k0; run < k1; run += 32) {       // every lane takes part in every product
            const int k = run + 8 * c;
            const bool in = k < K;
            const uint4 va = in && row0 ? ldg128(a0 + k) : none, vb = in && row1 ? ldg128(a1 + k) : none;
            const uint4 xa = in && t0 >= 0 ? ldg128(x0 + 2 * (size_t)k) : none;
            const uint4 xb = in && t1 >= 0 ? ldg128(x1 + 2 * (size_t)k) : none;
            mma_bf16_16816(d0, va.x, vb.x, va.y, vb.y, xa.x, xa.y);
            mma_bf16_16816(d0, va.z, vb.z, va.w, vb.w, xa.z, xa.w);
            if (two) {
                mma_bf16_16816(d1, va.x, vb.x, va.y, vb.y, xb.x, xb.y);
                mma_bf16_16816(d1, va.z, vb.z, va.w, vb.w, xb.z, xb.w);
            }
        }
        // sum[warp][token * 16 + row]
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int row = g + (i >= 2 ? 8 : 0), col = 2 * c + (i & 1);
            sum[warp][col * 16 + row] = d0[i];
            sum[warp][(col + 8) * 16 + row] = d1[i];
        }
        __syncthreads();
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kLowWarps; ++w) v += sum[w][tid];
        part[tid] = v;
        cluster.sync();
        // rank i finishes a share of the 256 sums
        const int each = 256 / size;
        if (tid < each) {
            const int at = rank * each + tid, t = tile.token[at / 16], j = j0 + at % 16;
            float all = 0.f;
            for (int q = 0; q < size; ++q) all += cluster.map_shared_rank(part, q)[at];
            if (t >= 0 && j < r)
                p.low[(size_t)t * p.parts * R + pt * R + j] = all * (p.scale ? p.scale[ad] : 1.f);
        }
        cluster.sync();
    }
}

// ---------------------------------------------------------------- second product

// out[t][n] = base[t][n] + sum_r low[t][r] B[n][r]: tokens are the rows of mma.m16n8k16, 16
// columns of a warp two products.  Which n is which product's column is chosen so that a lane's
// results are four consecutive columns; r is dealt to k-slots as k is above.
//
// The fp32 values of `low` go into the products as two bf16 parts (2^-18 of the value is lost), three
// (24 bits: nothing) where an fp32 result is asked for.  The parts of a value and their products can
// leave NaN where the value's own product is an infinity; what comes out NaN is summed again as it stands.
constexpr int kUpThreads = 128, kUpWarps = kUpThreads / 32;

struct Parts {
    uint32_t v[3];
};
// Two values as packed bf16 parts, each the next 8 bits of the value, rounded.
__device__ __forceinline__ Parts split(float a, float b, int parts) {
    Parts r = {};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        if (i < parts) {
            r.v[i] = f32x2_to_bf16x2(a, b);
            float ha, hb;
            bf16x2_to_f32(r.v[i], ha, hb);
            a -= ha;
            b -= hb;
            if (a != a) a = 0.f;        // an infinity or NaN is whole in its first part
            if (b != b) b = 0.f;
        }
    }
    return r;
}

__device__ __noinline__ float plain_up(const AdapterParams& p, int ad, int t, int pt, int n, int r) {
    const float* low = p.low + (size_t)t * p.parts * p.rank + pt * p.rank;
    const uint16_t* b = p.b + ((size_t)ad * p.N + n) * p.rank;
    float v = 0.f;
    for (int i = 0; i < r; ++i) v = fmaf(low[i], bf16_bits_to_f32(b[i]), v);
    return v;
}

__device__ __forceinline__ void load4(const Rows& m, int t, int n, int N, bool wide, float (&v)[4]) {
    const char* row = row_ptr(m, t);
    if (wide && n + 4 <= N) {
        if (m.f32) {
            const uint4 u = ldg128(row + 4 * (size_t)n);
            v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y); v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
        } else {
            const uint2 u = ldg64(row + 2 * (size_t)n);
            bf16x2_to_f32(u.x, v[0], v[1]);
            bf16x2_to_f32(u.y, v[2], v[3]);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = n + k < N ? row_load1(row, m.f32, n + k) : 0.f;
    }
}
__device__ __forceinline__ void put4(const Rows& m, int t, int n, int N, bool wide, const float (&v)[4]) {
    char* row = row_ptr(m, t);
    if (wide && n + 4 <= N) {
        if (m.f32)
            *reinterpret_cast<float4*>(row + 4 * (size_t)n) = make_float4(v[0], v[1], v[2], v[3]);
        else
            *reinterpret_cast<uint2*>(row + 2 * (size_t)n) = make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (n + k < N) row_store1(row, m.f32, n + k, v[k]);
    }
}

__global__ void __launch_bounds__(kUpThreads) adapters_up_kernel(const __grid_constant__ AdapterParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    griddep_wait();
    griddep_launch_dependents();
    const Tile* tiles;
    int n_tiles;
    if (p.tokens <= kFewTokens) {
        FewTiles& s = *reinterpret_cast<FewTiles*>(smem);
        make_tiles(p, s);
        tiles = s.tile;
        n_tiles = s.n;
    } else {
        tiles = reinterpret_cast<const Tile*>(p.tiles + 4);
        n_tiles = p.tiles[0];
    }
    const int R = p.rank, N = p.N, blocks = (N + 16 * kUpWarps - 1) / (16 * kUpWarps);
    const long long items = (long long)n_tiles * blocks;
    const int parts = p.y32.ptr ? 3 : 2;
    for (long long item = blockIdx.x; item < items; item += gridDim.x) {
        const Tile& tile = tiles[item / blocks];
        const int n0 = (int)(item % blocks) * 16 * kUpWarps + 16 * warp;
        if (n0 >= N) continue;
        const int ad = tile.adapter, t0 = tile.token[g], t1 = tile.token[g + 8], n = n0 + 4 * c;
        float d[2][4] = {};                  // [product][row g: 2 columns, row g + 8: 2 columns]
        float base0[4] = {}, base1[4] = {};
        if (p.base.ptr) {
            if (t0 >= 0) load4(p.base, t0, n, N, p.wide, base0);
            if (t1 >= 0) load4(p.base, t1, n, N, p.wide, base1);
        }
        int pt = 0;
        while (pt + 1 < p.parts && n0 >= p.part_end[pt]) ++pt;
        const int r = ad < 0 ? 0 : p.ranks ? min(max(p.ranks[ad], 0), R) : R;
        const float* low = p.low + pt * R;
        const size_t step = (size_t)p.parts * R;
        // column g of product i
        const int col0 = n0 + (g >> 1) * 4 + (g & 1), col1 = col0 + 2;
        const uint16_t* b0 = p.b + ((size_t)max(ad, 0) * N + min(col0, N - 1)) * R;
        const uint16_t* b1 = p.b + ((size_t)max(ad, 0) * N + min(col1, N - 1)) * R;
        for (int r0 = 0; r0 < r; r0 += 16) {
            const int at = r0 + 4 * c;
            uint2 w0 = {0, 0}, w1 = {0, 0};
            float4 s0 = {0.f, 0.f, 0.f, 0.f}, s1 = {0.f, 0.f, 0.f, 0.f};
            if (at < r) {
                if (col0 < N) w0 = ldg64(b0 + at);
                if (col1 < N) w1 = ldg64(b1 + at);
                if (t0 >= 0) s0 = ld_cg_f32x4(low + t0 * step + at);
                if (t1 >= 0) s1 = ld_cg_f32x4(low + t1 * step + at);
                if (at + 4 > r) {            // what lies past the rank is nobody's
                    const uint32_t m1 = at + 1 < r ? ~0u : 0xffffu, m2 = at + 2 < r ? ~0u : 0u;
                    w0.x &= m1; w1.x &= m1;
                    const uint32_t m3 = m2 & 0xffffu;     // at + 3 >= r here
                    w0.y &= m3; w1.y &= m3;
                    if (at + 1 >= r) s0.y = s1.y = 0.f;
                    if (at + 2 >= r) s0.z = s1.z = 0.f;
                    s0.w = s1.w = 0.f;
                }
            }
            const Parts a0 = split(s0.x, s0.y, parts), a1 = split(s1.x, s1.y, parts);
            const Parts a2 = split(s0.z, s0.w, parts), a3 = split(s1.z, s1.w, parts);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                if (i < parts) {
                    mma_bf16_16816(d[0], a0.v[i], a1.v[i], a2.v[i], a3.v[i], w0.x, w0.y);
                    mma_bf16_16816(d[1], a0.v[i], a1.v[i], a2.v[i], a3.v[i], w1.x, w1.y);
                }
            }
        }
        // columns n .. n + 3 of rows t0 and t1
        float v0[4] = {d[0][0], d[0][1], d[1][0], d[1][1]}, v1[4] = {d[0][2], d[0][3], d[1][2], d[1][3]};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (v0[k] != v0[k] && t0 >= 0 && n + k < N) v0[k] = plain_up(p, ad, t0, pt, n + k, r);
            if (v1[k] != v1[k] && t1 >= 0 && n + k < N) v1[k] = plain_up(p, ad, t1, pt, n + k, r);
            v0[k] += base0[k];
            v1[k] += base1[k];
        }
        const bool put = ad >= 0 || !p.in_place, put32 = p.y32.ptr && (ad >= 0 || !p.in_place32);
        if (t0 >= 0) {
            if (put) put4(p.y, t0, n, N, p.wide, v0);
            if (put32) put4(p.y32, t0, n, N, p.wide, v0);
        }
        if (t1 >= 0) {
            if (put) put4(p.y, t1, n, N, p.wide, v1);
            if (put32) put4(p.y32, t1, n, N, p.wide, v1);
        }
    }
}

// ---------------------------------------------------------------- host

static long long max_tiles(long long tokens, int num) {
    const long long kinds = tokens < num + 1 ? tokens : num + 1;
    return (tokens - kinds) / kTile + kinds + 1;
}

static size_t low_bytes(long long tokens, int rank, int parts) {
    return ((size_t)tokens * rank * parts * 4 + 255) / 256 * 256;
}

static size_t adapters_bytes(long long tokens, int num, int rank, int parts) {
    return DL_WORKSPACE_ZERO_BYTES + low_bytes(tokens, rank, parts) +
           (tokens > kFewTokens ? 16 + (size_t)max_tiles(tokens, num) * sizeof(Tile) : 0);
}

static dl_status check_adapters(const dl_adapters* a, AdapterParams& p) {
    if (!a) return host_fail(DL_ERR_INVALID_ARG, "adapters is NULL");
    if (a->num < 1 || a->num > kMaxAdapters)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "num=%d adapters are outside [1, %d]", a->num, kMaxAdapters);
    if (a->rank < 8 || a->rank > kMaxRank || a->rank % 8)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "rank=%d is not a multiple of 8 in [8, %d]", a->rank, kMaxRank);
    if (a->K < 8 || a->K % 8 || a->N < 1)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "K=%d must be a multiple of 8 and N=%d positive", a->K, a->N);
    if (a->parts < 1 || a->parts > kMaxParts)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "parts=%d is outside [1, %d]", a->parts, kMaxParts);
    int before = 0;
    for (int i = 0; i < a->parts; ++i) {
        const int end = a->part_end[i];
        if (end <= before || (i + 1 < a->parts ? end % 16 != 0 || end >= a->N : end != a->N))
            return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "part_end must rise in multiples of 16 up to N=%d", a->N);
        before = p.part_end[i] = end;
    }
    if (!a->a || !a->b) return host_fail(DL_ERR_INVALID_ARG, "a or b is NULL");
    if (((uintptr_t)a->a | (uintptr_t)a->b) & 15) return host_fail(DL_ERR_MISALIGNED, "a and b must be 16-byte aligned");
    if (((uintptr_t)a->scale | (uintptr_t)a->ranks) & 3)
        return host_fail(DL_ERR_MISALIGNED, "scale and ranks must be 4-byte aligned");
    p.a = static_cast<const uint16_t*>(a->a);
    p.b = static_cast<const uint16_t*>(a->b);
    p.scale = a->scale;
    p.ranks = a->ranks;
    p.num = a->num;
    p.rank = a->rank;
    p.K = a->K;
    p.N = a->N;
    p.parts = a->parts;
    return DL_OK;
}

static cudaError_t launch_low(const AdapterParams& p, long long items, int sm_count, size_t smem, cudaStream_t stream) {
    const long long most = 2LL * sm_count / kLowCluster * 2;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kLowCluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((items < most ? items : most) * kLowCluster));
    cfg.blockDim = dim3(kLowThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, adapters_low_kernel, p);
}

}  // namespace dl

extern "C" size_t dl_adapters_workspace_bytes(int tokens, int num, int rank, int parts) {
    if (tokens < 0 || num < 1 || num > dl::kMaxAdapters || rank < 8 || rank > dl::kMaxRank || rank % 8 || parts < 1 ||
        parts > dl::kMaxParts)
        return 0;
    return dl::adapters_bytes(tokens, num, rank, parts);
}

extern "C" dl_status dl_linear_adapters(const dl_adapters* adapters, const dl_rows* x, const int* index, const dl_rows* base,
                                        const dl_rows* y, const dl_rows* y_f32, int tokens, void* workspace,
                                        size_t ws_bytes, void* stream) {
    using namespace dl;
    AdapterParams p = {};
    dl_status s = check_adapters(adapters, p);
    if (s != DL_OK) return s;
    if (tokens < 0) return host_fail(DL_ERR_INVALID_ARG, "tokens=%d must be >= 0", tokens);
    if (tokens == 0) return host_ok();
    const int K = p.K, N = p.N;
    if (!x || !x->data || !index || !y || !y->data) return host_fail(DL_ERR_INVALID_ARG, "x, index or y is NULL");
    if (x->dtype != DL_ROWS_BF16) return host_fail(DL_ERR_INVALID_ARG, "x must be bf16");
    if (y->dtype != DL_ROWS_BF16) return host_fail(DL_ERR_INVALID_ARG, "y must be bf16");
    if (y_f32 && y_f32->data && y_f32->dtype != DL_ROWS_F32) return host_fail(DL_ERR_INVALID_ARG, "y_f32 must be fp32");
    if ((s = check_rows(x, "x", tokens, K, p.x)) != DL_OK || (s = check_rows(base, "base", tokens, N, p.base)) != DL_OK ||
        (s = check_rows(y, "y", tokens, N, p.y)) != DL_OK || (s = check_rows(y_f32, "y_f32", tokens, N, p.y32)) != DL_OK)
        return s;
    if (!rows_aligned16(p.x, tokens)) return host_fail(DL_ERR_MISALIGNED, "x's rows must be 16-byte aligned");
    if ((uintptr_t)index & 3) return host_fail(DL_ERR_MISALIGNED, "index must be 4-byte aligned");
    for (const Rows* out : {&p.y, &p.y32}) {
        const char* name = out == &p.y ? "y" : "y_f32";
        if (!same_rows(*out, p.base) && rows_meet(*out, tokens, N, p.base, tokens, N))
            return host_fail(DL_ERR_INVALID_ARG, "%s overlaps base in another layout", name);
        if (rows_meet(*out, tokens, N, p.x, tokens, K)) return host_fail(DL_ERR_INVALID_ARG, "%s overlaps x", name);
    }
    if (rows_meet(p.y, tokens, N, p.y32, tokens, N)) return host_fail(DL_ERR_INVALID_ARG, "y and y_f32 overlap");
    if (!workspace) return host_fail(DL_ERR_WORKSPACE, "workspace is NULL");
    if ((uintptr_t)workspace & 255) return host_fail(DL_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    const size_t need = adapters_bytes(tokens, p.num, p.rank, p.parts);
    if (ws_bytes < need) return host_fail(DL_ERR_WORKSPACE, "workspace has %zu bytes, %zu are needed", ws_bytes, need);
    char* scratch = static_cast<char*>(workspace) + DL_WORKSPACE_ZERO_BYTES;
    p.low = reinterpret_cast<float*>(scratch);
    p.tiles = reinterpret_cast<int*>(scratch + low_bytes(tokens, p.rank, p.parts));
    p.index = index;
    p.tokens = tokens;
    p.in_place = same_rows(p.y, p.base);
    p.in_place32 = p.y32.ptr && same_rows(p.y32, p.base);
    p.wide = true;
    for (const Rows* r : {&p.base, &p.y, &p.y32})
        if (r->ptr) p.wide = p.wide && !(((uintptr_t)r->ptr | (uintptr_t)r->stride) & (r->f32 ? 15 : 7));
    HostDevice dev;
    if ((s = host_device(dev)) != DL_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const long long tiles = max_tiles(tokens, p.num), groups = (p.rank + 15) / 16;
    const size_t smem = tokens <= kFewTokens ? sizeof(FewTiles) : 0;
    cudaError_t e = cudaSuccess;
    if (tokens > kFewTokens) {
        const size_t counters = (size_t)(p.num + 1) * 4;
        if (counters > 48 * 1024)
            e = cudaFuncSetAttribute(sort_tokens_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)counters);
        if (e == cudaSuccess) e = launch_dependent(sort_tokens_kernel, dim3(1), dim3(1024), counters, st, p);
    }
    if (e == cudaSuccess) e = launch_low(p, tiles * p.parts * groups, dev.sm_count, smem, st);
    if (e == cudaSuccess) {
        const long long items = tiles * ((N + 16 * kUpWarps - 1) / (16 * kUpWarps)), most = 16LL * dev.sm_count;
        e = launch_dependent(adapters_up_kernel, dim3((unsigned)(items < most ? items : most)), dim3(kUpThreads), smem, st, p);
    }
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "linear_adapters launch: %s", cudaGetErrorString(e));
    return host_ok();
}
