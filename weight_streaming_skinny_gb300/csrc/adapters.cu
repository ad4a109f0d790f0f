// Low-rank adapters of many requests beside a shared projection (dl_linear_adapters).
#include <cooperative_groups.h>

#include <atomic>

#include "dl_device.cuh"
#include "dl_host.h"
#include "rows.cuh"

namespace dl {

constexpr int kMaxParts = 8, kMaxRank = 256, kMaxAdapters = 16384;
constexpr int kTile = 16;                // tokens of a small tile: all of one adapter
constexpr int kFewTokens = 256;          // up to here every CTA makes the list of tiles for itself
constexpr int kBigTile = 128;            // tokens of a big tile
constexpr int kBigFrom = 64;             // tokens of an adapter from which on they go in big tiles
constexpr int kBigRank = 128;            // the largest rank whose second factor fits beside the big tiles' first one
constexpr int kMaxSplits = 8;            // CTAs that share K of a big tile

struct AdapterParams {
    const uint16_t *a, *b;
    const float* scale;
    const int* ranks;
    int num, rank, K, N, parts;
    int part_end[kMaxParts];
    Rows x, base, y, y32;
    const int* index;
    int tokens;
    float* low;              // [tokens][parts * rank] scaled first products (small tiles)
    int* tiles;              // more than kFewTokens tokens: what sort_tokens_kernel writes
    int big_from;            // kBigFrom, or none if ranks are too large
    bool in_place, in_place32;   // base is y, y32: rows without an adapter stay as they are
    bool wide;               // four consecutive columns of base, y and y32 are aligned to their size
    // big tiles
    float* low_big;          // [tokens][parts * rank], by place in `order`, without scale
    WaitCtl wait;
};

// Tokens of one adapter, up to kTile of them; the others -1.
struct Tile {
    int adapter;             // -1: tokens without one
    int token[kTile];
};
// Tokens order[first .. first + count) of one adapter.
struct BigTile {
    int adapter, first, count, unused;
};

// The lists of more than kFewTokens tokens.
struct Lists {
    int *counts;             // small tiles, big tiles
    int* order;              // [tokens] the big tiles' tokens
    BigTile* big;
    Tile* small;
};
__host__ __device__ inline long long max_big(long long tokens, int num) {
    return tokens / kBigTile + (tokens / kBigFrom < num + 1 ? tokens / kBigFrom : num + 1) + 1;
}
__host__ __device__ inline long long max_small(long long tokens, int num) {
    return tokens / kTile + (tokens < num + 1 ? tokens : num + 1) + 1;
}
__host__ __device__ inline Lists lists_of(int* at, long long tokens, int num) {
    Lists l;
    l.counts = at;
    l.big = reinterpret_cast<BigTile*>(at + 4);
    l.order = reinterpret_cast<int*>(l.big + max_big(tokens, num));
    l.small = reinterpret_cast<Tile*>(l.order + tokens);
    return l;
}

__device__ __forceinline__ int adapter_of(const AdapterParams& p, int t) {
    const int a = p.index[t];
    return a >= 0 && a < p.num ? a : -1;
}
__device__ __forceinline__ int rank_of(const AdapterParams& p, int adapter) {
    return adapter < 0 ? 0 : p.ranks ? min(max(p.ranks[adapter], 0), p.rank) : p.rank;
}

// The small tiles of at most kFewTokens tokens, made by every CTA for itself, all alike.  A token's place
// among those of its adapter is the number of earlier ones; every kTile-th opens a tile, and tiles are numbered
// by the tokens that open them.  Up to 32 tokens one warp sees all; beyond, a table of the adapters that
// occur, by hash, holds how many tokens of it each warp has.  (Where in the table an adapter is does
// not matter.)
constexpr int kSlots = 512;
struct FewTiles {
    Tile tile[kFewTokens];
    int slot[kSlots];                            // adapter + 2 of each slot, 0: free
    unsigned long long held[kSlots];             // its tokens in each warp, a byte each (32 at most)
    unsigned char number[kSlots][kFewTokens / kTile];   // of its tiles
    int opened[kFewTokens / 32];
    int n;
};

__device__ __forceinline__ int nth_bit(unsigned m, int n) {
    for (; n > 0; --n) m &= m - 1;
    return __ffs(m) - 1;
}

__device__ __forceinline__ int make_tiles(const AdapterParams& p, FewTiles& s) {
    static_assert(kFewTokens == 256, "a byte for each of 8 warps");
    const int T = p.tokens, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const unsigned below = (1u << lane) - 1;
    const int mine = t < T ? adapter_of(p, t) : -2;
    for (int i = t; i < T * (int)(sizeof(Tile) / 4); i += blockDim.x) reinterpret_cast<int*>(s.tile)[i] = -1;
    if (T <= 32) {
        __syncthreads();
        if (warp == 0) {
            const unsigned same = __match_any_sync(~0u, mine);
            const int place = __popc(same & below);
            const unsigned m = __ballot_sync(~0u, t < T && place % kTile == 0);
            if (t < T) {
                const int opener = nth_bit(same, place / kTile * kTile);
                Tile& tile = s.tile[__popc(m & ((1u << opener) - 1))];
                if (opener == t) tile.adapter = mine;
                tile.token[place % kTile] = t;
            }
            if (lane == 0) s.n = __popc(m);
        }
        __syncthreads();
        return s.n;
    }
    for (int i = t; i < kSlots; i += blockDim.x) {
        s.slot[i] = 0;
        s.held[i] = 0;
    }
    __syncthreads();
    unsigned same = 0;
    int at = 0, place = 0;
    bool opens = false;
    if (t < kFewTokens) {
        same = __match_any_sync(~0u, mine);
        const int leader = __ffs(same) - 1;
        if (t < T && lane == leader) {
            at = (mine * 0x9E3779B1u) >> 23;     // 9 bits
            while (true) {
                const int found = atomicCAS(&s.slot[at], 0, mine + 2);
                if (found == 0 || found == mine + 2) break;
                at = (at + 1) % kSlots;
            }
            reinterpret_cast<unsigned char*>(&s.held[at])[warp] = (unsigned char)__popc(same);
        }
        at = __shfl_sync(~0u, at, leader);
    }
    __syncthreads();
    if (t < kFewTokens) {
        // the bytes of the warps before this one
        const unsigned long long before = s.held[at] & ((1ull << (8 * warp)) - 1);
        place = __dp4a((unsigned)before, 0x01010101u, __dp4a((unsigned)(before >> 32), 0x01010101u, 0u)) + __popc(same & below);
        opens = t < T && place % kTile == 0;
        const unsigned m = __ballot_sync(~0u, opens);
        if (lane == 0) s.opened[warp] = __popc(m);
        same = m;                                // openers of this warp
    }
    __syncthreads();
    int n = 0, first = 0;
#pragma unroll
    for (int w = 0; w < kFewTokens / 32; ++w) {
        if (w < warp) first += s.opened[w];
        n += s.opened[w];
    }
    if (opens) {
        const int number = first + __popc(same & below);
        s.number[at][place / kTile] = (unsigned char)number;
        s.tile[number].adapter = mine;
    }
    __syncthreads();
    if (t < T) s.tile[s.number[at][place / kTile]].token[place % kTile] = t;
    __syncthreads();
    return n;
}

// The lists of many tokens, by one CTA: a counting sort by adapter.  Which tokens of an adapter share a
// tile, and their order in it, do not change any result.
__global__ void __launch_bounds__(1024) sort_tokens_kernel(const __grid_constant__ AdapterParams p) {
    extern __shared__ unsigned count[];  // of each adapter, then its next place; the last: without one
    __shared__ int warp_sum[3][32];
    constexpr unsigned kBig = 1u << 31;  // a place in `order`, not in the small tiles
    constexpr int kEach = 4;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Lists l = lists_of(p.tiles, p.tokens, p.num);
    griddep_wait();
    griddep_launch_dependents();
    for (int i = tid; i <= p.num; i += 1024) count[i] = 0;
    __syncthreads();
    for (long long t0 = 0; t0 < p.tokens; t0 += 1024 * kEach) {
        int a[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const long long t = t0 + 1024 * k + tid;
            a[k] = t < p.tokens ? adapter_of(p, (int)t) : -2;
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const unsigned same = __match_any_sync(~0u, a[k]);
            if (a[k] != -2 && lane == __ffs(same) - 1) atomicAdd(&count[a[k] < 0 ? p.num : a[k]], __popc(same));
        }
    }
    __syncthreads();
    int total[3] = {0, 0, 0};            // small tiles, big tiles, tokens of big tiles
    for (int i0 = 0; i0 <= p.num; i0 += 1024) {
        const int i = i0 + tid, n = i <= p.num ? (int)count[i] : 0;
        const bool big = n >= p.big_from;
        const int mine[3] = {big ? 0 : (n + kTile - 1) / kTile, big ? (n + kBigTile - 1) / kBigTile : 0, big ? n : 0};
        int inc[3] = {mine[0], mine[1], mine[2]};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                const int v = __shfl_up_sync(~0u, inc[j], o);
                if (lane >= o) inc[j] += v;
            }
        __syncthreads();
        if (lane == 31)
            for (int j = 0; j < 3; ++j) warp_sum[j][warp] = inc[j];
        __syncthreads();
        int first[3];
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            first[j] = total[j] + inc[j] - mine[j];
            for (int w = 0; w < 32; ++w) {
                if (w < warp) first[j] += warp_sum[j][w];
                total[j] += warp_sum[j][w];
            }
        }
        const int ad = i < p.num ? i : -1;
        for (int j = 0; j < mine[0]; ++j) {
            Tile& tile = l.small[first[0] + j];
            tile.adapter = ad;
            for (int k = min(n - j * kTile, kTile); k < kTile; ++k) tile.token[k] = -1;
        }
        for (int j = 0; j < mine[1]; ++j)
            l.big[first[1] + j] = BigTile{ad, first[2] + j * kBigTile, min(n - j * kBigTile, kBigTile), 0};
        if (i <= p.num) count[i] = big ? kBig | (unsigned)first[2] : (unsigned)first[0] * kTile;
    }
    __syncthreads();
    for (long long t0 = 0; t0 < p.tokens; t0 += 1024 * kEach) {
        int a[kEach];
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const long long t = t0 + 1024 * k + tid;
            a[k] = t < p.tokens ? adapter_of(p, (int)t) : -2;
        }
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const unsigned same = __match_any_sync(~0u, a[k]);
            const int leader = __ffs(same) - 1;
            unsigned at = 0;
            if (a[k] != -2 && lane == leader) at = atomicAdd(&count[a[k] < 0 ? p.num : a[k]], __popc(same));
            at = __shfl_sync(~0u, at, leader) + __popc(same & ((1u << lane) - 1));
            const int t = (int)(t0 + 1024 * k + tid);
            if (a[k] == -2) continue;
            if (at & kBig)
                l.order[at & ~kBig] = t;
            else
                l.small[at / kTile].token[at % kTile] = t;
        }
    }
    if (tid == 0) {
        l.counts[0] = total[0];
        l.counts[1] = total[1];
    }
}

// ---------------------------------------------------------------- small tiles: first product

// low[t][j] = scale * sum_k A[j][k] x[t][k]: a cluster of CTAs shares K, a warp takes 16 rows of A and
// a tile's 16 tokens over its part of K.  A (and x) go from global memory straight into
// the operands of mma.m16n8k16: the sum over k may take its terms in any order, so a lane's
// 16-byte load of 8 consecutive k is the k-slots that it holds in two products.
constexpr int kLowThreads = 256, kLowWarps = kLowThreads / 32;
constexpr int kLowCluster = 8;

template <bool FEW>
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
    if (FEW) {
        FewTiles& s = *reinterpret_cast<FewTiles*>(smem);
        n_tiles = make_tiles(p, s);
        tiles = s.tile;
    } else {
        const Lists l = lists_of(p.tiles, p.tokens, p.num);
        n_tiles = l.counts[0];
        tiles = l.small;
    }
    const int R = p.rank, K = p.K;
    const unsigned groups = (R + 15) / 16;
    // this warp's part of K: whole runs of 32
    const int runs = (K + 31) / 32, workers = size * kLowWarps, worker = rank * kLowWarps + warp;
    const int k0 = (int)((long long)runs * worker / workers) * 32;
    const int k1 = (int)((long long)runs * (worker + 1) / workers) * 32;
    const unsigned per = p.parts * groups, items = n_tiles * per;      // fits: a launch of more is refused
    for (unsigned item = blockIdx.x / size; item < items; item += gridDim.x / size) {
        const unsigned i = item % per;
        const int j0 = (int)(i % groups) * 16, pt = (int)(i / groups);
        const Tile& tile = tiles[item / per];
        const int ad = tile.adapter;
        if (ad < 0) continue;
        const int r = rank_of(p, ad);
        if (j0 >= r) continue;
        const int t0 = tile.token[g], t1 = tile.token[g + 8];
        const bool two = tile.token[8] >= 0, row0 = j0 + g < r, row1 = j0 + g + 8 < r;
        const uint16_t* a0 = p.a + (((size_t)ad * p.parts + pt) * R + j0 + g) * K + 8 * c;
        const uint16_t* a1 = a0 + (size_t)8 * K;
        const char *x0 = row_ptr(p.x, max(t0, 0)) + 16 * c, *x1 = row_ptr(p.x, max(t1, 0)) + 16 * c;
        float d0[4] = {}, d1[4] = {};
        const uint4 none = {0, 0, 0, 0};
        auto step = [&](int run, bool in) {              // every lane takes part in every product
            const uint4 va = in && row0 ? ldg128(a0 + run) : none, vb = in && row1 ? ldg128(a1 + run) : none;
            const uint4 xa = in && t0 >= 0 ? ldg128(x0 + 2 * run) : none;
            mma_bf16_16816(d0, va.x, vb.x, va.y, vb.y, xa.x, xa.y);
            mma_bf16_16816(d0, va.z, vb.z, va.w, vb.w, xa.z, xa.w);
            if (two) {
                const uint4 xb = in && t1 >= 0 ? ldg128(x1 + 2 * run) : none;
                mma_bf16_16816(d1, va.x, vb.x, va.y, vb.y, xb.x, xb.y);
                mma_bf16_16816(d1, va.z, vb.z, va.w, vb.w, xb.z, xb.w);
            }
        };
        int run = k0;
        for (; run + 128 <= k1 && run + 128 <= K; run += 128) {
            uint4 va[4], vb[4], xa[4], xb[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                va[i] = row0 ? ldg128(a0 + run + 32 * i) : none;
                vb[i] = row1 ? ldg128(a1 + run + 32 * i) : none;
                xa[i] = t0 >= 0 ? ldg128(x0 + 2 * (run + 32 * i)) : none;
                xb[i] = t1 >= 0 ? ldg128(x1 + 2 * (run + 32 * i)) : none;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mma_bf16_16816(d0, va[i].x, vb[i].x, va[i].y, vb[i].y, xa[i].x, xa[i].y);
                mma_bf16_16816(d0, va[i].z, vb[i].z, va[i].w, vb[i].w, xa[i].z, xa[i].w);
                if (two) {
                    mma_bf16_16816(d1, va[i].x, vb[i].x, va[i].y, vb[i].y, xb[i].x, xb[i].y);
                    mma_bf16_16816(d1, va[i].z, vb[i].z, va[i].w, vb[i].w, xb[i].z, xb[i].w);
                }
            }
        }
        for (; run < k1; run += 32) step(run, run + 8 * c < K);
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
#pragma unroll
            for (int q = 0; q < kLowCluster; ++q)
                if (q < size) all += cluster.map_shared_rank(part, q)[at];
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

__device__ __forceinline__ int part_of(const AdapterParams& p, int n) {
    int pt = 0;
    while (pt + 1 < p.parts && n >= p.part_end[pt]) ++pt;
    return pt;
}

// Sums of four columns from n on that came out NaN, as they stand; low: the token's first products, times
// scale.
__device__ __noinline__ void plain_up(const AdapterParams& p, const float* low, float scale, const uint16_t* b, int n, int r,
                                      float (&v)[4]) {
    for (int k = 0; k < 4; ++k) {
        if (v[k] == v[k] || n + k >= p.N) continue;
        const float* s = low + part_of(p, n + k) * p.rank;
        v[k] = 0.f;
        for (int i = 0; i < r; ++i) v[k] = fmaf(s[i] * scale, bf16_bits_to_f32(b[(size_t)(n + k) * p.rank + i]), v[k]);
    }
}

// The bits of four values of r from `at` on that lie within the rank; what lies past it is nobody's.
__device__ __forceinline__ uint2 rank_mask(int at, int r) {
    return make_uint2((at < r ? 0xffffu : 0u) | (at + 1 < r ? 0xffff0000u : 0u),
                      (at + 2 < r ? 0xffffu : 0u) | (at + 3 < r ? 0xffff0000u : 0u));
}

// A token's results in one tensor: 16 columns of a warp's, four of them this lane's, from n on.
__device__ __forceinline__ void put_wide(char* row, bool f32, int n, const float (&v)[4]) {
    if (f32)
        *reinterpret_cast<float4*>(row + 4 * (size_t)n) = make_float4(v[0], v[1], v[2], v[3]);
    else
        *reinterpret_cast<uint2*>(row + 2 * (size_t)n) = make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void load_wide(const char* row, bool f32, int n, float (&v)[4]) {
    if (f32) {
        const uint4 u = ldg128(row + 4 * (size_t)n);
        v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y); v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
    } else {
        const uint2 u = ldg64(row + 2 * (size_t)n);
        bf16x2_to_f32(u.x, v[0], v[1]);
        bf16x2_to_f32(u.y, v[2], v[3]);
    }
}

// Small tiles: a warp takes U times 16 columns of a tile, B's values of 16 C at a time.  What does not depend
// on the first products (the tiles, base, B) is fetched before they are waited for: the kernel that
// makes them lets this one start only after it had waited for all earlier ones.
constexpr int kUpThreads = 256, kUpWarps = kUpThreads / 32;

template <bool FEW, int U, int C>
__global__ void __launch_bounds__(kUpThreads, 2) adapters_up_kernel(const __grid_constant__ AdapterParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const Tile* tiles;
    int n_tiles;
    if (FEW) {
        FewTiles& s = *reinterpret_cast<FewTiles*>(smem);
        n_tiles = make_tiles(p, s);
        tiles = s.tile;
    } else {
        const Lists l = lists_of(p.tiles, p.tokens, p.num);
        n_tiles = l.counts[0];
        tiles = l.small;
    }
    const int R = p.rank, N = p.N, parts = p.y32.ptr ? 3 : 2;
    const unsigned units = (N + 16 * U - 1) / (16 * U), items = n_tiles * units;    // fits: a launch of more is refused
    const size_t step = (size_t)p.parts * R;
    bool waited = false;
    for (unsigned item = blockIdx.x * kUpWarps + warp; item < items; item += gridDim.x * kUpWarps) {
        const Tile& tile = tiles[item / units];
        const int n0 = (int)(item % units) * 16 * U;
        const int ad = tile.adapter, t0 = tile.token[g], t1 = tile.token[g + 8];
        const int r = rank_of(p, ad);
        const bool whole = n0 + 16 * U <= N, fast = whole && p.wide;
        const uint16_t* b = p.b + (size_t)max(ad, 0) * N * R;
        float base[U][2][4];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) base[u][0][k] = base[u][1][k] = 0.f;
        if (p.base.ptr) {
            const char *from0 = row_ptr(p.base, max(t0, 0)), *from1 = row_ptr(p.base, max(t1, 0));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int n = n0 + 16 * u + 4 * c;
                if (fast) {
                    if (t0 >= 0) load_wide(from0, p.base.f32, n, base[u][0]);
                    if (t1 >= 0) load_wide(from1, p.base.f32, n, base[u][1]);
                } else {
                    if (t0 >= 0) load4(p.base, t0, n, N, p.wide, base[u][0]);
                    if (t1 >= 0) load4(p.base, t1, n, N, p.wide, base[u][1]);
                }
            }
        }
        float d[U][2][4] = {};               // [product][row g: 2 columns, row g + 8: 2 columns]
        const int col0 = n0 + (g >> 1) * 4 + (g & 1);
        for (int r0 = 0; r0 < r; r0 += 16 * C) {
            uint2 w[C][U][2];
            const uint16_t* bl = b + (size_t)col0 * R + r0 + 4 * c;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int q = 0; q < C; ++q) {
                        const bool in = r0 + 16 * q + 4 * c < r && (whole || col0 + 16 * u + 2 * i < N);
                        w[q][u][i] = in ? ldg64(bl + (16 * u + 2 * i) * R + 16 * q) : make_uint2(0, 0);
                    }
            if (!waited) {
                griddep_wait();
                griddep_launch_dependents();
                waited = true;
            }
            int held = -1;                   // the part whose first products `a` has
            Parts a[C][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int pt = part_of(p, n0 + 16 * u);
                if (pt != held) {
                    held = pt;
                    const float *low0 = p.low + t0 * step + pt * R + r0 + 4 * c, *low1 = p.low + t1 * step + pt * R + r0 + 4 * c;
                    float4 s0[C], s1[C];
#pragma unroll
                    for (int q = 0; q < C; ++q) {
                        const bool in = r0 + 16 * q + 4 * c < r;
                        s0[q] = in && t0 >= 0 ? ld_cg_f32x4(low0 + 16 * q) : make_float4(0.f, 0.f, 0.f, 0.f);
                        s1[q] = in && t1 >= 0 ? ld_cg_f32x4(low1 + 16 * q) : make_float4(0.f, 0.f, 0.f, 0.f);
                    }
#pragma unroll
                    for (int q = 0; q < C; ++q) {
                        const int at = r0 + 16 * q + 4 * c;
                        const bool in1 = at + 1 < r, in2 = at + 2 < r, in3 = at + 3 < r;
                        a[q][0] = split(s0[q].x, in1 ? s0[q].y : 0.f, parts);
                        a[q][1] = split(s1[q].x, in1 ? s1[q].y : 0.f, parts);
                        a[q][2] = split(in2 ? s0[q].z : 0.f, in3 ? s0[q].w : 0.f, parts);
                        a[q][3] = split(in2 ? s1[q].z : 0.f, in3 ? s1[q].w : 0.f, parts);
                    }
                }
#pragma unroll
                for (int q = 0; q < C; ++q) {
                    const int at = r0 + 16 * q + 4 * c;
                    if (r0 + 16 * q >= r) break;
                    const uint2 m = rank_mask(at, r);
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        if (i < parts) {
                            mma_bf16_16816(d[u][0], a[q][0].v[i], a[q][1].v[i], a[q][2].v[i], a[q][3].v[i], w[q][u][0].x & m.x,
                                           w[q][u][0].y & m.y);
                            mma_bf16_16816(d[u][1], a[q][0].v[i], a[q][1].v[i], a[q][2].v[i], a[q][3].v[i], w[q][u][1].x & m.x,
                                           w[q][u][1].y & m.y);
                        }
                    }
                }
            }
        }
        if (!waited) {                       // (no earlier kernel still reads or writes y)
            griddep_wait();
            griddep_launch_dependents();
            waited = true;
        }
        float odd = 0.f;                     // NaN if any sum is, or infinite
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int k = 0; k < 4; ++k) odd = fmaf(d[u][0][k], 0.f, fmaf(d[u][1][k], 0.f, odd));
        const bool put = ad >= 0 || !p.in_place, put32 = p.y32.ptr && (ad >= 0 || !p.in_place32);
#pragma unroll
        for (int h = 0; h < 2; ++h) {        // rows t0 and t1
            const int t = h ? t1 : t0;
            if (t < 0) continue;
            char *to = row_ptr(p.y, t), *to32 = row_ptr(p.y32, t);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int n = n0 + 16 * u + 4 * c;
                float v[4] = {d[u][0][2 * h], d[u][0][2 * h + 1], d[u][1][2 * h], d[u][1][2 * h + 1]};
                if (odd != odd) plain_up(p, p.low + t * step, 1.f, b, n, r, v);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] += base[u][h][k];
                if (fast) {
                    if (put) put_wide(to, false, n, v);
                    if (put32) put_wide(to32, true, n, v);
                } else {
                    if (put) put4(p.y, t, n, N, p.wide, v);
                    if (put32) put4(p.y32, t, n, N, p.wide, v);
                }
            }
        }
    }
    if (!waited) griddep_wait();
}

// ---------------------------------------------------------------- big tiles

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One K step of 16 of two bf16 operands: kind::f16, fp32 accumulator, 128 rows, n columns.
__host__ __device__ constexpr uint32_t umma_idesc_bf16(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void umma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// First product of big tiles: low_big[place][j] = sum_k A[j][k] x[token][k], a product of 128 tokens
// and up to 256 rows of A on the tensor cores, the sums in tensor memory.  It is bound by the read of x;
// all threads gather its rows (and A's) into 128-byte swizzled stages of 64 k, several ahead, and one
// thread issues the products.  A cluster shares K: each CTA leaves its sums in its shared memory,
// where the cluster's CTAs add them up, a share of the tokens each, always in the same order.
constexpr int kBigThreads = 256;
constexpr int kBigStages = 4;
constexpr int kBigCols = 256;            // rows of A of one CTA, at most

struct BigSmem {
    int cols, stage, total;              // columns of the accumulator, bytes of a stage, and of all
};
__host__ __device__ inline BigSmem big_smem(int columns) {
    BigSmem s;
    s.cols = (columns < kBigCols ? columns + 15 : kBigCols) / 16 * 16;
    s.stage = (kBigTile + s.cols) * 128;     // four of them hold the sums, 128 x (cols + 4) x 4 bytes, too
    s.total = 1024 + kBigStages * s.stage + 256;
    return s;
}

__global__ void __launch_bounds__(kBigThreads) adapters_low_big_kernel(const __grid_constant__ AdapterParams p) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ __align__(16) unsigned char raw[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int splits = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const Lists l = lists_of(p.tiles, p.tokens, p.num);
    const int SR = p.parts * p.rank, K = p.K;
    const BigSmem shape = big_smem(SR);
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u, bars = base + kBigStages * shape.stage;
    const uint32_t slot = bars + 8 * kBigStages;
    // The lists are complete and the buffers free: the kernel before this one let it start only after
    // it had waited for sort_tokens_kernel.  (Its own results are other ones; the wait is at the end.)
    const int n_tiles = l.counts[1];
    griddep_launch_dependents();
    if ((int)blockIdx.y >= n_tiles) {
        griddep_wait();
        return;
    }
    uint32_t tmem_cols = 32;
    while ((int)tmem_cols < shape.cols) tmem_cols *= 2;
    if (warp == 0) tmem_alloc(slot, tmem_cols);
    if (tid == 0) {
        for (int i = 0; i < kBigStages; ++i) mbar_init(bars + 8 * i, 1);
        fence_mbarrier_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot));
    // this CTA's columns and part of K
    const int j0 = (int)blockIdx.z * kBigCols, cols = min(SR - j0, kBigCols);
    const int steps_all = (K + 63) / 64;
    const int s0 = (int)((long long)steps_all * rank / splits), s1 = (int)((long long)steps_all * (rank + 1) / splits);
    const int n = s1 - s0;
    const uint32_t idesc = umma_idesc_bf16(shape.cols);
    const int chunk = tid & 7, row0 = tid >> 3;
    const uint32_t put = (uint32_t)(row0 * 128 + ((chunk ^ (row0 & 7)) << 4));      // rows 32 apart keep row & 7
    float* sums = reinterpret_cast<float*>(raw + (base - smem_u32(raw)));
    const int pitch = shape.cols + 4;
    int used = 0;                        // steps of earlier tiles
    bool dead = false;                   // a wait gave up: the CTA goes on with the cluster, without its copies and products
    for (int ti = blockIdx.y; ti < n_tiles; ti += gridDim.y) {
        const BigTile tile = l.big[ti];
        if (tile.adapter < 0) continue;
        const int r = rank_of(p, tile.adapter);
        // what this thread copies: a 16-byte chunk of four rows of x and of every 32nd row of A; a row
        // that is not there arrives as zeros
        const char* xr[kBigTile / 32];
        int xb[kBigTile / 32];
#pragma unroll
        for (int i = 0; i < kBigTile / 32; ++i) {
            const int row = row0 + 32 * i;
            xb[i] = row < tile.count ? 16 : 0;
            xr[i] = (xb[i] ? row_ptr(p.x, l.order[tile.first + row]) : p.x.ptr) + 16 * chunk + s0 * 128;
        }
        const char* ar = reinterpret_cast<const char*>(p.a + ((size_t)tile.adapter * SR + j0 + row0) * K) + 16 * chunk + s0 * 128;
        const size_t a32 = (size_t)K * 64;
        unsigned mine = 0;
        for (int i = 0; 32 * i + row0 < cols; ++i) mine |= ((j0 + 32 * i + row0) % p.rank < r ? 1u : 0u) << i;
        auto load = [&](int s) {         // step s of this tile
            const uint32_t to = base + (uint32_t)((used + s) % kBigStages) * shape.stage + put;
            const int off = s * 128;
            const bool in = (s0 + s) * 64 + 8 * chunk < K;           // (the last step may end early)
            const char* none = p.x.ptr;
#pragma unroll
            for (int i = 0; i < kBigTile / 32; ++i) copy16_async(to + i * 4096, in ? xr[i] + off : none, in ? xb[i] : 0);
            const char* from = ar + off;
#pragma unroll 2
            for (int i = 0; 32 * i + row0 < shape.cols; ++i, from += a32) {
                const bool take = in && (mine >> i & 1);
                copy16_async(to + kBigTile * 128 + i * 4096, take ? from : none, take ? 16 : 0);
            }
        };
        bool bad = dead;
        for (int s = 0; s < kBigStages - 1; ++s) {
            if (s < n && !dead) load(s);
            copies_commit();
        }
        for (int s = 0; s < n; ++s) {
            copies_wait<kBigStages - 2>();
            fence_async_smem();
            if (__syncthreads_or(bad)) break;
            if (tid == 0) {
                tc_fence_after_sync();
                const uint32_t at = base + (uint32_t)((used + s) % kBigStages) * shape.stage;
                const uint64_t xa = umma_desc_sw128(at), wa = umma_desc_sw128(at + kBigTile * 128);
#pragma unroll
                for (int k = 0; k < 4; ++k) umma_bf16(tmem, xa + 2 * k, wa + 2 * k, idesc, s > 0 || k > 0);
                umma_commit(bars + 8 * ((used + s) % kBigStages));
            }
            const int next = s + kBigStages - 1;
            if (next < n) {
                // the stage of step s - 1 is free once its products have read it
                if (s > 0) {
                    const int u = used + s - 1;
                    bad = !mbar_wait_bounded(bars + 8 * (u % kBigStages), (u / kBigStages) & 1, p.wait, kErrConsumerWait);
                }
                if (!bad) load(next);
            }
            copies_commit();
        }
        if (!bad) {
            const int u = used + n - 1;
            bad = !mbar_wait_bounded(bars + 8 * (u % kBigStages), (u / kBigStages) & 1, p.wait, kErrConsumerWait);
        }
        used += n;
        copies_wait<0>();
        dead = __syncthreads_or(bad);
        tc_fence_after_sync();
        // a thread has a token's row; two warps share 32 tokens' columns
        const int row = 32 * (warp & 3) + lane;
        const bool alone = splits == 1;
        float* out = p.low_big + (size_t)tile.first * SR + j0;
        float* to = alone ? out + (size_t)row * SR : sums + row * pitch;
        for (int j = 16 * (warp >> 2); j < shape.cols; j += 32) {
            float v[16];
            tmem_ld16(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + j, v);
            tmem_wait_ld();
            if (row < tile.count) {
#pragma unroll
                for (int k = 0; k < 16; k += 4)
                    if (j + k < cols) *reinterpret_cast<float4*>(to + j + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            }
        }
        tc_fence_before_sync();
        if (!alone) {
            cluster.sync();
            // this CTA's share of the tokens
            const int first = tile.count * rank / splits, last = tile.count * (rank + 1) / splits;
            for (int i = tid; i < (last - first) * (cols / 4); i += kBigThreads) {
                const int t = first + i / (cols / 4), j = i % (cols / 4) * 4;
                float4 v = {0.f, 0.f, 0.f, 0.f};
                for (int q = 0; q < splits; ++q) {
                    const float4 w = *reinterpret_cast<const float4*>(cluster.map_shared_rank(sums, q) + t * pitch + j);
                    v.x += w.x; v.y += w.y; v.z += w.z; v.w += w.w;
                }
                *reinterpret_cast<float4*>(out + (size_t)t * SR + j) = v;
            }
            cluster.sync();              // the others have read this CTA's sums: its stages are free
        } else {
            __syncthreads();
        }
        tc_fence_after_sync();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem, tmem_cols);
    griddep_wait();
}

// Second product of big tiles: a warp has 16 of the tile's tokens, whose first products it keeps in shared
// memory as bf16 parts in the order of the operands; the CTA goes over blocks of 64 columns of a part, B's
// rows a few blocks ahead in a ring, base one block ahead in registers.  All tiles' blocks are dealt
// to the CTAs in equal runs.  Bound by base and out.
constexpr int kUpBlock = 64, kUpRing = 3;

__host__ __device__ constexpr int up_big_smem(int chunks, int parts) {
    return kUpWarps * chunks * parts * 512 + kUpRing * kUpBlock * chunks * 32;
}

// Blocks of columns: each lies in one part.
struct Blocks {
    int part, n0, end;       // the part, the block's first column, the part's end
};
__device__ __forceinline__ int count_blocks(const AdapterParams& p) {
    int n = 0;
    for (int i = 0; i < p.parts; ++i) n += (p.part_end[i] - (i ? p.part_end[i - 1] : 0) + kUpBlock - 1) / kUpBlock;
    return n;
}
__device__ __forceinline__ Blocks block_at(const AdapterParams& p, int b) {
    Blocks k = {0, 0, p.part_end[0]};
    while (k.part + 1 < p.parts) {
        const int n = (k.end - k.n0 + kUpBlock - 1) / kUpBlock;
        if (b < n) break;
        b -= n;
        ++k.part;
        k.n0 = k.end;
        k.end = p.part_end[k.part];
    }
    k.n0 += b * kUpBlock;
    return k;
}

// C: runs of 16 r, at least rank / 16; BASE 0: none, or rows that do not allow wide accesses, 1: bf16,
// 2: fp32; P: parts of a first product
template <int C, int BASE, int P>
__global__ void __launch_bounds__(kUpThreads, 2) adapters_up_big_kernel(const __grid_constant__ AdapterParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const Lists l = lists_of(p.tiles, p.tokens, p.num);
    // the first products are there: the kernel before this one let it start after it had waited for them
    const int n_tiles = l.counts[1];
    griddep_launch_dependents();
    const int R = p.rank, N = p.N;
    uint4* mine = reinterpret_cast<uint4*>(smem) + warp * C * P * 32 + lane;
    const uint32_t ring = smem_u32(smem) + kUpWarps * C * P * 512;
    constexpr int kStage = kUpBlock * C * 32, kGranules = kUpBlock * C * 2;         // 16 bytes each
    auto swap = [](int row) { return C >= 4 ? row : C == 2 ? row >> 1 : 0; };
    uint32_t piece_at[C];                // this lane's 8 bytes of a run of 16 r, in its row of eight
#pragma unroll
    for (int q = 0; q < C; ++q) piece_at[q] = g * 32 * C + 16 * ((2 * q + (c >> 1)) ^ swap(g)) + 8 * (c & 1);
    const size_t step = (size_t)p.parts * R;
    const int blocks = count_blocks(p);
    const long long all = (long long)n_tiles * blocks;
    long long at = all * blockIdx.x / gridDim.x;
    const long long end = all * (blockIdx.x + 1) / gridDim.x;
    while (at < end) {
        const BigTile tile = l.big[at / blocks];
        const int b0 = (int)(at % blocks), b1 = (int)min((long long)blocks, b0 + end - at);
        at += b1 - b0;
        const int ad = tile.adapter, r = rank_of(p, ad);
        const float scale = ad >= 0 && p.scale ? p.scale[ad] : 1.f;
        const bool active = 16 * warp < tile.count;
        const int i0 = 16 * warp + g, i1 = i0 + 8;
        const int t0 = i0 < tile.count ? l.order[tile.first + i0] : -1, t1 = i1 < tile.count ? l.order[tile.first + i1] : -1;
        const uint16_t* b = p.b + (size_t)max(ad, 0) * N * R;
        const char *from0 = row_ptr(p.base, max(t0, 0)), *from1 = row_ptr(p.base, max(t1, 0));
        char *to0 = row_ptr(p.y, max(t0, 0)), *to1 = row_ptr(p.y, max(t1, 0));
        char *to320 = row_ptr(p.y32, max(t0, 0)), *to321 = row_ptr(p.y32, max(t1, 0));
        // A block of B into its ring stage: columns in the order of the products' operands, 16-byte pieces
        // exchanged by row so that eight rows' reads meet no bank twice more than they must.  What lies past
        // the rank or the part arrives as zeros.
        auto load = [&](int blk) {
            if (r == 0) return;
            const Blocks k = block_at(p, blk);
            const uint32_t to = ring + (uint32_t)((blk - b0) % kUpRing) * kStage;
#pragma unroll
            for (int j = 0; j < (kGranules + kUpThreads - 1) / kUpThreads; ++j) {
                const int i = tid + j * kUpThreads, row = i / (2 * C), piece = i % (2 * C);
                if (kGranules % kUpThreads && i >= kGranules) break;
                const int rg = row & 7, n = k.n0 + (row >> 4) * 16 + (rg >> 1) * 4 + (rg & 1) + (row >> 3 & 1) * 2;
                const int bytes = n < k.end ? min(max(2 * (r - 8 * piece), 0), 16) : 0;
                copy16_async(to + row * 32 * C + 16 * (piece ^ swap(rg)), bytes ? b + (size_t)n * R + 8 * piece : p.b, bytes);
            }
        };
        uint4 next0[4], next1[4];
        auto fetch = [&](int blk) {      // base of block `blk`
            const Blocks k = block_at(p, min(blk, b1 - 1));
#pragma unroll
            for (int u = 0; BASE != 0 && u < 4; ++u) {
                const int n = k.n0 + 16 * u + 4 * c;
                const bool in = blk < b1 && n + 4 <= k.end;
                if (BASE == 1) {
                    const uint2 none = {0, 0};
                    const uint2 x = in && t0 >= 0 ? ldg64(from0 + 2 * (size_t)n) : none;
                    const uint2 y = in && t1 >= 0 ? ldg64(from1 + 2 * (size_t)n) : none;
                    next0[u].x = x.x; next0[u].y = x.y;
                    next1[u].x = y.x; next1[u].y = y.y;
                } else {
                    const uint4 none = {0, 0, 0, 0};
                    next0[u] = in && t0 >= 0 ? ldg128(from0 + 4 * (size_t)n) : none;
                    next1[u] = in && t1 >= 0 ? ldg128(from1 + 4 * (size_t)n) : none;
                }
            }
        };
#pragma unroll
        for (int i = 0; i < kUpRing - 1; ++i) {
            if (b0 + i < b1) load(b0 + i);
            copies_commit();
        }
        fetch(b0);
        int held = -1;                   // the part whose first products are in `mine`
        const float* low0 = p.low_big + (size_t)(tile.first + i0) * step;
        const bool put = ad >= 0 || !p.in_place, put32 = P == 3 && (ad >= 0 || !p.in_place32);
        for (int blk = b0; blk < b1; ++blk) {
            copies_wait<kUpRing - 2>();
            __syncthreads();
            if (blk + kUpRing - 1 < b1) load(blk + kUpRing - 1);
            copies_commit();
            if (!active) continue;
            const Blocks k = block_at(p, blk);
            if (k.part != held && r > 0) {
                held = k.part;
                __syncwarp();
                float4 s0[C], s1[C];
#pragma unroll
                for (int q = 0; q < C; ++q) {
                    const float* low = low0 + held * R + 16 * q + 4 * c;
                    const bool in = 16 * q + 4 * c < r;
                    s0[q] = in && t0 >= 0 ? ld_cg_f32x4(low) : make_float4(0.f, 0.f, 0.f, 0.f);
                    s1[q] = in && t1 >= 0 ? ld_cg_f32x4(low + 8 * step) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int q = 0; q < C; ++q) {
                    const int rr = 16 * q + 4 * c;
                    const bool in1 = rr + 1 < r, in2 = rr + 2 < r, in3 = rr + 3 < r;
                    const Parts a0 = split(s0[q].x * scale, in1 ? s0[q].y * scale : 0.f, P);
                    const Parts a1 = split(s1[q].x * scale, in1 ? s1[q].y * scale : 0.f, P);
                    const Parts a2 = split(in2 ? s0[q].z * scale : 0.f, in3 ? s0[q].w * scale : 0.f, P);
                    const Parts a3 = split(in2 ? s1[q].z * scale : 0.f, in3 ? s1[q].w * scale : 0.f, P);
#pragma unroll
                    for (int i = 0; i < P; ++i) mine[(q * P + i) * 32] = make_uint4(a0.v[i], a1.v[i], a2.v[i], a3.v[i]);
                }
                __syncwarp();
            }
            float d[4][2][4] = {};
            if (r > 0) {
                const uint32_t bt = ring + (uint32_t)((blk - b0) % kUpRing) * kStage;
#pragma unroll
                for (int q = 0; q < C; ++q) {
                    uint4 a[P];
#pragma unroll
                    for (int i = 0; i < P; ++i) a[i] = mine[(q * P + i) * 32];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint2 w;
                            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                         : "=r"(w.x), "=r"(w.y) : "r"(bt + piece_at[q] + (16 * u + 8 * h) * 32 * C));
#pragma unroll
                            for (int j = 0; j < P; ++j) mma_bf16_16816(d[u][h], a[j].x, a[j].y, a[j].z, a[j].w, w.x, w.y);
                        }
                }
            }
            float odd = 0.f;             // NaN if any sum is, or infinite
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
                for (int j = 0; j < 4; ++j) odd = fmaf(d[u][0][j], 0.f, fmaf(d[u][1][j], 0.f, odd));
            if (odd != odd) {
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if ((h ? t1 : t0) < 0) continue;
                        float v[4] = {d[u][0][2 * h], d[u][0][2 * h + 1], d[u][1][2 * h], d[u][1][2 * h + 1]};
                        plain_up(p, low0 + (h ? 8 * step : 0), scale, b, k.n0 + 16 * u + 4 * c, r, v);
                        d[u][0][2 * h] = v[0]; d[u][0][2 * h + 1] = v[1]; d[u][1][2 * h] = v[2]; d[u][1][2 * h + 1] = v[3];
                    }
            }
            if (k.n0 + kUpBlock <= k.end && p.wide) {
                if (BASE != 0) {
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint4 raw = h ? next1[u] : next0[u];
                            float from[4];
                            if (BASE == 1) {
                                bf16x2_to_f32(raw.x, from[0], from[1]);
                                bf16x2_to_f32(raw.y, from[2], from[3]);
                            } else {
                                from[0] = __uint_as_float(raw.x); from[1] = __uint_as_float(raw.y);
                                from[2] = __uint_as_float(raw.z); from[3] = __uint_as_float(raw.w);
                            }
#pragma unroll
                            for (int j = 0; j < 4; ++j) d[u][j >> 1][2 * h + (j & 1)] += from[j];
                        }
                    fetch(blk + 1);      // base is in the sums: the next block's may come
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if ((h ? t1 : t0) < 0) continue;
                    char *to = (h ? to1 : to0) + 2 * (size_t)(k.n0 + 4 * c), *to32 = (h ? to321 : to320) + 4 * (size_t)(k.n0 + 4 * c);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float v[4] = {d[u][0][2 * h], d[u][0][2 * h + 1], d[u][1][2 * h], d[u][1][2 * h + 1]};
                        if (put) put_wide(to, false, 16 * u, v);
                        if (put32) put_wide(to32, true, 16 * u, v);
                    }
                }
            } else {
                // the part's last columns, or rows that do not allow wide accesses
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int t = h ? t1 : t0, n = k.n0 + 16 * u + 4 * c;
                        if (t < 0 || n >= k.end) continue;
                        float v[4] = {d[u][0][2 * h], d[u][0][2 * h + 1], d[u][1][2 * h], d[u][1][2 * h + 1]}, from[4] = {};
                        if (p.base.ptr) load4(p.base, t, n, k.end, p.wide, from);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[j] += from[j];
                        if (put) put4(p.y, t, n, k.end, p.wide, v);
                        if (put32) put4(p.y32, t, n, k.end, p.wide, v);
                    }
                fetch(blk + 1);
            }
        }
        copies_wait<0>();
        __syncthreads();                 // the ring is free for the next tile
    }
    griddep_wait();
}

// ---------------------------------------------------------------- host

// CTAs that share K of the big tiles of `tokens` tokens, a power of two: enough to fill the GPU if they are
// of few adapters (clusters of 8 leave some of a GPC's SMs out: 128 are counted), with four steps of
// 64 k each at least.
static int big_splits(long long tokens, int K) {
    const long long tiles = (tokens + kBigTile - 1) / kBigTile;
    int n = 1;
    while (n < kMaxSplits && 2 * n * tiles <= 128 && 2 * n * 256 <= K) n *= 2;
    return n;
}

static size_t up256(size_t n) { return (n + 255) / 256 * 256; }
static size_t low_bytes(long long tokens, int rank, int parts) { return up256((size_t)tokens * rank * parts * 4); }
static size_t low_big_bytes(long long tokens, int rank, int parts) {
    return tokens > kFewTokens && rank <= kBigRank ? low_bytes(tokens, rank, parts) : 0;
}
static size_t lists_bytes(long long tokens, int num) {
    return tokens > kFewTokens ? up256(16 + (size_t)max_big(tokens, num) * sizeof(BigTile) + (size_t)tokens * 4 +
                                       (size_t)max_small(tokens, num) * sizeof(Tile)) : 0;
}

static size_t adapters_bytes(long long tokens, int num, int rank, int parts) {
    return DL_WORKSPACE_ZERO_BYTES + low_bytes(tokens, rank, parts) + low_big_bytes(tokens, rank, parts) + lists_bytes(tokens, num);
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

template <class F>
static cudaError_t raise_smem(F kernel, size_t bytes) {
    return bytes > 48 * 1024 ? cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) : cudaSuccess;
}

template <bool FEW>
static cudaError_t launch_small(const AdapterParams& p, long long tiles, int sm_count, cudaStream_t stream, bool up) {
    const size_t smem = FEW ? sizeof(FewTiles) : 0;
    if (up) {
        // few columns a warp while that leaves warps for every SM
        const long long fine = tiles * ((p.N + 15) / 16), coarse = tiles * ((p.N + 63) / 64);
        const bool small = fine <= 8LL * sm_count;
        const long long ctas = ((small ? fine : coarse) + kUpWarps - 1) / kUpWarps, most = 2LL * sm_count;
        const dim3 grid((unsigned)(ctas < most ? ctas : most));
        return small ? launch_dependent(adapters_up_kernel<FEW, 1, 4>, grid, dim3(kUpThreads), smem, stream, p)
                     : launch_dependent(adapters_up_kernel<FEW, 4, 2>, grid, dim3(kUpThreads), smem, stream, p);
    }
    const long long items = tiles * p.parts * ((p.rank + 15) / 16), most = 4LL * sm_count / kLowCluster;
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
    return cudaLaunchKernelEx(&cfg, adapters_low_kernel<FEW>, p);
}

static cudaError_t launch_low_big(const AdapterParams& p, long long tiles, int sm_count, cudaStream_t stream) {
    const int columns = p.parts * p.rank, groups = (columns + kBigCols - 1) / kBigCols, splits = big_splits(p.tokens, p.K);
    const long long most = 4LL * sm_count / (splits * groups) + 1;
    const size_t smem = big_smem(columns).total;
    const cudaError_t e = raise_smem(adapters_low_big_kernel, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = splits;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits, (unsigned)(tiles < most ? tiles : most), groups);
    cfg.blockDim = dim3(kBigThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, adapters_low_big_kernel, p);
}

template <int C, int BASE, int P>
static cudaError_t launch_up_big(const AdapterParams& p, int sm_count, cudaStream_t stream) {
    constexpr int smem = up_big_smem(C, P);
    const cudaError_t e = raise_smem(adapters_up_big_kernel<C, BASE, P>, smem);
    if (e != cudaSuccess) return e;
    const int ctas = 2 * (smem + 1024) <= 228 * 1024 ? 2 : 1;
    return launch_dependent(adapters_up_big_kernel<C, BASE, P>, dim3(ctas * sm_count), dim3(kUpThreads), smem, stream, p);
}

template <int C>
static cudaError_t launch_up_big_rank(const AdapterParams& p, int sm_count, cudaStream_t stream) {
    const int base = !p.base.ptr || !p.wide ? 0 : p.base.f32 ? 2 : 1;
    if (p.y32.ptr)
        return base == 0 ? launch_up_big<C, 0, 3>(p, sm_count, stream)
               : base == 1 ? launch_up_big<C, 1, 3>(p, sm_count, stream) : launch_up_big<C, 2, 3>(p, sm_count, stream);
    return base == 0 ? launch_up_big<C, 0, 2>(p, sm_count, stream)
           : base == 1 ? launch_up_big<C, 1, 2>(p, sm_count, stream) : launch_up_big<C, 2, 2>(p, sm_count, stream);
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
    p.low_big = reinterpret_cast<float*>(scratch + low_bytes(tokens, p.rank, p.parts));
    p.tiles = reinterpret_cast<int*>(scratch + low_bytes(tokens, p.rank, p.parts) + low_big_bytes(tokens, p.rank, p.parts));
    p.big_from = p.rank <= kBigRank ? kBigFrom : 0x7fffffff;
    p.index = index;
    p.tokens = tokens;
    p.in_place = same_rows(p.y, p.base);
    p.in_place32 = p.y32.ptr && same_rows(p.y32, p.base);
    p.wide = true;
    for (const Rows* r : {&p.base, &p.y, &p.y32})
        if (r->ptr) p.wide = p.wide && !(((uintptr_t)r->ptr | (uintptr_t)r->stride) & (r->f32 ? 15 : 7));
    const long long small = tokens <= kFewTokens ? tokens : max_small(tokens, p.num);
    if (small * ((N + 15) / 16) > 0x7fff0000LL || small * p.parts * ((p.rank + 15) / 16) > 0x7fff0000LL)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "tokens=%d with N=%d exceed one launch", tokens, N);
    HostDevice dev;
    if ((s = host_device(dev)) != DL_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.wait = WaitCtl{dev.err_word, dev.wait_limit_ns};
    cudaError_t e;
    if (tokens <= kFewTokens) {
        if ((e = launch_small<true>(p, small, dev.sm_count, st, false)) == cudaSuccess)
            e = launch_small<true>(p, small, dev.sm_count, st, true);
    } else {
        // Each list's kernels find how much there is on the device.  Both first products may run at the
        // same time, then both second ones.
        const long long big = max_big(tokens, p.num);
        const size_t counters = (size_t)(p.num + 1) * 4;
        if ((e = raise_smem(sort_tokens_kernel, counters)) == cudaSuccess)
            e = launch_dependent(sort_tokens_kernel, dim3(1), dim3(1024), counters, st, p);
        if (e == cudaSuccess) e = launch_small<false>(p, small, dev.sm_count, st, false);
        if (e == cudaSuccess && p.rank <= kBigRank) e = launch_low_big(p, big, dev.sm_count, st);
        if (e == cudaSuccess) e = launch_small<false>(p, small, dev.sm_count, st, true);
        if (e == cudaSuccess && p.rank <= kBigRank)
            e = p.rank <= 16   ? launch_up_big_rank<1>(p, dev.sm_count, st)
                : p.rank <= 32 ? launch_up_big_rank<2>(p, dev.sm_count, st)
                : p.rank <= 64 ? launch_up_big_rank<4>(p, dev.sm_count, st)
                               : launch_up_big_rank<8>(p, dev.sm_count, st);
    }
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "linear_adapters launch: %s", cudaGetErrorString(e));
    return host_ok();
}
