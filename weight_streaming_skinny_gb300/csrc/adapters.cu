// Low-rank adapters of many requests beside a shared projection (dl_linear_adapters).
#include <cooperative_groups.h>

#include <type_traits>

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
    uint16_t* low;           // [tokens][2 or 3][parts * rank] scaled first products in bf16 parts (small tiles)
    int* tiles;              // more than kFewTokens tokens: what sort_tokens_kernel writes
    int big_from;            // kBigFrom, or none if ranks are too large
    bool in_place, in_place32;   // base is y, y32: rows without an adapter stay as they are
    bool wide;               // groups of eight columns of base, y and y32 are 16-byte aligned
    // big tiles
    float* low_big;          // [tokens][parts * rank], by place in `order`, without scale
    WaitCtl wait;
};

// Up to kTile tokens of one adapter.
struct Tile {
    int adapter, rank, count;    // adapter -1, rank 0: tokens without one
    float scale;
    int token[kTile];
    __device__ int at(int i) const { return i < count ? token[i] : -1; }
};
// Tokens order[first .. first + count) of one adapter.
struct BigTile {
    int adapter, first, count, rank;
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
__device__ __forceinline__ float scale_of(const AdapterParams& p, int adapter) {
    return adapter >= 0 && p.scale ? p.scale[adapter] : 1.f;
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
// The sum of a number's bytes.
__device__ __forceinline__ int byte_sum(unsigned long long v) {
    return __dp4a((unsigned)v, 0x01010101u, __dp4a((unsigned)(v >> 32), 0x01010101u, 0u));
}

__device__ __forceinline__ int make_tiles(const AdapterParams& p, FewTiles& s) {
    static_assert(kFewTokens == 256, "a byte for each of 8 warps");
    const int T = p.tokens, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    const unsigned below = (1u << lane) - 1;
    if (T <= 32) {
        if (warp == 0) {
            const int mine = lane < T ? adapter_of(p, lane) : -2, r = rank_of(p, mine);
            const float scale = scale_of(p, mine);
            const unsigned same = __match_any_sync(~0u, mine);
            const int place = __popc(same & below);
            const unsigned m = __ballot_sync(~0u, lane < T && place % kTile == 0);
            if (lane < T) {
                const int opener = nth_bit(same, place / kTile * kTile);
                Tile& tile = s.tile[__popc(m & ((1u << opener) - 1))];
                if (opener == lane) {
                    tile.adapter = mine;
                    tile.rank = r;
                    tile.scale = scale;
                    tile.count = min(__popc(same) - place, kTile);
                }
                tile.token[place % kTile] = lane;
            }
            if (lane == 0) s.n = __popc(m);
        }
        __syncthreads();
        return s.n;
    }
    const int mine = t < T ? adapter_of(p, t) : -2;
    const int r = rank_of(p, mine);      // (these loads overlap what follows)
    const float scale = scale_of(p, mine);
    for (int i = t; i < kSlots; i += blockDim.x) {
        s.slot[i] = 0;
        s.held[i] = 0;
    }
    const unsigned same = __match_any_sync(~0u, mine);
    const int leader = __ffs(same) - 1;
    int at = 0;
    __syncthreads();
    if (t < T && lane == leader) {
        at = (mine * 0x9E3779B1u) >> 23;         // 9 bits
        while (true) {
            const int found = atomicCAS(&s.slot[at], 0, mine + 2);
            if (found == 0 || found == mine + 2) break;
            at = (at + 1) % kSlots;
        }
        reinterpret_cast<unsigned char*>(&s.held[at])[warp] = (unsigned char)__popc(same);
    }
    at = __shfl_sync(~0u, at, leader);
    __syncthreads();
    // the bytes of the warps before this one, and of all
    const unsigned long long held = s.held[at];
    const int place = byte_sum(held & ((1ull << (8 * warp)) - 1)) + __popc(same & below);
    const bool opens = t < T && place % kTile == 0;
    const unsigned m = __ballot_sync(~0u, opens);
    if (lane == 0) s.opened[warp] = __popc(m);
    __syncthreads();
    int n = 0, first = 0;
#pragma unroll
    for (int w = 0; w < kFewTokens / 32; ++w) {
        if (w < warp) first += s.opened[w];
        n += s.opened[w];
    }
    if (opens) {
        const int number = first + __popc(m & below);
        s.number[at][place / kTile] = (unsigned char)number;
        Tile& tile = s.tile[number];
        tile.adapter = mine;
        tile.rank = r;
        tile.scale = scale;
        tile.count = min(byte_sum(held) - place, kTile);
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
        const int ad = i < p.num ? i : -1, r = n ? rank_of(p, ad) : 0;
        for (int j = 0; j < mine[0]; ++j) {
            Tile& tile = l.small[first[0] + j];
            tile.adapter = ad;
            tile.rank = r;
            tile.scale = scale_of(p, ad);
            tile.count = min(n - j * kTile, kTile);
        }
        for (int j = 0; j < mine[1]; ++j)
            l.big[first[1] + j] = BigTile{ad, first[2] + j * kBigTile, min(n - j * kBigTile, kBigTile), r};
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

// ---------------------------------------------------------------- parts

// The fp32 first products go into the second ones as two bf16 parts (2^-18 of the value is lost), three
// (24 bits: nothing) where an fp32 result is asked for.  The parts of a value and their products can
// leave NaN where the value's own product is an infinity; what comes out NaN is summed again as it stands.
// Two values as packed bf16 parts, each the next 8 bits of the value, rounded.  (An infinity's later parts are
// NaN, and so is then what they are multiplied to.)
template <int P>
__device__ __forceinline__ void split(float a, float b, uint32_t (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        v[i] = f32x2_to_bf16x2(a, b);
        if (i + 1 < P) {
            float ha, hb;
            bf16x2_to_f32(v[i], ha, hb);
            a -= ha;
            b -= hb;
        }
    }
}

// ---------------------------------------------------------------- small tiles: first product

// low[t][j] = scale * sum_k A[j][k] x[t][k], as the bf16 parts that the second product takes: a cluster of CTAs shares K, a warp takes 16 rows of A and
// a tile's 16 tokens over its part of K.  A (and x) go from global memory straight into
// the operands of mma.m16n8k16: the sum over k may take its terms in any order, so a lane's
// 16-byte load of 8 consecutive k is the k-slots that it holds in two products.
template <int N>
using Int = std::integral_constant<int, N>;
constexpr int kLowThreads = 256, kLowWarps = kLowThreads / 32;
constexpr int kLowCluster = 8;           // at most

__global__ void __launch_bounds__(kLowThreads, 2) adapters_low_kernel(const __grid_constant__ AdapterParams p) {
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
    static_assert((kLowWarps & (kLowWarps - 1)) == 0, "a shift divides");
    const int shift = 31 - __clz(workers);
    const int k0 = (int)((long long)runs * worker >> shift) * 32, k1 = (int)((long long)runs * (worker + 1) >> shift) * 32;
    const unsigned per = p.parts * groups, items = n_tiles * per;      // fits: a launch of more is refused
    bool waiting = false;
    for (unsigned item = blockIdx.x / size; item < items; item += gridDim.x / size) {
        const unsigned i = item % per;
        const int j0 = (int)(i % groups) * 16, pt = (int)(i / groups);
        const Tile& tile = tiles[item / per];
        const int ad = tile.adapter, r = tile.rank;
        if (j0 >= r) continue;
        const int t0 = tile.at(g), t1 = tile.at(g + 8);
        const bool two = tile.count > 8, row0 = j0 + g < r, row1 = j0 + g + 8 < r;
        const uint16_t* a0 = p.a + (((size_t)ad * p.parts + pt) * R + j0 + g) * K + 8 * c;
        const uint16_t* a1 = a0 + (size_t)8 * K;
        const char *x0 = row_ptr(p.x, max(t0, 0)) + 16 * c, *x1 = row_ptr(p.x, max(t1, 0)) + 16 * c;
        float d0[4] = {}, d1[4] = {};
        const uint4 none = {0, 0, 0, 0};
        // `n` runs at a time, their loads all in flight (as far as this warp's part and K go); every lane takes
        // part in every product
        auto steps = [&](auto count, auto second, int run) {
            constexpr int n = decltype(count)::value;
            constexpr bool both = decltype(second)::value;
            uint4 va[n], vb[n], xa[n], xb[both ? n : 1];
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const int k = run + 32 * i;
                const bool in = k < k1 && k + 8 * c < K;
                va[i] = in && row0 ? ldg128(a0 + k) : none;
                vb[i] = in && row1 ? ldg128(a1 + k) : none;
                xa[i] = in && t0 >= 0 ? ldg128(x0 + 2 * k) : none;
                if (both) xb[i] = in && t1 >= 0 ? ldg128(x1 + 2 * k) : none;
            }
#pragma unroll
            for (int i = 0; i < n; ++i) {
                mma_bf16_16816(d0, va[i].x, vb[i].x, va[i].y, vb[i].y, xa[i].x, xa[i].y);
                mma_bf16_16816(d0, va[i].z, vb[i].z, va[i].w, vb[i].w, xa[i].z, xa[i].w);
                if (both) {
                    mma_bf16_16816(d1, va[i].x, vb[i].x, va[i].y, vb[i].y, xb[i].x, xb[i].y);
                    mma_bf16_16816(d1, va[i].z, vb[i].z, va[i].w, vb[i].w, xb[i].z, xb[i].w);
                }
            }
        };
        if (two) {
            for (int run = k0; run < k1; run += 128) steps(Int<4>(), std::true_type(), run);
        } else {
            for (int run = k0; run < k1; run += 256) steps(Int<8>(), std::false_type(), run);
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
        if (waiting) cluster.barrier_wait();     // the others have read the last item's sums
        part[tid] = v;
        cluster.sync();
        // rank i finishes a share of the 256 sums
        const int each = 256 / size;
        if (tid < each) {
            const int at = rank * each + tid, t = tile.at(at / 16), j = j0 + at % 16;
            float all = 0.f;
#pragma unroll
            for (int q = 0; q < kLowCluster; ++q)
                if (q < size) all += cluster.map_shared_rank(part, q)[at];
            if (t >= 0 && j < R) {       // (zeros past the rank: it may end inside four that are read at once)
                const size_t step = (size_t)p.parts * R;
                uint16_t* to = p.low + (size_t)t * (p.y32.ptr ? 3 : 2) * step + pt * R + j;
                uint32_t v[3];
                split(j < r ? all * tile.scale : 0.f, 0.f, v);
                to[0] = (uint16_t)v[0];
                to[step] = (uint16_t)v[1];
                if (p.y32.ptr) to[2 * step] = (uint16_t)v[2];
            }
        }
        cluster.barrier_arrive();
        waiting = true;
    }
    if (waiting) cluster.barrier_wait();
}

// ---------------------------------------------------------------- second product

// out[t][n] = base[t][n] + sum_r low[t][r] B[n][r]: tokens are the rows of the product, 16 for a warp,
// B's rows its columns.  32 consecutive columns are four products of 8 whose results lie four lanes to a
// row, two columns a lane; which column is which product's is chosen so that a lane's eight results are
// consecutive: lane c of a row has columns 8 c .. 8 c + 7, product i has 2 i and 2 i + 1 of each lane's.

// Eight columns of a row from n on, as far as `end`; `wide`: whole and aligned.
__device__ __forceinline__ void load_cols(const char* row, bool f32, int n, int end, bool wide, float (&v)[8]) {
    if (wide) {
        row_load8(row, f32, n, v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = n + k < end ? row_load1(row, f32, n + k) : 0.f;
    }
}
__device__ __forceinline__ void put_cols(char* row, bool f32, int n, int end, bool wide, const float (&v)[8]) {
    if (wide) {
        row_store8(row, f32, n, v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (n + k < end) row_store1(row, f32, n + k, v[k]);
    }
}

__device__ __forceinline__ int part_of(const AdapterParams& p, int n) {
    int pt = 0;
    while (pt + 1 < p.parts && n >= p.part_end[pt]) ++pt;
    return pt;
}

// Sums of eight columns from n on that came out NaN, as they stand; `low`: a token's first products, times scale,
// in fp32 (PACKED 0) or in that many bf16 parts.
template <int PACKED>
__device__ __noinline__ void plain_up(const AdapterParams& p, const void* low, float scale, const uint16_t* b, int n, int r,
                                      float (&v)[8]) {
    const size_t step = (size_t)p.parts * p.rank;
    for (int k = 0; k < 8; ++k) {
        if (v[k] == v[k] || n + k >= p.N) continue;
        const int at = part_of(p, n + k) * p.rank;
        v[k] = 0.f;
        for (int i = 0; i < r; ++i) {
            float s = 0.f;
            if (PACKED == 0) {
                s = static_cast<const float*>(low)[at + i];
            } else {
                const uint16_t* q = static_cast<const uint16_t*>(low) + at + i;
                s = bf16_bits_to_f32(q[0]);
                if (fabsf(s) <= 3.4028235e38f)       // (an infinity's later parts are NaN)
                    for (int j = 1; j < PACKED; ++j) s += bf16_bits_to_f32(q[j * step]);
            }
            v[k] = fmaf(s * scale, bf16_bits_to_f32(b[(size_t)(n + k) * p.rank + i]), v[k]);
        }
    }
}

// The bits of four values of r from `at` on that lie within the rank; what lies past it is nobody's.
__device__ __forceinline__ uint2 rank_mask(int at, int r) {
    return make_uint2((at < r ? 0xffffu : 0u) | (at + 1 < r ? 0xffff0000u : 0u),
                      (at + 2 < r ? 0xffffu : 0u) | (at + 3 < r ? 0xffff0000u : 0u));
}

// Small tiles: a warp takes 64 columns of a tile, 16 r at a time.  What does not depend on the first products
// (the tiles, base, B) is fetched before they are waited for: the kernel that makes them lets this one start only
// after it had waited for all earlier ones.  Bound by instructions and latencies: a tile of few tokens costs as
// much as one of 16, so each lane has all its loads of 16 r in flight at once.
// BASE 0: none, 1: bf16, 2: fp32; P: parts of a first product (3: there is an fp32 result)
constexpr int kUpThreads = 256, kUpWarps = kUpThreads / 32, kUpUnit = 64;

template <int BASE, int P>
__global__ void __launch_bounds__(kUpThreads, 2) adapters_up_kernel(const __grid_constant__ AdapterParams p) {
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const Tile* tiles;
    int n_tiles;
    if (p.tokens <= kFewTokens) {
        FewTiles& s = *reinterpret_cast<FewTiles*>(smem);
        n_tiles = make_tiles(p, s);
        tiles = s.tile;
    } else {
        const Lists l = lists_of(p.tiles, p.tokens, p.num);
        n_tiles = l.counts[0];
        tiles = l.small;
    }
    const int R = p.rank, N = p.N;
    const unsigned units = (N + kUpUnit - 1) / kUpUnit, items = n_tiles * units;    // fits: a launch of more is refused
    const size_t step = (size_t)p.parts * R;
    bool waited = false;
    for (unsigned item = blockIdx.x * kUpWarps + warp; item < items; item += gridDim.x * kUpWarps) {
        const Tile& tile = tiles[item / units];
        const int n0 = (int)(item % units) * kUpUnit, n = n0 + 8 * c;
        const int ad = tile.adapter, r = tile.rank, t0 = tile.at(g), t1 = tile.at(g + 8);
        const bool whole = n0 + kUpUnit <= N, wide = whole && p.wide;
        uint4 base[2][2][BASE == 2 ? 2 : 1];             // [row][32 columns]: eight of this lane
        if (BASE != 0 && wide) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if ((h ? t1 : t0) < 0) continue;
                const char* from = row_ptr(p.base, h ? t1 : t0) + (size_t)n * (BASE == 2 ? 4 : 2);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    base[h][u][0] = ldg128(from + u * (BASE == 2 ? 128 : 64));
                    if (BASE == 2) base[h][u][BASE == 2] = ldg128(from + u * 128 + 16);
                }
            }
        }
        // the parts of these columns: more than one only at a part's end
        const int first = part_of(p, n0), last = part_of(p, min(n0 + kUpUnit, N) - 1);
        float d[8][4] = {};                  // [product][row g: 2 columns, row g + 8: 2 columns]
        const int col = n0 + (g >> 1) * 8 + (g & 1);     // of product 0; the others' are 2, 4, 6, 32, .. further
        const uint16_t* b = p.b + ((size_t)max(ad, 0) * N + col) * R + 4 * c;
        const uint16_t *low0 = p.low + (size_t)max(t0, 0) * P * step + 4 * c, *low1 = p.low + (size_t)max(t1, 0) * P * step + 4 * c;
        for (int r0 = 0; r0 < r; r0 += 16) {
            const bool in = r0 + 4 * c < r;
            uint2 w[8];
            if (whole) {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = in ? ldg64(b + (2 * (i & 3) + 32 * (i >> 2)) * R + r0) : make_uint2(0, 0);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = 2 * (i & 3) + 32 * (i >> 2);
                    w[i] = in && col + at < N ? ldg64(b + at * R + r0) : make_uint2(0, 0);
                }
            }
            if (!waited) {
                griddep_wait();
                griddep_launch_dependents();
                waited = true;
            }
            if (r0 + 16 > r) {               // what lies past the rank is nobody's
                const uint2 m = rank_mask(r0 + 4 * c, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = make_uint2(w[i].x & m.x, w[i].y & m.y);
            }
            for (int pt = first; pt <= last; ++pt) {
                uint2 a0[P], a1[P];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    a0[j] = in && t0 >= 0 ? ldg64(low0 + j * step + pt * R + r0) : make_uint2(0, 0);
                    a1[j] = in && t1 >= 0 ? ldg64(low1 + j * step + pt * R + r0) : make_uint2(0, 0);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // the columns of this part: 16 are brought by the lanes of four g
                    const int at = n0 + 32 * (i >> 2) + (g >= 4 ? 16 : 0);
                    const bool mine = first == last || (at < p.part_end[pt] && (pt == 0 || at >= p.part_end[pt - 1]));
                    const uint2 v = mine ? w[i] : make_uint2(0, 0);
#pragma unroll
                    for (int j = 0; j < P; ++j) mma_bf16_16816(d[i], a0[j].x, a1[j].x, a0[j].y, a1[j].y, v.x, v.y);
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
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) odd = fmaf(d[i][k], 0.f, odd);
        const bool put = ad >= 0 || !p.in_place, put32 = P == 3 && (ad >= 0 || !p.in_place32);
#pragma unroll
        for (int h = 0; h < 2; ++h) {        // rows t0 and t1
            const int t = h ? t1 : t0;
            if (t < 0) continue;
            char *to = row_ptr(p.y, t), *to32 = row_ptr(p.y32, t);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int at = n + 32 * u;
                float v[8], from[8] = {};
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = d[4 * u + (k >> 1)][2 * h + (k & 1)];
                if (odd != odd) plain_up<P>(p, p.low + (size_t)t * P * step, 1.f, p.b + (size_t)max(ad, 0) * N * R, at, r, v);
                if (BASE != 0) {
                    if (!wide) {
                        load_cols(row_ptr(p.base, t), BASE == 2, at, N, false, from);
                    } else if (BASE == 1) {
                        const uint4 x = base[h][u][0];
                        bf16x2_to_f32(x.x, from[0], from[1]);
                        bf16x2_to_f32(x.y, from[2], from[3]);
                        bf16x2_to_f32(x.z, from[4], from[5]);
                        bf16x2_to_f32(x.w, from[6], from[7]);
                    } else {
                        const uint4 x = base[h][u][0], y = base[h][u][BASE == 2];
                        const uint32_t q[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int k = 0; k < 8; ++k) from[k] = __uint_as_float(q[k]);
                    }
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] += from[k];
                if (put) put_cols(to, false, at, N, wide, v);
                if (put32) put_cols(to32, true, at, N, wide, v);
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
constexpr int kBigCols = 256;            // rows of A of one CTA, at most

struct BigSmem {
    int cols, stage, stages, total;      // columns of the accumulator, bytes of a stage, stages, bytes of all
};
__host__ __device__ inline BigSmem big_smem(int columns) {
    BigSmem s;
    s.cols = (columns < kBigCols ? columns + 15 : kBigCols) / 16 * 16;
    s.stage = (kBigTile + s.cols) * 128;
    s.stages = (224 * 1024) / s.stage;       // 4 to 12; four hold the sums, 128 x (cols + 4) x 4 bytes, too
    if (s.stages > 6) s.stages = 6;
    s.total = 1024 + s.stages * s.stage + 256;
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
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u, bars = base + shape.stages * shape.stage;
    const uint32_t slot = bars + 8 * shape.stages;
    const int stages = shape.stages;
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
        for (int i = 0; i < stages; ++i) mbar_init(bars + 8 * i, 1);
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
    // the stage that the next step's products read, how often it has been read, and its place
    int stage = 0, parity = 0;
    bool dead = false;                   // a wait gave up: the CTA goes on with the cluster, without its copies and products
    for (int ti = blockIdx.y; ti < n_tiles; ti += gridDim.y) {
        const BigTile tile = l.big[ti];
        if (tile.adapter < 0) continue;
        const int r = tile.rank;
        // What this thread copies: a 16-byte chunk of four rows of x and of every 32nd row of A.  Rows that are not
        // there are zeros in every stage, written once: no copy touches them.
        const char* xr[kBigTile / 32];
#pragma unroll
        for (int i = 0; i < kBigTile / 32; ++i) {
            const int row = row0 + 32 * i;
            xr[i] = row < tile.count ? row_ptr(p.x, l.order[tile.first + row]) + 16 * chunk + s0 * 128 : nullptr;
        }
        const char* ar = reinterpret_cast<const char*>(p.a + ((size_t)tile.adapter * SR + j0 + row0) * K) + 16 * chunk + s0 * 128;
        const size_t a32 = (size_t)K * 64;
        unsigned mine = 0;
        for (int i = 0; 32 * i + row0 < cols; ++i) mine |= ((j0 + 32 * i + row0) % p.rank < r ? 1u : 0u) << i;
        for (int i = 0; i < stages; ++i) {
            const uint32_t to = base + i * shape.stage + put;
#pragma unroll
            for (int j = 0; j < kBigTile / 32; ++j)
                if (!xr[j]) sts128(to + j * 4096, 0, 0, 0, 0);
            for (int j = 0; 32 * j + row0 < shape.cols; ++j)
                if (!(mine >> j & 1)) sts128(to + kBigTile * 128 + j * 4096, 0, 0, 0, 0);
        }
        // step s of this tile into the stage at `to`
        auto load = [&](int s, uint32_t to) {
            const int off = s * 128;
            const char* from = ar + off;
            to += put;
            if ((s0 + s + 1) * 64 <= K) {
#pragma unroll
                for (int i = 0; i < kBigTile / 32; ++i)
                    if (xr[i]) copy16_async(to + i * 4096, xr[i] + off, 16);
                to += kBigTile * 128;
#pragma unroll
                for (int i = 0; i < kBigCols / 32; ++i) {
                    if (mine >> i & 1) copy16_async(to + i * 4096, from, 16);
                    from += a32;
                }
            } else {                     // the last step of K ends early
                const int bytes = (s0 + s) * 64 + 8 * chunk < K ? 16 : 0;
#pragma unroll
                for (int i = 0; i < kBigTile / 32; ++i)
                    if (xr[i]) copy16_async(to + i * 4096, bytes ? xr[i] + off : p.x.ptr, bytes);
                to += kBigTile * 128;
                for (int i = 0; i < kBigCols / 32; ++i)
                    if (mine >> i & 1) copy16_async(to + i * 4096, bytes ? from + i * a32 : p.x.ptr, bytes);
            }
        };
        bool bad = dead;
        int fill = stage;                // the stage that the next copies go to
        for (int s = 0; s < stages - 1; ++s) {
            if (s < n && !dead) load(s, base + (uint32_t)fill * shape.stage);
            if (++fill == stages) fill = 0;
            copies_commit();
        }
        int before = 0, parity_before = 0;       // of step s - 1
        for (int s = 0; s < n; ++s) {
            if (stages == 4) copies_wait<2>();
            else if (stages == 5) copies_wait<3>();
            else copies_wait<4>();
            fence_async_smem();
            if (__syncthreads_or(bad)) break;
            if (tid == 0) {
                tc_fence_after_sync();
                const uint32_t at = base + (uint32_t)stage * shape.stage;
                const uint64_t xa = umma_desc_sw128(at), wa = umma_desc_sw128(at + kBigTile * 128);
#pragma unroll
                for (int k = 0; k < 4; ++k) umma_bf16(tmem, xa + 2 * k, wa + 2 * k, idesc, s > 0 || k > 0);
                umma_commit(bars + 8 * stage);
            }
            const int next = s + stages - 1;
            if (next < n) {
                // the stage of step s - 1 is free once its products have read it
                if (s > 0) bad = !mbar_wait_bounded(bars + 8 * before, parity_before, p.wait, kErrConsumerWait);
                if (!bad) load(next, base + (uint32_t)fill * shape.stage);
                if (++fill == stages) fill = 0;
            }
            copies_commit();
            before = stage;
            parity_before = parity;
            if (++stage == stages) stage = 0, parity ^= 1;
        }
        if (!bad) bad = !mbar_wait_bounded(bars + 8 * before, parity_before, p.wait, kErrConsumerWait);
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
                float4 w[kMaxSplits];
#pragma unroll
                for (int q = 0; q < kMaxSplits; ++q)
                    if (q < splits) w[q] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(sums, q) + t * pitch + j);
#pragma unroll
                for (int q = 0; q < kMaxSplits; ++q) {
                    if (q >= splits) break;
                    v.x += w[q].x; v.y += w[q].y; v.z += w[q].z; v.w += w[q].w;
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

// Second product of big tiles, out[t][n] = base[t][n] + sum_r low[t][r] B[n][r] for 128 tokens and blocks of 64
// columns: bound by base and out.  A block is one product on the tensor cores, 128 x 64 over r and the parts of
// the first products, which lie in shared memory as bf16 operands; B's rows come a few blocks ahead into a
// ring, base a block ahead into registers, and while a block is multiplied the one before leaves tensor
// memory.  The rows of B are put into the order that gives a lane eight consecutive columns (as above).
// All tiles' blocks are dealt to the CTAs in equal runs.
constexpr int kUpBlock = 64, kUpRing = 3, kUpCtas = 2, kUpTmem = 2 * kUpBlock;
static_assert(kUpCtas * kUpTmem <= 512, "tensor memory of an SM");

// A: parts of 128 rows, B: ring stages of 64, each in pieces of 64 r with rows of 128 bytes, swizzled.
__host__ __device__ inline int up_big_smem(int rank, int parts) {
    const int pieces = (rank + 63) / 64;
    return 1024 + (parts * kBigTile + kUpRing * kUpBlock) * 128 * pieces + 64;
}

// Blocks of columns, each in one part.
__device__ __forceinline__ int part_blocks(const AdapterParams& p, int part) {
    return (p.part_end[part] - (part ? p.part_end[part - 1] : 0) + kUpBlock - 1) / kUpBlock;
}

// 64 columns of 16 rows of tensor memory, as the products of mma.m16n8 lie: v[i] has columns 8 i + 2 c and + 1 of
// rows g and g + 8.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t taddr, float (&v)[8][4]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(&v[0][0]);
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x8.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}

// BASE 0: none, or rows that do not allow wide accesses, 1: bf16, 2: fp32; P: parts of a first product
template <int BASE, int P>
__global__ void __launch_bounds__(kUpThreads, kUpCtas) adapters_up_big_kernel(const __grid_constant__ AdapterParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const Lists l = lists_of(p.tiles, p.tokens, p.num);
    const int R = p.rank, N = p.N, pieces = (R + 63) / 64;
    const uint32_t a_at = (smem_u32(raw) + 1023u) & ~1023u, ring = a_at + P * kBigTile * 128 * pieces;
    const uint32_t stage_bytes = kUpBlock * 128 * pieces, bars = ring + kUpRing * stage_bytes, slot = bars + 16;
    // the first products are there: the kernel before this one let it start after it had waited for them
    const int n_tiles = l.counts[1];
    int blocks = 0;
    for (int i = 0; i < p.parts; ++i) blocks += part_blocks(p, i);
    const long long all = (long long)n_tiles * blocks;
    long long at = all * blockIdx.x / gridDim.x;
    const long long end = all * (blockIdx.x + 1) / gridDim.x;
    if (at == end) {
        griddep_launch_dependents();
        griddep_wait();
        return;
    }
    if (warp == 0) tmem_alloc(slot, kUpTmem);
    if (tid == 0) {
        mbar_init(bars, 1);
        mbar_init(bars + 8, 1);
        fence_mbarrier_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // only now: a kernel after this one that allocates tensor memory before it waits must find this one's taken
    griddep_launch_dependents();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot));
    const uint32_t idesc = umma_idesc_bf16(kUpBlock);
    const int row0 = 32 * (warp & 3) + 16 * (warp >> 2);        // this warp's rows of the tile
    const size_t step = (size_t)p.parts * R;
    unsigned made = 0;                   // products so far: the next one's accumulator and phase
    bool bad = false;
    while (at < end && !bad) {
        // a run of blocks of one tile and part: columns n0 on, the part ends at n_end
        const BigTile tile = l.big[at / blocks];
        int b0 = (int)(at % blocks), part = 0, n_end = p.part_end[0], n0 = 0;
        for (int n; b0 >= (n = part_blocks(p, part)); n_end = p.part_end[++part]) {
            b0 -= n;
            n0 = n_end;
        }
        const int runs = (int)min((long long)(part_blocks(p, part) - b0), end - at);
        n0 += b0 * kUpBlock;
        at += runs;
        const int ad = tile.adapter, r = tile.rank, steps = (r + 15) / 16;
        const float scale = ad >= 0 && p.scale ? p.scale[ad] : 1.f;
        const bool active = row0 < tile.count;
        const int i0 = row0 + g, i1 = i0 + 8;
        const int t0 = i0 < tile.count ? l.order[tile.first + i0] : -1, t1 = i1 < tile.count ? l.order[tile.first + i1] : -1;
        const uint16_t* b = p.b + (size_t)max(ad, 0) * N * R;
        const bool put = ad >= 0 || !p.in_place, put32 = P == 3 && (ad >= 0 || !p.in_place32);
        const char *from0 = row_ptr(p.base, max(t0, 0)) + (size_t)(n0 + 8 * c) * (BASE == 2 ? 4 : 2);
        const char *from1 = row_ptr(p.base, max(t1, 0)) + (size_t)(n0 + 8 * c) * (BASE == 2 ? 4 : 2);
        char *to0 = row_ptr(p.y, max(t0, 0)) + (size_t)(n0 + 8 * c) * 2, *to1 = row_ptr(p.y, max(t1, 0)) + (size_t)(n0 + 8 * c) * 2;
        // B's rows of a block, four threads a row, into its ring stage; what lies past the rank or the part
        // arrives as zeros
        const int b_row = tid >> 2, b_col = (b_row >> 5) * 32 + ((b_row & 7) >> 1) * 8 + (b_row >> 3 & 3) * 2 + (b_row & 1);
        const uint16_t* b_from = b + (size_t)(n0 + b_col) * R + 8 * (tid & 3);
        const size_t b_step = (size_t)kUpBlock * R;
        const uint32_t b_to = ring + b_row * 128;
        int b_left = n_end - n0 - b_col, b_stage = 0;    // the part's columns from this thread's of the next block on
        auto load = [&]() {              // the next block
            if (r > 0 && b_left > -kUpBlock) {
                const uint32_t to = b_to + (uint32_t)b_stage * stage_bytes;
#pragma unroll 2
                for (int i = tid & 3, j = 0; i < 2 * steps; i += 4, j += 32) {
                    const int bytes = b_left > 0 ? min(2 * (r - 8 * i), 16) : 0;
                    copy16_async(to + (i >> 3) * (kUpBlock * 128) + 16 * ((i & 7) ^ (b_row & 7)), bytes > 0 ? b_from + j : p.b, max(bytes, 0));
                }
            }
            if (++b_stage == kUpRing) b_stage = 0;
            b_left -= kUpBlock;
            b_from += b_step;
            copies_commit();
        };
        // The tile's first products of a part, two threads a row
        auto take = [&]() {
            const int row = tid >> 1;
            const float* low = p.low_big + (size_t)(tile.first + min(row, tile.count - 1)) * step + part * R;
            for (int i = tid & 1; i < 2 * steps; i += 2) {
                float v[8] = {};
                if (row < tile.count && 8 * i < r) {     // (8 i + 8 is within the row)
                    const float4 x = ld_cg_f32x4(low + 8 * i), y = ld_cg_f32x4(low + 8 * i + 4);
                    v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
                    v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
                }
                uint32_t out[P][4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool in0 = 8 * i + 2 * k < r, in1 = 8 * i + 2 * k + 1 < r;
                    uint32_t s[P];
                    split(in0 ? v[2 * k] * scale : 0.f, in1 ? v[2 * k + 1] * scale : 0.f, s);
#pragma unroll
                    for (int j = 0; j < P; ++j) out[j][k] = s[j];
                }
#pragma unroll
                for (int j = 0; j < P; ++j)
                    sts128(a_at + (j * pieces + (i >> 3)) * (kBigTile * 128) + row * 128 + 16 * ((i & 7) ^ (row & 7)), out[j][0],
                           out[j][1], out[j][2], out[j][3]);
            }
        };
        uint4 base[2][2][BASE == 2 ? 2 : 1];     // [row][32 columns]: eight columns of this lane
        auto fetch = [&](int i) {        // of block i
            if (BASE == 0 || !active || i >= runs || n0 + (i + 1) * kUpBlock > n_end) return;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if ((h ? t1 : t0) < 0) continue;
                const char* from = (h ? from1 : from0) + (size_t)i * (kUpBlock * (BASE == 2 ? 4 : 2));
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    base[h][v][0] = ldg128(from + v * (BASE == 2 ? 128 : 64));
                    if (BASE == 2) base[h][v][BASE == 2] = ldg128(from + v * 128 + 16);
                }
            }
        };
        // The results of block i, whose product (if there is one) has accumulator `acc`
        auto finish = [&](int i, unsigned acc) {
            if (!active) return;
            float d[8][4] = {};
            if (r > 0) {
                tmem_ld_16x64(tmem + ((uint32_t)row0 << 16) + acc * kUpBlock, d);
                tmem_wait_ld();
            }
            float odd = 0.f;             // NaN if any sum is, or infinite
#pragma unroll
            for (int k = 0; k < 8; ++k)
#pragma unroll
                for (int j = 0; j < 4; ++j) odd = fmaf(d[k][j], 0.f, odd);
            const bool wide = n0 + (i + 1) * kUpBlock <= n_end && p.wide;
            if (wide && odd == odd) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        if (BASE == 1) {
                            const uint4 x = base[h][v][0];
                            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float lo, hi;
                                bf16x2_to_f32(w[j], lo, hi);
                                d[4 * v + j][2 * h] += lo;
                                d[4 * v + j][2 * h + 1] += hi;
                            }
                        } else if (BASE == 2) {
                            const uint4 x = base[h][v][0], y = base[h][v][BASE == 2];
                            const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                            for (int j = 0; j < 8; ++j) d[4 * v + (j >> 1)][2 * h + (j & 1)] += __uint_as_float(w[j]);
                        }
                    }
                fetch(i + 1);            // base is in the sums: the next block's may come
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if ((h ? t1 : t0) < 0) continue;
                    char* to = (h ? to1 : to0) + (size_t)i * (kUpBlock * 2);
                    char* to32 = P == 3 ? row_ptr(p.y32, h ? t1 : t0) + (size_t)(n0 + i * kUpBlock + 8 * c) * 4 : nullptr;
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        float x[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = d[4 * v + (j >> 1)][2 * h + (j & 1)];
                        if (put) row_store8(to, false, 32 * v, x);
                        if (put32) row_store8(to32, true, 32 * v, x);
                    }
                }
            } else {
                // the part's last columns, rows that do not allow wide accesses, or NaN
                const float* low = p.low_big + (size_t)(tile.first + i0) * step;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const int t = h ? t1 : t0, n = n0 + i * kUpBlock + 32 * v + 8 * c;
                        if (t < 0 || n >= n_end) continue;
                        float x[8], from[8] = {};
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = d[4 * v + (j >> 1)][2 * h + (j & 1)];
                        if (odd != odd) plain_up<0>(p, low + (h ? 8 * step : 0), scale, b, n, r, x);
                        if (p.base.ptr) load_cols(row_ptr(p.base, t), p.base.f32, n, n_end, wide, from);
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] += from[j];
                        if (put) put_cols(row_ptr(p.y, t), false, n, n_end, wide, x);
                        if (put32) put_cols(row_ptr(p.y32, t), true, n, n_end, wide, x);
                    }
                fetch(i + 1);
            }
        };
        load();
        load();
        fetch(0);
        if (r > 0) take();
        for (int i = 0; i <= runs; ++i) {
            if (r > 0) {
                copies_wait<kUpRing - 2>();
                // the product before has read its operands: they may be replaced
                if (i > 0 && !bad)
                    bad = !mbar_wait_bounded(bars + 8 * ((made - 1) & 1), ((made - 1) >> 1) & 1, p.wait, kErrConsumerWait);
                fence_async_smem();
                tc_fence_before_sync();
                bad = __syncthreads_or(bad);
                tc_fence_after_sync();
                if (bad) break;
                if (i < runs) {
                    if (tid == 0) {
                        const uint32_t bt = ring + (uint32_t)(i % kUpRing) * stage_bytes;
                        for (int j = 0; j < P; ++j)
                            for (int q = 0; q < steps; ++q)
                                umma_bf16(tmem + (made & 1) * kUpBlock,
                                          umma_desc_sw128(a_at + (j * pieces + (q >> 2)) * (kBigTile * 128)) + 2 * (q & 3),
                                          umma_desc_sw128(bt + (q >> 2) * (kUpBlock * 128)) + 2 * (q & 3), idesc, j + q > 0);
                        umma_commit(bars + 8 * (made & 1));
                    }
                    load();
                    ++made;
                }
            }
            if (i > 0) finish(i - 1, (made - (i < runs ? 2 : 1)) & 1);
        }
        copies_wait<0>();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem, kUpTmem);
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
static size_t low_bytes(long long tokens, int rank, int parts) { return up256((size_t)tokens * rank * parts * 6); }
static size_t low_big_bytes(long long tokens, int rank, int parts) {
    return tokens > kFewTokens && rank <= kBigRank ? up256((size_t)tokens * rank * parts * 4) : 0;
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

static cudaError_t launch_small(const AdapterParams& p, long long tiles, int sm_count, cudaStream_t stream, bool up) {
    const size_t smem = p.tokens <= kFewTokens ? sizeof(FewTiles) : 0;
    if (up) {
        const long long ctas = (tiles * ((p.N + kUpUnit - 1) / kUpUnit) + kUpWarps - 1) / kUpWarps, most = 2LL * sm_count;
        const dim3 grid((unsigned)(ctas < most ? ctas : most)), block(kUpThreads);
        const int base = !p.base.ptr ? 0 : p.base.f32 ? 2 : 1;
        if (p.y32.ptr)
            return base == 0 ? launch_dependent(adapters_up_kernel<0, 3>, grid, block, smem, stream, p)
                   : base == 1 ? launch_dependent(adapters_up_kernel<1, 3>, grid, block, smem, stream, p)
                               : launch_dependent(adapters_up_kernel<2, 3>, grid, block, smem, stream, p);
        return base == 0 ? launch_dependent(adapters_up_kernel<0, 2>, grid, block, smem, stream, p)
               : base == 1 ? launch_dependent(adapters_up_kernel<1, 2>, grid, block, smem, stream, p)
                           : launch_dependent(adapters_up_kernel<2, 2>, grid, block, smem, stream, p);
    }
    // Eight CTAs share K while all of them find places, two to an SM in whole clusters (128 SMs of which do),
    // four beyond
    // (of one part, so that sums do not depend on how many parts there are)
    const long long groups = (p.rank + 15) / 16, items = tiles * p.parts * groups;
    const int size = tiles * groups * kLowCluster <= 2 * 128 ? kLowCluster : kLowCluster / 2;
    const long long most = 2LL * sm_count / size;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = size;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((items < most ? items : most) * size));
    cfg.blockDim = dim3(kLowThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, adapters_low_kernel, p);
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

template <int BASE, int P>
static cudaError_t launch_up_big(const AdapterParams& p, int sm_count, cudaStream_t stream) {
    const int smem = up_big_smem(p.rank, P);
    const cudaError_t e = raise_smem(adapters_up_big_kernel<BASE, P>, smem);
    if (e != cudaSuccess) return e;
    int ctas = 228 * 1024 / (smem + 1024);
    ctas = ctas > kUpCtas ? kUpCtas : ctas;
    return launch_dependent(adapters_up_big_kernel<BASE, P>, dim3(ctas * sm_count), dim3(kUpThreads), smem, stream, p);
}

template <int P>
static cudaError_t launch_up_big_base(const AdapterParams& p, int sm_count, cudaStream_t stream) {
    if (!p.base.ptr || !p.wide) return launch_up_big<0, P>(p, sm_count, stream);
    return p.base.f32 ? launch_up_big<2, P>(p, sm_count, stream) : launch_up_big<1, P>(p, sm_count, stream);
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
    p.low = reinterpret_cast<uint16_t*>(scratch);
    p.low_big = reinterpret_cast<float*>(scratch + low_bytes(tokens, p.rank, p.parts));
    p.tiles = reinterpret_cast<int*>(scratch + low_bytes(tokens, p.rank, p.parts) + low_big_bytes(tokens, p.rank, p.parts));
    p.big_from = p.rank <= kBigRank ? kBigFrom : 0x7fffffff;
    p.index = index;
    p.tokens = tokens;
    p.in_place = same_rows(p.y, p.base);
    p.in_place32 = p.y32.ptr && same_rows(p.y32, p.base);
    p.wide = true;
    for (const Rows* r : {&p.base, &p.y, &p.y32})
        if (r->ptr) p.wide = p.wide && rows_aligned16(*r, tokens);
    const long long small = tokens <= kFewTokens ? tokens : max_small(tokens, p.num);
    if (small * ((N + 15) / 16) > 0x7fff0000LL || small * p.parts * ((p.rank + 15) / 16) > 0x7fff0000LL)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "tokens=%d with N=%d exceed one launch", tokens, N);
    HostDevice dev;
    if ((s = host_device(dev)) != DL_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.wait = WaitCtl{dev.err_word, dev.wait_limit_ns};
    cudaError_t e;
    if (tokens <= kFewTokens) {
        if ((e = launch_small(p, small, dev.sm_count, st, false)) == cudaSuccess)
            e = launch_small(p, small, dev.sm_count, st, true);
    } else {
        // Each list's kernels find how much there is on the device.  Both first products may run at the
        // same time, then both second ones.
        const long long big = max_big(tokens, p.num);
        const size_t counters = (size_t)(p.num + 1) * 4;
        if ((e = raise_smem(sort_tokens_kernel, counters)) == cudaSuccess)
            e = launch_dependent(sort_tokens_kernel, dim3(1), dim3(1024), counters, st, p);
        if (e == cudaSuccess) e = launch_small(p, small, dev.sm_count, st, false);
        if (e == cudaSuccess && p.rank <= kBigRank) e = launch_low_big(p, big, dev.sm_count, st);
        if (e == cudaSuccess) e = launch_small(p, small, dev.sm_count, st, true);
        if (e == cudaSuccess && p.rank <= kBigRank)
            e = p.y32.ptr ? launch_up_big_base<3>(p, dev.sm_count, st) : launch_up_big_base<2>(p, dev.sm_count, st);
    }
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "linear_adapters launch: %s", cudaGetErrorString(e));
    return host_ok();
}
