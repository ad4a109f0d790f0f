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
constexpr int kBigFrom = 64;             // tokens in a row of one adapter from which on they go in big tiles
// Tokens of one adapter in no order: 40, and as many as make this times all tokens and the rank (8192 -> 8192, in small
// tiles and in big ones: 4096 tokens, 64 of each adapter, rank 16, 32, 64: 99 and 115, 122 and 116, 157 and 119 us; 128 of
// each: 95 and 76, 116 and 78, 150 and 82; rank 64, 1000 tokens, 125 of each: 48 and 39, 300, 150 of each: 22 and 32).
constexpr int kListFrom = 40;
constexpr long long kListWork = 6LL << 20;
static_assert(kListFrom <= kBigFrom && 2 * kListFrom <= kBigTile, "max_big");
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
    int big_from, list_from; // tokens from which on there are big tiles: in a row, in no order (ranks too large: none)
    bool in_place, in_place32;   // base is y, y32: rows without an adapter stay as they are
    bool wide;               // groups of eight columns of base, y and y32 are 16-byte aligned
    // big tiles
    float* low_big;          // [tokens][parts * rank] first products without scale
    int withhold;            // test hook: CTA 0 of each product never copies its k-th stage (0: none)
    WaitCtl wait;
};

// Up to kTile tokens of one adapter.
struct Tile {
    int adapter, rank, count;    // adapter -1, rank 0: tokens without one
    float scale;
    int token[kTile];
    __device__ int at(int i) const { return i < count ? token[i] : -1; }
};
// Up to kBigTile tokens of one adapter: first .. first + count - 1, or, first < 0, those that the list `order` names
// from ~first on.
struct BigTile {
    int adapter, first, count, rank;
};

// The lists of more than kFewTokens tokens.
struct Lists {
    int *counts;             // small tiles, big tiles
    int* start;              // [tokens + 1] where the adapter changes
    int* order;              // [tokens] of big tiles whose tokens are not in a row
    BigTile* big;
    Tile* small;
};
// (each adapter's, or each run's, n tokens make ceil(n / kBigTile) <= n / kListFrom of them)
__host__ __device__ inline long long max_big(long long tokens) { return tokens / kListFrom + 1; }
__host__ __device__ inline long long max_small(long long tokens, int num) {
    return tokens / kTile + (tokens < num + 1 ? tokens : num + 1) + 1;
}
__host__ __device__ inline Lists lists_of(int* at, long long tokens) {
    Lists l;
    l.counts = at;
    l.big = reinterpret_cast<BigTile*>(at + 4);
    l.start = reinterpret_cast<int*>(l.big + max_big(tokens));
    l.order = l.start + tokens + 1;
    l.small = reinterpret_cast<Tile*>(l.order + tokens);
    return l;
}
// Token `row` of a big tile.
__device__ __forceinline__ int token_of(const Lists& l, const BigTile& t, int row) {
    return t.first >= 0 ? t.first + row : l.order[~t.first + row];
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

// The lists of many tokens, by one CTA.  Tokens of one adapter in a row, enough of them, make big tiles; the
// others are sorted by adapter (counted, then placed): an adapter that has enough of them left gets big tiles
// with a list of its tokens, one that has fewer small tiles.  Which tokens of an adapter share a tile, and their
// order in it, do not change any result.
constexpr int kStartsHere = 8192;        // tokens whose runs' starts fit shared memory beside the counts
__global__ void __launch_bounds__(1024) sort_tokens_kernel(const __grid_constant__ AdapterParams p) {
    extern __shared__ int count[];       // of each adapter, then its next place; the last: without one
    __shared__ int warp_sum[2][32];
    Scan scan{warp_sum};
    const int tid = threadIdx.x, T = p.tokens;
    int total;
    const Lists l = lists_of(p.tiles, T);
    int* start = T <= kStartsHere ? count + p.num + 1 : l.start;
    griddep_wait();
    griddep_launch_dependents();
    for (int i = tid; i <= p.num; i += 1024) count[i] = 0;
    // where the adapter changes, four tokens in a row a thread
    int runs = 0;
    for (long long t0 = 4LL * tid; t0 - 4 * tid < T; t0 += 4096) {
        int a[5];
#pragma unroll
        for (int k = 0; k < 5; ++k) {
            const long long t = t0 + k - 1;
            a[k] = t >= 0 && t < T ? adapter_of(p, (int)t) : -2;
        }
        int mine = 0;
        bool starts[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            starts[k] = t0 + k < T && a[k + 1] != a[k];
            mine += starts[k];
        }
        int at = runs + scan(mine, total) - mine;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (starts[k]) start[at++] = (int)(t0 + k);
        runs += total;
    }
    if (tid == 0) start[runs] = T;
    __syncthreads();
    int big = 0;
    for (int i0 = 0; i0 < runs; i0 += 1024) {
        const int i = i0 + tid;
        int mine = 0, first = 0, n = 0, ad = -1;
        if (i < runs) {
            first = start[i];
            n = start[i + 1] - first;
            ad = adapter_of(p, first);
            if (n >= p.big_from) mine = (n + kBigTile - 1) / kBigTile;
            else atomicAdd(&count[ad < 0 ? p.num : ad], n);
        }
        const int r = mine ? rank_of(p, ad) : 0;
        BigTile* to = l.big + big + scan(mine, total) - mine;
        for (int j = 0; j < mine; ++j) to[j] = BigTile{ad, first + j * kBigTile, min(n - j * kBigTile, kBigTile), r};
        big += total;
    }
    __syncthreads();
    // an adapter's places: in small tiles, or (~place) in the list that big ones name
    int small = 0, listed = 0;
    for (int i0 = 0; i0 <= p.num; i0 += 1024) {
        const int i = i0 + tid, n = i <= p.num ? count[i] : 0, ad = i < p.num ? i : -1;
        const bool gathered = ad >= 0 && n >= p.list_from;
        const int mine = gathered ? 0 : (n + kTile - 1) / kTile, mine_big = gathered ? (n + kBigTile - 1) / kBigTile : 0;
        const int first = small + scan(mine, total) - mine, r = n ? rank_of(p, ad) : 0;
        small += total;
        const int place = listed + scan(gathered ? n : 0, total) - (gathered ? n : 0);
        listed += total;
        const float scale = mine ? scale_of(p, ad) : 1.f;
        for (int j = 0; j < mine; ++j) {
            Tile& tile = l.small[first + j];
            tile.adapter = ad;
            tile.rank = r;
            tile.scale = scale;
            tile.count = min(n - j * kTile, kTile);
        }
        BigTile* to = l.big + big + scan(mine_big, total) - mine_big;
        big += total;
        for (int j = 0; j < mine_big; ++j) to[j] = BigTile{ad, ~(place + j * kBigTile), min(n - j * kBigTile, kBigTile), r};
        if (i <= p.num) count[i] = gathered ? ~place : first * kTile;
    }
    __syncthreads();
    for (int i = tid; i < runs; i += 1024) {
        const int first = start[i], n = start[i + 1] - first;
        if (n >= p.big_from) continue;
        const int ad = adapter_of(p, first);
        int& next = count[ad < 0 ? p.num : ad];
        if (*(volatile int*)&next < 0) {                 // (which of the two it is never changes)
            const int at = ~atomicSub(&next, n);
            for (int k = 0; k < n; ++k) l.order[at + k] = first + k;
        } else {
            const int at = atomicAdd(&next, n);
            for (int k = 0; k < n; ++k) l.small[(at + k) / kTile].token[(at + k) % kTile] = first + k;
        }
    }
    if (tid == 0) {
        l.counts[0] = small;
        l.counts[1] = big;
    }
}

// ---------------------------------------------------------------- parts

// The fp32 first products go into the second ones as two bf16 parts (2^-17 of the value is lost: the first
// leaves half its step at most, 2^-8 of the value, which the second holds; of anything less it loses 2^-9), three (24
// bits: nothing) where an fp32 result is asked for.  The parts of a value and their products can
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

// One value's three parts.  A finite one beyond bf16's largest number and half a step, where split() rounds the first part
// to an infinity, begins with that number.  Where three are taken, its second one is cut, not rounded: 8 bits each
// hold all 24.  Of two the second is cut only where both would add up to 2^128, within 2^-17 of fp32's largest
// number, and 2^-16 of the value is lost.
__device__ __forceinline__ void split_one(float a, bool three, uint32_t (&v)[3]) {
    const bool large = fabsf(a) <= 3.4028235e38f && fabsf(a) >= 0x1.ffp127f;
    v[0] = large ? __float_as_uint(a) >> 16 : f32x2_to_bf16x2(a, 0.f);
    a -= __uint_as_float(v[0] << 16);
    v[1] = f32x2_to_bf16x2(a, 0.f);
    if (large && (three || fabsf(__uint_as_float(v[1] << 16)) >= 0x1p120f)) v[1] = __float_as_uint(a) >> 16;
    v[2] = f32x2_to_bf16x2(a - __uint_as_float(v[1] << 16), 0.f);
}

// ---------------------------------------------------------------- small tiles: first product

// low[t][j] = scale * sum_k A[j][k] x[t][k], as the bf16 parts that the second product takes: a cluster of CTAs
// shares K, a warp takes 16 rows of A and a tile's 16 tokens over its part of K.  A (and x) go from global
// memory straight into the operands of mma.m16n8k16: the sum over k may take its terms in any order, so
// a lane's 16-byte load of 8 consecutive k is the k-slots that it holds in two products.  Bound by the latency of
// its chain (index, list, A and x, joins): 6 to 9 us of 16 tokens, K 29568, and of 256, K 8192, of 64 adapters.
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
        const Lists l = lists_of(p.tiles, p.tokens);
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
                split_one(j < r ? all * tile.scale : 0.f, p.y32.ptr != nullptr, v);
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

// Four or eight consecutive r of a row, zeros if not `in`: the k-slots that a lane holds in one product or in two.
__device__ __forceinline__ void load_r(const uint16_t* p, bool in, uint2 (&v)[1]) { v[0] = in ? ldg64(p) : make_uint2(0, 0); }
__device__ __forceinline__ void load_r(const uint16_t* p, bool in, uint2 (&v)[2]) {
    const uint4 x = in ? ldg128(p) : make_uint4(0, 0, 0, 0);
    v[0] = make_uint2(x.x, x.y);
    v[1] = make_uint2(x.z, x.w);
}

// Small tiles: a warp takes 64 columns of a tile, 16 or 32 r at a time.  What does not depend on the first products
// (the tiles, base, B) is fetched before they are waited for: the kernel that makes them lets this one start only
// after it had waited for all earlier ones.  Bound by instructions and latencies: a tile of few tokens costs as
// much as one of 16, so each lane has all its loads of these r in flight at once.  Ranks up to 32 by 16, beyond by 32
// (250 tokens of 64 adapters, 8192 -> 8192: rank 16, 64, 128 21, 45, 78 us and 23, 39.5, 67).
// BASE 0: none, 1: bf16, 2: fp32; P: parts of a first product (3: there is an fp32 result); 16 Q r at a time
constexpr int kUpThreads = 256, kUpWarps = kUpThreads / 32, kUpUnit = 64;

template <int BASE, int P, int Q>
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
        const Lists l = lists_of(p.tiles, p.tokens);
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
        const uint16_t* b = p.b + ((size_t)max(ad, 0) * N + col) * R + 4 * Q * c;
        const uint16_t* low0 = p.low + (size_t)max(t0, 0) * P * step + 4 * Q * c;
        const uint16_t* low1 = p.low + (size_t)max(t1, 0) * P * step + 4 * Q * c;
        for (int r0 = 0; r0 < r; r0 += 16 * Q) {
            const int mine_from = r0 + 4 * Q * c;
            const bool in = mine_from < r;
            uint2 w[8][Q];
            if (whole) {
#pragma unroll
                for (int i = 0; i < 8; ++i) load_r(b + (2 * (i & 3) + 32 * (i >> 2)) * R + r0, in, w[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int at = 2 * (i & 3) + 32 * (i >> 2);
                    load_r(b + at * R + r0, in && col + at < N, w[i]);
                }
            }
            if (!waited) {
                griddep_wait();
                griddep_launch_dependents();
                waited = true;
            }
            if (r0 + 16 * Q > r) {           // what lies past the rank is nobody's
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const uint2 m = rank_mask(mine_from + 4 * q, r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i][q] = make_uint2(w[i][q].x & m.x, w[i][q].y & m.y);
                }
            }
            for (int pt = first; pt <= last; ++pt) {
                uint2 a0[P][Q], a1[P][Q];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    load_r(low0 + j * step + pt * R + r0, in && t0 >= 0, a0[j]);
                    load_r(low1 + j * step + pt * R + r0, in && t1 >= 0, a1[j]);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // the columns of this part: 16 are brought by the lanes of four g
                    const int at = n0 + 32 * (i >> 2) + (g >= 4 ? 16 : 0);
                    const bool mine = first == last || (at < p.part_end[pt] && (pt == 0 || at >= p.part_end[pt - 1]));
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const uint2 v = mine ? w[i][q] : make_uint2(0, 0);
#pragma unroll
                        for (int j = 0; j < P; ++j) mma_bf16_16816(d[i], a0[j][q].x, a1[j][q].x, a0[j][q].y, a1[j][q].y, v.x, v.y);
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

__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void fence_async_cluster() { asm volatile("fence.proxy.async.shared::cluster;" ::: "memory"); }

// One K step of 16 of two bf16 operands: kind::f16, fp32 accumulator, 128 rows, n columns.
__host__ __device__ constexpr uint32_t umma_idesc_bf16(int n) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void umma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
}

// First product of big tiles: low_big[token][j] = sum_k A[j][k] x[token][k], a product of 128 tokens
// and up to 256 rows of A on the tensor cores, the sums in tensor memory.  It is bound by what an SM reads
// from L2: a tile's x once, A once a tile.  One thread has x and A copied into 128-byte swizzled stages of 64 k,
// another one issues the products.  Where the tokens are not in a row, eight warps copy x in pieces of 16 bytes (30 us
// for 4096 tokens, K 8192, rank 64; by tile::gather4, four rows an instruction, 53; in a row 25).  A cluster shares
// K: each CTA leaves its sums in its shared memory, where the cluster's CTAs add them up, a share of the tokens
// each, always in the same order (left to the second product to add, they cost it 48 us more).  Rows of A past the
// rank, and of x past the tile, are read like the others: what they make are values that nobody takes.
constexpr int kBigWarps = 8, kBigThreads = 32 * (kBigWarps + 2);
constexpr int kBigCols = 256;            // rows of A of one CTA, at most

// 16 bytes into shared memory, zeros if not `in`; and waits for all but the last N groups of such.
__device__ __forceinline__ void copy16(uint32_t dst, const char* src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy16_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy16_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kBigStages = 224 * 1024;   // bytes of all stages, at most
struct BigSmem {
    int cols, stage, stages, total;      // columns of the accumulator, bytes of a stage, stages, bytes of all
};
__host__ __device__ inline BigSmem big_smem(int columns) {
    BigSmem s;
    s.cols = (columns < kBigCols ? columns + 15 : kBigCols) / 16 * 16;
    s.stage = (kBigTile + s.cols) * 128;
    s.stages = kBigStages / s.stage;         // 4 to 8; four hold the sums, 128 x (cols + 4) x 4 bytes, too
    if (s.stages > 8) s.stages = 8;
    s.total = 1024 + s.stages * s.stage + 256;
    return s;
}

__global__ void __launch_bounds__(kBigThreads) adapters_low_big_kernel(const __grid_constant__ CUtensorMap map_x,
                                                                       const __grid_constant__ CUtensorMap map_a,
                                                                       const __grid_constant__ AdapterParams p) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    extern __shared__ __align__(16) unsigned char raw[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int splits = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const Lists l = lists_of(p.tiles, p.tokens);
    const int SR = p.parts * p.rank, K = p.K;
    const BigSmem shape = big_smem(SR);
    const int stages = shape.stages;
    const uint32_t base = (smem_u32(raw) + 1023u) & ~1023u, bars = base + stages * shape.stage;
    const uint32_t full = bars, empty = bars + 8 * stages, copied = bars + 16 * stages, done = bars + 24 * stages, slot = done + 8;
    // The lists are complete and the buffers free: the kernel before this one let it start only after
    // it had waited for sort_tokens_kernel.  (Its own results are other ones; the wait is at the end.)
    const int n_tiles = l.counts[1];
    if ((int)blockIdx.y >= n_tiles) {
        griddep_launch_dependents();
        griddep_wait();
        return;
    }
    uint32_t tmem_cols = 32;
    while ((int)tmem_cols < shape.cols) tmem_cols *= 2;
    if (warp == 0) tmem_alloc(slot, tmem_cols);
    if (tid == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(empty + 8 * i, 1);
            mbar_init(copied + 8 * i, kBigWarps);
        }
        mbar_init(done, 1);
        fence_mbarrier_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    griddep_launch_dependents();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot));
    // this CTA's columns and part of K
    const int j0 = (int)blockIdx.z * kBigCols, cols = min(SR - j0, kBigCols);
    const int steps_all = (K + 63) / 64;
    const int s0 = (int)((long long)steps_all * rank / splits), s1 = (int)((long long)steps_all * (rank + 1) / splits);
    const int n = s1 - s0;
    const uint32_t idesc = umma_idesc_bf16(shape.cols);
    float* sums = reinterpret_cast<float*>(raw + (base - smem_u32(raw)));
    const int pitch = shape.cols + 4;
    int stage = 0, turn = 0;             // of the next step: its stage, and how often all stages have been used before
    int tiles_done = 0;
    unsigned copies = 0;                 // parities of `copied`, which gathered tiles alone use
    bool dead = false;                   // a wait gave up: the CTA goes on with the cluster, without its copies and products
    for (int ti = blockIdx.y; ti < n_tiles; ti += gridDim.y) {
        const BigTile tile = l.big[ti];
        if (tile.adapter < 0) continue;
        const bool gathered = tile.first < 0;
        bool bad = dead;
        if (dead) {
        } else if (warp == kBigWarps) {
            if (lane == 0) {
                for (int s = 0; s < n && !bad; ++s) {
                    if (turn > 0) bad = !mbar_wait_bounded(empty + 8 * stage, (turn - 1) & 1, p.wait, kErrProducerWait);
                    if (bad) break;
                    const uint32_t to = base + (uint32_t)stage * shape.stage, bar = full + 8 * stage;
                    mbar_arrive_expect_tx(bar, shape.stage - (gathered ? kBigTile * 128 : 0));
                    if (blockIdx.x + blockIdx.y + blockIdx.z > 0 || turn * stages + stage + 1 != p.withhold) {
                        if (!gathered) tma_load_2d(to, &map_x, bar, (s0 + s) * 64, tile.first, policy_evict_first());
                        tma_load_2d(to + kBigTile * 128, &map_a, bar, (s0 + s) * 64, tile.adapter * SR + j0, policy_evict_last());
                    }
                    if (++stage == stages) stage = 0, ++turn;
                }
            }
            __syncwarp();
        } else if (warp < kBigWarps && gathered) {
            // eight threads a row of 128 bytes, four rows a thread; a step's copies are given away when those of
            // kAhead steps more are on their way
            constexpr int kAhead = 3;
            const char* from[4];
            uint32_t at[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = (tid >> 3) + 32 * i;
                from[i] = row_ptr(p.x, token_of(l, tile, min(row, tile.count - 1))) + 16 * (tid & 7);
                at[i] = base + row * 128 + 16 * ((tid & 7) ^ (row & 7));
            }
            int given = stage;
            for (int s = 0; s < n + kAhead; ++s) {
                if (s < n) {
                    if (turn > 0) bad = !mbar_wait_bounded(empty + 8 * stage, (turn - 1) & 1, p.wait, kErrProducerWait);
                    if (__any_sync(~0u, bad)) break;
                    const int k = (s0 + s) * 64;
                    const bool in = k + 8 * (tid & 7) < K;
#pragma unroll
                    for (int i = 0; i < 4; ++i) copy16(at[i] + (uint32_t)stage * shape.stage, in ? from[i] + 2 * k : from[i], in);
                    if (++stage == stages) stage = 0, ++turn;
                }
                copy16_commit();
                if (s >= kAhead) {
                    copy16_wait<kAhead>();
                    fence_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(copied + 8 * given);
                    if (++given == stages) given = 0;
                }
            }
            copy16_wait<0>();
            bad = __any_sync(~0u, bad);
        } else if (warp < kBigWarps) {
            turn += (stage + n) / stages;
            stage = (stage + n) % stages;
        } else if (warp == kBigWarps + 1 && lane == 0) {
            for (int s = 0; s < n && !bad; ++s) {
                bad = !mbar_wait_bounded(full + 8 * stage, turn & 1, p.wait, kErrConsumerWait);
                if (gathered && !bad) {
                    bad = !mbar_wait_bounded(copied + 8 * stage, copies >> stage & 1, p.wait, kErrConsumerWait);
                    copies ^= 1u << stage;
                }
                if (bad) break;
                tc_fence_after_sync();
                const uint32_t at = base + (uint32_t)stage * shape.stage;
                const uint64_t xa = umma_desc_sw128(at), wa = umma_desc_sw128(at + kBigTile * 128);
#pragma unroll
                for (int k = 0; k < 4; ++k) umma_bf16(tmem, xa + 2 * k, wa + 2 * k, idesc, s > 0 || k > 0);
                umma_commit(empty + 8 * stage);
                if (++stage == stages) stage = 0, ++turn;
            }
            if (!bad) umma_commit(done);
        }
        // (one thread waits for the products; the others sleep at the barrier)
        if (warp == kBigWarps + 1 && lane == 0 && !bad) bad = !mbar_wait_bounded(done, tiles_done & 1, p.wait, kErrConsumerWait);
        ++tiles_done;
        tc_fence_before_sync();
        if (__syncthreads_or(bad)) {
            // Nothing more is copied or multiplied; what is on its way arrives before the CTA leaves.
            if (!dead && warp == kBigWarps && lane == 0)
                for (int i = 0; i < stages; ++i) mbar_wait_bounded(full + 8 * i, (turn - (i >= stage ? 1 : 0)) & 1, p.wait, kErrDrainWait);
            dead = true;
            __syncthreads();
        }
        tc_fence_after_sync();
        // a thread has a token's row; two warps share 32 tokens' columns
        const bool alone = splits == 1;
        float* out = p.low_big + j0;
        if (warp < kBigWarps) {
            const int row = 32 * (warp & 3) + lane;
            float* to = alone ? out + (size_t)token_of(l, tile, min(row, tile.count - 1)) * SR : sums + row * pitch;
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
        }
        tc_fence_before_sync();
        if (!alone) {
            cluster.sync();
            // this CTA's share of the tokens, four columns a thread, two of them at a time
            const int first = tile.count * rank / splits, quads = cols / 4;
            const int all = (tile.count * (rank + 1) / splits - first) * quads;
            for (int i0 = tid; i0 < all; i0 += 2 * kBigThreads) {
                float4 w[2][kMaxSplits];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int i = min(i0 + h * kBigThreads, all - 1), t = first + i / quads, j = i % quads * 4;
#pragma unroll
                    for (int q = 0; q < kMaxSplits; ++q)
                        if (q < splits) w[h][q] = *reinterpret_cast<const float4*>(cluster.map_shared_rank(sums, q) + t * pitch + j);
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int i = i0 + h * kBigThreads, t = first + i / quads, j = i % quads * 4;
                    float4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int q = 0; q < kMaxSplits; ++q) {
                        if (q >= splits) break;
                        v.x += w[h][q].x; v.y += w[h][q].y; v.z += w[h][q].z; v.w += w[h][q].w;
                    }
                    if (i < all) *reinterpret_cast<float4*>(out + (size_t)token_of(l, tile, t) * SR + j) = v;
                }
            }
            // The others have read this CTA's sums: its stages are free, for copies that another proxy writes than the
            // one that wrote and read the sums.
            fence_async_cluster();
            cluster.sync();
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
// the first products, which lie in tensor memory as bf16 operands (35 us at 4096 tokens, N 10240, rank 64; with
// them in shared memory, read again for every block, 38).  One thread has B's rows and base copied
// into a ring of stages and, from there again, the finished blocks to y; another one issues the products, two
// accumulators in turn; eight warps add base, half a row of 64 a thread.  All tiles' blocks are dealt to the
// CTAs in equal runs.  Tiles that whole copies do not fit (fewer than 128 tokens, or not in a row) are copied by the
// eight warps in pieces of 16 bytes, a warp its own rows, through the same stages (37 us for 4096 tokens in no
// order, N 8192; a thread straight from and to its own row, 59).  Rows that are not aligned, and a part's end inside
// a piece, go element by element.
// Stages: three (35 us as above; two 40, four 41).
constexpr int kUpBlock = 64, kUpCtas = 2, kUpStages = 3, kUpBigThreads = kUpThreads + 64;

// Shared memory, stages of: B (64 rows), y (and, of bf16, base before it), base of fp32 (and y_f32 after it) or
// y_f32.  Rows of 128 bytes, swizzled; B in pieces of 64 r, fp32 in halves of 32 columns.
struct UpSmem {
    int stage, wide_at, total;           // bytes of a stage; of it before the fp32 halves; of all
};
__host__ __device__ inline UpSmem up_smem(int rank, bool f32) {
    UpSmem s;
    s.wide_at = kUpBlock * 128 * ((rank + 63) / 64) + kBigTile * 128;
    s.stage = s.wide_at + (f32 ? 2 * kBigTile * 128 : 0);
    s.total = 1024 + kUpStages * s.stage + 256;      // (195 KB at most)
    return s;
}
// Tensor memory: two accumulators, then the parts, a row a lane, two r a column.
__host__ __device__ inline int up_tmem(int rank, int parts) {
    return 2 * kUpBlock + parts * ((rank + 15) / 16 * 8) <= 256 ? 256 : 512;     // (at most 128 + 3 x 64)
}

// Blocks of columns, each in one part.
__device__ __forceinline__ int part_blocks(const AdapterParams& p, int part) {
    return (p.part_end[part] - (part ? p.part_end[part - 1] : 0) + kUpBlock - 1) / kUpBlock;
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, uint32_t src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(m)), "r"(src), "r"(c0), "r"(c1) : "memory");
}

// 32 consecutive columns of this thread's row of tensor memory.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
                   "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}

// Four columns of this thread's row.
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};"
                 ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// D += A B^T of 128 x n over 16 k, A in tensor memory (eight columns), B in shared memory.
__device__ __forceinline__ void umma_bf16_from_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
                 ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

struct UpMaps {
    CUtensorMap b, base, y, y32;
};

// BASE 0: none, 1: bf16, 2: fp32; P: parts of a first product (3: there is an fp32 result)
template <int BASE, int P>
__global__ void __launch_bounds__(kUpBigThreads, kUpCtas) adapters_up_big_kernel(const __grid_constant__ UpMaps maps,
                                                                                  const __grid_constant__ AdapterParams p) {
    extern __shared__ __align__(16) unsigned char raw[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Lists l = lists_of(p.tiles, p.tokens);
    const int R = p.rank, N = p.N, pieces = (R + 63) / 64, S = kUpStages, part_columns = (R + 15) / 16 * 8;
    const UpSmem shape = up_smem(R, BASE == 2 || P == 3);
    const uint32_t ring = (smem_u32(raw) + 1023u) & ~1023u, bars = ring + S * shape.stage;
    // stages filled and finished, sums made (two accumulators) and read, the first products of a run in place
    const uint32_t full = bars, written = bars + 32, made = bars + 64, taken = bars + 80, ready = bars + 96, slot = bars + 104;
    const int y_at = kUpBlock * 128 * pieces;
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
    if (warp == 0) tmem_alloc(slot, up_tmem(R, P));
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(written + 8 * i, kUpWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(made + 8 * i, 1);
            mbar_init(taken + 8 * i, kUpWarps);
        }
        mbar_init(ready, kUpWarps);
        fence_mbarrier_init();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    // only now: a kernel after this one that allocates tensor memory before it waits must find this one's taken
    griddep_launch_dependents();
    uint32_t tmem;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(slot));
    const uint32_t parts_at = tmem + 2 * kUpBlock;
    const size_t step = (size_t)p.parts * R;
    // Blocks so far give a stage and its phase, products an accumulator and its, runs with products `ready`'s.
    int stage = 0, turn = 0;             // of the next block
    unsigned products = 0, runs_made = 0;
    bool bad = false;
    auto advance = [&]() {
        if (++stage == S) stage = 0, ++turn;
    };
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
        const int ad = tile.adapter, r = tile.rank, steps = (r + 15) / 16, used = (steps + 3) / 4;
        const bool put = ad >= 0 || !p.in_place, put32 = P == 3 && (ad >= 0 || !p.in_place32);
        if (!put && !put32) continue;
        auto whole = [&](int i) { return tile.count == kBigTile && tile.first >= 0 && p.wide && n0 + (i + 1) * kUpBlock <= n_end; };
        if (warp == kUpWarps) {          // copies
            if (lane == 0) {
                const int first = stage, first_turn = turn;
                auto load = [&](int i) {
                    const uint32_t to = ring + stage * shape.stage, bar = full + 8 * stage;
                    const int n = n0 + i * kUpBlock;
                    const bool with = BASE != 0 && whole(i);
                    mbar_arrive_expect_tx(bar, used * (kUpBlock * 128) + (with ? (BASE == 2 ? 2 : 1) * kBigTile * 128 : 0));
                    if (blockIdx.x == 0 && turn * S + stage + 1 == p.withhold) return advance();
                    for (int k = 0; k < used; ++k)
                        tma_load_2d(to + k * (kUpBlock * 128), &maps.b, bar, 64 * k, ad * N + n, policy_evict_last());
                    if (with) {
                        if (BASE == 2) {
                            tma_load_2d(to + shape.wide_at, &maps.base, bar, n, tile.first, policy_evict_first());
                            tma_load_2d(to + shape.wide_at + kBigTile * 128, &maps.base, bar, n + 32, tile.first, policy_evict_first());
                        } else {
                            tma_load_2d(to + y_at, &maps.base, bar, n, tile.first, policy_evict_first());
                        }
                    }
                    advance();
                };
                int loaded = 0;
                while (loaded < min(S, runs)) load(loaded++);
                int st = first, tn = first_turn;
                for (int i = 0; i < runs; ++i) {
                    bad = !mbar_wait_bounded(written + 8 * st, tn & 1, p.wait, kErrProducerWait);
                    if (bad) break;
                    if (whole(i)) {
                        const uint32_t from = ring + st * shape.stage;
                        const int n = n0 + i * kUpBlock;
                        if (put) tma_store_2d(&maps.y, from + y_at, n, tile.first);
                        if (put32) {
                            tma_store_2d(&maps.y32, from + shape.wide_at, n, tile.first);
                            tma_store_2d(&maps.y32, from + shape.wide_at + kBigTile * 128, n + 32, tile.first);
                        }
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                    if (loaded < runs) {
                        asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        load(loaded++);
                    }
                    if (++st == S) st = 0, ++tn;
                }
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                if (bad)                 // what is on its way arrives before the CTA leaves
                    for (int i = 0; i < min(S, loaded); ++i) {
                        if (--stage < 0) stage = S - 1, --turn;
                        mbar_wait_bounded(full + 8 * stage, turn & 1, p.wait, kErrDrainWait);
                    }
            }
            bad = __any_sync(~0u, bad);
            continue;
        }
        if (warp == kUpWarps + 1) {      // products
            if (r > 0) {
                const uint32_t idesc = umma_idesc_bf16(kUpBlock);
                const uint64_t ring_desc = umma_desc_sw128(ring);
                bad = !mbar_wait_bounded(ready, runs_made & 1, p.wait, kErrConsumerWait);
                ++runs_made;
                for (int i = 0; i < runs; ++i) {
                    const unsigned acc = products & 1, before = products >> 1;
                    if (!bad && before > 0) bad = !mbar_wait_bounded(taken + 8 * acc, (before - 1) & 1, p.wait, kErrConsumerWait);
                    if (!bad) bad = !mbar_wait_bounded(full + 8 * stage, turn & 1, p.wait, kErrConsumerWait);
                    if (__any_sync(~0u, bad)) break;
                    const uint32_t b_at = ring + stage * shape.stage;
                    if (r & 15) {        // what lies past the rank in the last 16 r, NaN perhaps, becomes zeros
#pragma unroll 1
                        for (int k = r >> 3; k < 2 * steps; ++k)
                            for (int row = lane; row < kUpBlock; row += 32) {
                                const uint32_t at16 = b_at + (k >> 3) * (kUpBlock * 128) + row * 128 + 16 * ((k & 7) ^ (row & 7));
                                const uint4 v = lds128(at16);
                                uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    w[j] &= (8 * k + 2 * j < r ? 0xffffu : 0u) | (8 * k + 2 * j + 1 < r ? 0xffff0000u : 0u);
                                sts128(at16, w[0], w[1], w[2], w[3]);
                            }
                        fence_async_smem();
                        __syncwarp();
                    }
                    tc_fence_after_sync();
                    if (lane == 0) {
                        const uint64_t bt = ring_desc + (uint64_t)(stage * shape.stage >> 4);
                        for (int k = 0; k < used; ++k)
#pragma unroll
                            for (int j = 0; j < P; ++j)
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    if (4 * k + q < steps)
                                        umma_bf16_from_tmem(tmem + acc * kUpBlock, parts_at + j * part_columns + 8 * (4 * k + q),
                                                            bt + (uint64_t)(k * (kUpBlock * 128 >> 4) + 2 * q), idesc, k + j + q > 0);
                        umma_commit(made + 8 * acc);
                    }
                    __syncwarp();
                    ++products;
                    advance();
                }
                bad = __any_sync(~0u, bad);
            } else {
                for (int i = 0; i < runs; ++i) advance();
            }
            continue;
        }
        // Eight warps: a thread has a token's row and 32 of a block's 64 columns.
        const float scale = scale_of(p, ad);
        const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;
        const bool mine = row < tile.count;
        const int t = token_of(l, tile, mine ? row : 0);
        if (r > 0) {
            // The run's first products, two threads a row, 8 r at a time each.  (All products of the run before are
            // done: this thread has waited for the last.)
            const float* low = p.low_big + (size_t)t * step + part * R;
            const uint32_t to = parts_at + ((uint32_t)(32 * quarter) << 16);
#pragma unroll 1
            for (int i0 = half; i0 < 2 * steps; i0 += 4) {
                float4 x[2][2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {            // (8 r from one below R on are within the row)
                    const int at = min(8 * (i0 + 2 * k), R - 8);
                    x[k][0] = ld_cg_f32x4(low + at);
                    x[k][1] = ld_cg_f32x4(low + at + 4);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = i0 + 2 * k;
                    if (i >= 2 * steps) break;
                    const float v[8] = {x[k][0].x, x[k][0].y, x[k][0].z, x[k][0].w, x[k][1].x, x[k][1].y, x[k][1].z, x[k][1].w};
                    uint32_t out[P][4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool in0 = mine && 8 * i + 2 * j < r, in1 = mine && 8 * i + 2 * j + 1 < r;
                        uint32_t s[P];
                        split(in0 ? v[2 * j] * scale : 0.f, in1 ? v[2 * j + 1] * scale : 0.f, s);
#pragma unroll
                        for (int n = 0; n < P; ++n) out[n][j] = s[n];
                    }
#pragma unroll
                    for (int j = 0; j < P; ++j) tmem_st4(to + j * part_columns + 4 * i, out[j]);
                }
            }
            tmem_wait_st();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(ready);
        }
        // Of tiles that are not copied, blocks of whole pieces of 16 bytes: a warp brings and takes its own 32 rows'
        // halves of the stage, whole rows by neighbouring lanes, base a block ahead.
        const bool listed = p.wide && (tile.first < 0 || tile.count < kBigTile);
        auto in_pieces = [&](int i) { return listed && (n0 + (i + 1) * kUpBlock <= n_end || n_end % 8 == 0); };
        // this lane's k-th piece: where in the stage, of which token, from which column on
        auto piece = [&](int i, int k, bool f32, int at, uint32_t& to, int& token, int& c) {
            const int r32 = k * (f32 ? 4 : 8) + (lane >> (f32 ? 3 : 2)), q = lane & (f32 ? 7 : 3), rw = 32 * quarter + r32;
            token = __shfl_sync(~0u, t, r32);
            c = n0 + i * kUpBlock + 32 * half + q * (f32 ? 4 : 8);
            const uint32_t base_at = ring + at * shape.stage;
            to = f32 ? base_at + shape.wide_at + half * (kBigTile * 128) + rw * 128 + 16 * (q ^ (rw & 7))
                     : base_at + y_at + rw * 128 + 16 * ((4 * half + q) ^ (rw & 7));
            return rw < tile.count && c < n_end;
        };
        auto fetch = [&](int i, int at) {
            if (BASE != 0 && in_pieces(i)) {
#pragma unroll
                for (int k = 0; k < (BASE == 2 ? 8 : 4); ++k) {
                    uint32_t to;
                    int token, c;
                    if (piece(i, k, BASE == 2, at, to, token, c))
                        copy16(to, row_ptr(p.base, token) + (size_t)c * (BASE == 2 ? 4 : 2), true);
                }
            }
            copy16_commit();
        };
        for (int i = 0; i < runs; ++i) {
            bad = !mbar_wait_bounded(full + 8 * stage, turn & 1, p.wait, kErrConsumerWait);
            if (listed && i == 0) fetch(0, stage);
            float d[32];
            if (r > 0) {
                const unsigned acc = products & 1;
                if (!bad) bad = !mbar_wait_bounded(made + 8 * acc, (products >> 1) & 1, p.wait, kErrConsumerWait);
                bad = __any_sync(~0u, bad);
                if (bad) break;
                ++products;
                tc_fence_after_sync();
                tmem_ld32(tmem + ((uint32_t)(32 * quarter) << 16) + acc * kUpBlock + 32 * half, d);
                tmem_wait_ld();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(taken + 8 * acc);
            } else {
                bad = __any_sync(~0u, bad);
                if (bad) break;
#pragma unroll
                for (int k = 0; k < 32; ++k) d[k] = 0.f;
            }
            float odd = 0.f;             // NaN if any sum is, or infinite
#pragma unroll
            for (int k = 0; k < 32; ++k) odd = fmaf(d[k], 0.f, odd);
            const int n = n0 + i * kUpBlock + 32 * half;
            if (odd != odd && mine) {
                const float* low = p.low_big + (size_t)t * step;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = d[8 * k + j];
                    plain_up<0>(p, low, scale, p.b + (size_t)max(ad, 0) * N * R, n + 8 * k, r, x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[8 * k + j] = x[j];
                }
            }
            if (!listed) {
            } else if (i + 1 < runs) {
                const int next = stage + 1 == S ? 0 : stage + 1;
                if (in_pieces(i + 1)) bad = !mbar_wait_bounded(full + 8 * next, (turn + (next == 0)) & 1, p.wait, kErrConsumerWait);
                bad = __any_sync(~0u, bad);
                if (bad) break;
                fetch(i + 1, next);
            } else {
                copy16_commit();
            }
            const bool pieces_here = in_pieces(i);
            if (pieces_here || whole(i)) {
                if (pieces_here) {
                    copy16_wait<1>();
                    __syncwarp();
                }
                const uint32_t to = ring + stage * shape.stage, y_row = to + y_at + row * 128, swap = row & 7;
                const uint32_t f_row = to + shape.wide_at + half * (kBigTile * 128) + row * 128;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t y16 = y_row + 16 * ((4 * half + k) ^ swap);
                    const uint32_t f0 = f_row + 16 * ((2 * k) ^ swap), f1 = f_row + 16 * ((2 * k + 1) ^ swap);
                    float* v = d + 8 * k;
                    if (BASE == 1) {
                        const uint4 x = lds128(y16);
                        float from[8];
                        bf16x2_to_f32(x.x, from[0], from[1]);
                        bf16x2_to_f32(x.y, from[2], from[3]);
                        bf16x2_to_f32(x.z, from[4], from[5]);
                        bf16x2_to_f32(x.w, from[6], from[7]);
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += from[j];
                    } else if (BASE == 2) {
                        const uint4 x = lds128(f0), y = lds128(f1);
                        const uint32_t q[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] += __uint_as_float(q[j]);
                    }
                    sts128(y16, f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7]));
                    if (P == 3) {
                        sts128(f0, __float_as_int(v[0]), __float_as_int(v[1]), __float_as_int(v[2]), __float_as_int(v[3]));
                        sts128(f1, __float_as_int(v[4]), __float_as_int(v[5]), __float_as_int(v[6]), __float_as_int(v[7]));
                    }
                }
                if (pieces_here) {
                    __syncwarp();
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t from;
                        int token, c;
                        if (piece(i, k, false, stage, from, token, c) && put)
                            *reinterpret_cast<uint4*>(row_ptr(p.y, token) + (size_t)c * 2) = lds128(from);
                    }
                    if (P == 3) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            uint32_t from;
                            int token, c;
                            if (piece(i, k, true, stage, from, token, c) && put32)
                                *reinterpret_cast<uint4*>(row_ptr(p.y32, token) + (size_t)c * 4) = lds128(from);
                        }
                    }
                }
                fence_async_smem();
            } else if (mine) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = n + 8 * k;
                    if (c >= n_end) continue;
                    const bool wide = p.wide && c + 8 <= n_end;
                    float v[8], from[8] = {};
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = d[8 * k + j];
                    if (BASE != 0) load_cols(row_ptr(p.base, t), BASE == 2, c, n_end, wide, from);
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] += from[j];
                    if (put) put_cols(row_ptr(p.y, t), false, c, n_end, wide, v);
                    if (put32) put_cols(row_ptr(p.y32, t), true, c, n_end, wide, v);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(written + 8 * stage);
            advance();
        }
    }
    if (warp == kUpWarps && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    copy16_wait<0>();
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 0) tmem_dealloc(tmem, up_tmem(R, P));
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
    return tokens > kFewTokens ? up256(16 + (size_t)max_big(tokens) * sizeof(BigTile) + (2 * (size_t)tokens + 1) * 4 +
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
    if ((long long)a->num * a->N > 0x7fffff00LL)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "num=%d adapters of N=%d rows exceed 2^31 - 256", a->num, a->N);
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

template <int Q>
static cudaError_t launch_up(const AdapterParams& p, dim3 grid, dim3 block, size_t smem, cudaStream_t stream) {
    const int base = !p.base.ptr ? 0 : p.base.f32 ? 2 : 1;
    if (p.y32.ptr)
        return base == 0   ? launch_dependent(adapters_up_kernel<0, 3, Q>, grid, block, smem, stream, p)
               : base == 1 ? launch_dependent(adapters_up_kernel<1, 3, Q>, grid, block, smem, stream, p)
                           : launch_dependent(adapters_up_kernel<2, 3, Q>, grid, block, smem, stream, p);
    return base == 0   ? launch_dependent(adapters_up_kernel<0, 2, Q>, grid, block, smem, stream, p)
           : base == 1 ? launch_dependent(adapters_up_kernel<1, 2, Q>, grid, block, smem, stream, p)
                       : launch_dependent(adapters_up_kernel<2, 2, Q>, grid, block, smem, stream, p);
}

static cudaError_t launch_small(const AdapterParams& p, long long tiles, int sm_count, cudaStream_t stream, bool up) {
    const size_t smem = p.tokens <= kFewTokens ? sizeof(FewTiles) : 0;
    if (up) {
        const long long ctas = (tiles * ((p.N + kUpUnit - 1) / kUpUnit) + kUpWarps - 1) / kUpWarps, most = 2LL * sm_count;
        const dim3 grid((unsigned)(ctas < most ? ctas : most)), block(kUpThreads);
        return p.rank <= 32 ? launch_up<1>(p, grid, block, smem, stream) : launch_up<2>(p, grid, block, smem, stream);
    }
    // CTAs that share K, by the pieces of work that there can be (of one part, so that sums do not depend on how many
    // parts there are): eight while all of them find places, two to an SM in whole clusters (128 SMs of which do),
    // then as few as fill the GPU (8192 -> 8192, 64 adapters; of 4, 2 and 1 CTAs, 80 pieces: 19.2, 19.8, 23 us; 158: 30, 28, 30;
    // 256: 36, 34, 32; 632: 107, 83, 78).
    const long long any = p.tokens / kTile + p.num + 1, groups = (p.rank + 15) / 16;
    const long long pieces = (p.tokens < any ? p.tokens : any) * groups, items = tiles * p.parts * groups;
    const int size = pieces <= 32 ? kLowCluster : pieces <= 100 ? 4 : pieces <= 200 ? 2 : 1;
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

// A tensor map of rows: boxes of 128 bytes of columns and `high` rows, 128-byte swizzled.
static dl_status rows_map(CUtensorMap& map, const void* data, bool f32, long long rows, long long columns, long long stride, int high) {
    EncodeTiled encode;
    const dl_status s = host_encode(encode);
    if (s != DL_OK) return s;
    const cuuint64_t dims[2] = {(cuuint64_t)columns, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)stride};
    const cuuint32_t box[2] = {f32 ? 32u : 64u, (cuuint32_t)high}, ones[2] = {1, 1};
    const CUresult r = encode(&map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                              const_cast<void*>(data), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? DL_OK : host_fail(DL_ERR_CUDA, "a tensor map of %lld rows: CUresult %d", rows, (int)r);
}

struct BigMaps {
    CUtensorMap x, a;
    UpMaps up;
};
static dl_status big_maps(const AdapterParams& p, BigMaps& m) {
    const int SR = p.parts * p.rank;
    dl_status s = rows_map(m.x, p.x.ptr, false, p.tokens, p.K, p.x.stride, kBigTile);
    if (s == DL_OK) s = rows_map(m.a, p.a, false, (long long)p.num * SR, p.K, 2LL * p.K, big_smem(SR).cols);
    if (s == DL_OK) s = rows_map(m.up.b, p.b, false, (long long)p.num * p.N, p.rank, 2LL * p.rank, kUpBlock);
    m.up.base = m.up.y = m.up.y32 = m.up.b;
    if (!p.wide) return s;               // (no copies then)
    if (s == DL_OK && p.base.ptr) s = rows_map(m.up.base, p.base.ptr, p.base.f32, p.tokens, p.N, p.base.stride, kBigTile);
    if (s == DL_OK) s = rows_map(m.up.y, p.y.ptr, false, p.tokens, p.N, p.y.stride, kBigTile);
    if (s == DL_OK && p.y32.ptr) s = rows_map(m.up.y32, p.y32.ptr, true, p.tokens, p.N, p.y32.stride, kBigTile);
    return s;
}

static cudaError_t launch_low_big(const AdapterParams& p, const BigMaps& m, long long tiles, int sm_count, cudaStream_t stream) {
    const int columns = p.parts * p.rank, groups = (columns + kBigCols - 1) / kBigCols, splits = big_splits(p.tokens, p.K);
    const long long most = 4LL * sm_count / (splits * groups) + 1;
    const size_t smem = big_smem(columns).total;
    const cudaError_t e = raise_smem<adapters_low_big_kernel>(1024 + kBigStages + 256);
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
    return cudaLaunchKernelEx(&cfg, adapters_low_big_kernel, m.x, m.a, p);
}

template <int BASE, int P>
static cudaError_t launch_up_big(AdapterParams& p, const BigMaps& m, int sm_count, cudaStream_t stream) {
    constexpr bool f32 = BASE == 2 || P == 3;
    // two CTAs to an SM where their stages and their 256 of tensor memory's 512 columns fit twice
    constexpr int kSm = 227 * 1024;
    const int smem = up_smem(p.rank, f32).total;
    const int ctas = up_tmem(p.rank, P) == 256 && 2 * (smem + 1024) <= kSm ? kUpCtas : 1;
    const cudaError_t e = raise_smem<adapters_up_big_kernel<BASE, P>>(up_smem(kBigRank, f32).total);
    if (e != cudaSuccess) return e;
    return launch_dependent(adapters_up_big_kernel<BASE, P>, dim3(ctas * sm_count), dim3(kUpBigThreads), smem, stream, m.up, p);
}

template <int P>
static cudaError_t launch_up_big_base(AdapterParams& p, const BigMaps& m, int sm_count, cudaStream_t stream) {
    if (!p.base.ptr) return launch_up_big<0, P>(p, m, sm_count, stream);
    return p.base.f32 ? launch_up_big<2, P>(p, m, sm_count, stream) : launch_up_big<1, P>(p, m, sm_count, stream);
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
    p.big_from = p.list_from = 0x7fffffff;
    if (p.rank <= kBigRank) {
        p.big_from = kBigFrom;
        const long long need = kListWork / ((long long)tokens * p.rank) + 1;
        p.list_from = need > kListFrom ? (int)need : kListFrom;
    }
    p.index = index;
    p.tokens = tokens;
    p.in_place = same_rows(p.y, p.base);
    p.in_place32 = p.y32.ptr && same_rows(p.y32, p.base);
    p.wide = true;
    for (const Rows* r : {&p.base, &p.y, &p.y32})
        if (r->ptr) p.wide = p.wide && rows_aligned16(*r, tokens);
    const long long small = tokens <= kFewTokens ? tokens : max_small(tokens, p.num);
    if (tokens > 0x7fff0000 || small * ((N + 15) / 16) > 0x7fff0000LL || small * p.parts * ((p.rank + 15) / 16) > 0x7fff0000LL)
        return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "tokens=%d with N=%d exceed one launch", tokens, N);
    HostDevice dev;
    if ((s = host_device(dev)) != DL_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.wait = WaitCtl{dev.err_word, dev.wait_limit_ns};
    p.withhold = dev.withhold_stage;
    cudaError_t e;
    if (tokens <= kFewTokens) {
        if ((e = launch_small(p, small, dev.sm_count, st, false)) == cudaSuccess)
            e = launch_small(p, small, dev.sm_count, st, true);
    } else {
        // Each list's kernels find how much there is on the device.  Both first products may run at the
        // same time, then both second ones.
        const long long big = max_big(tokens);
        BigMaps maps;
        if (p.rank <= kBigRank && (s = big_maps(p, maps)) != DL_OK) return s;
        const size_t counters = ((size_t)p.num + 1 + (tokens <= kStartsHere ? tokens + 1 : 0)) * 4;
        if ((e = raise_smem<sort_tokens_kernel>((kMaxAdapters + 1 + kStartsHere + 1) * 4)) == cudaSuccess)
            e = launch_dependent(sort_tokens_kernel, dim3(1), dim3(1024), counters, st, p);
        if (e == cudaSuccess) e = launch_small(p, small, dev.sm_count, st, false);
        if (e == cudaSuccess && p.rank <= kBigRank) e = launch_low_big(p, maps, big, dev.sm_count, st);
        if (e == cudaSuccess) e = launch_small(p, small, dev.sm_count, st, true);
        if (e == cudaSuccess && p.rank <= kBigRank)
            e = p.y32.ptr ? launch_up_big_base<3>(p, maps, dev.sm_count, st) : launch_up_big_base<2>(p, maps, dev.sm_count, st);
    }
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "linear_adapters launch: %s", cudaGetErrorString(e));
    return host_ok();
}
