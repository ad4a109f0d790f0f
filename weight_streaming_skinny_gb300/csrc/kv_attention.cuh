// Attention over the paged 8-bit cache on the 5th-generation tensor cores.
//
// The mathematics.  For one key/value head and the rows r (a new token and one
// of the query heads that share the key/value head), over the cached tokens j:
//     t_jr = c * ks_j * (q_r . k_j) + log2 vs_j ,   c = scale * log2 e,
//     P_jr = 2^(t_jr + n_r) ,   o_r = sum_j P_jr v_j / sum_j (P_jr / vs_j),
// k_j, v_j the stored codes and ks_j, vs_j the scales of their blocks.  Folding
// vs_j into the exponent makes P_jr the token's true weight on its codes, so n_r
// (kept so that the largest P_jr of the row lies near the top of the e4m3
// range) bounds what is multiplied, and costs nothing per element.
//
// Both products run as tcgen05.mma kind::f8f6f4 on the codes exactly as they
// lie in the cache; nothing converts keys or values:
//     S^T [128 tokens x rows] = K [128 x D] . Q^T       (tokens on TMEM lanes)
//     O^T [D x rows]         += V^T [D x 128] . P^T
// The 16-bit side is split into two e4m3 parts, x = hi + lo: a bf16 query has
// 8 significant bits and a part has 4, so hi + lo is exact down to 2^-17 of
// the row's largest element (each row is scaled to the top of the range).
// P = hi + lo / 16 with the parts in separate accumulator columns: relative
// error at most 2^-8 (rms 4e-4, a quarter of a bf16 rounding's) down to 2^-14
// of the row's largest, 2^-22 of it absolute below.  Scores, maxima,
// exponentials, sums and accumulators are fp32.
//
// A CTA runs a contiguous range of 128-token tiles of the whole call (sequence,
// row tile, head, tile), the same number for every CTA to within one: the work
// of a long sequence spreads over the chip, and many short ones pack.  A
// sequence that ends up on several CTAs leaves partial sums in the workspace,
// joined in a fixed order by attention_combine_kernel.
#pragma once

#include "kv_cache.cuh"

namespace dl {

constexpr int kTile = 128;              // tokens of a tile

struct AttnParams {
    const uint16_t* q;
    uint16_t* out;
    float* lse;
    const float *k_scale, *v_scale;
    long long q_stride, scale_page_stride, scale_head_stride;
    int num_pages, kv_heads, q_heads, group;
    int page_size, page_shift, block_shift;
    int tile_tokens, row_tiles;         // new tokens of a row tile, row tiles of max_q
    float scale_log2;                   // scale * log2(e)
    Sequences s;
    float* partial;                     // [grid][2][RP][D] then [grid][2][RP][2]
    struct AttnSplit* split;            // [grid]
    unsigned* err_word;
    unsigned long long wait_limit_ns;
};

// A split item, at the index of the CTA that begins it (n = 0: none).
struct AttnSplit {
    int n;                              // CTAs that share it, consecutive
    int slot0;                          // which of the first CTA's two slots it uses
    int row0, rows, head;               // first token row, rows, key/value head
};

// One row tile of a sequence.
struct AttnEntry {
    int b, row0, tokens;                // its first token row and its new tokens
    int seen0;                          // cached tokens its first token sees (< 1: it has no place)
    int seen_first, seen_last;          // the same not below 0, and its last token's
    int tiles;                          // at least 1 where tokens > 0 (rows that see nothing get zeros)
};

__device__ __forceinline__ AttnEntry attn_entry(const AttnParams& p, int e) {
    AttnEntry r;
    r.b = p.row_tiles == 1 ? e : e / p.row_tiles;
    const int i0 = p.row_tiles == 1 ? 0 : (e - r.b * p.row_tiles) * p.tile_tokens;
    const SequenceView v = sequence_view(p.s, r.b, p.page_size);
    r.row0 = v.row0 + i0;
    r.tokens = max(min(p.tile_tokens, v.n_work - i0), 0);
    r.seen0 = v.len - v.n + i0 + 1;
    r.seen_first = max(r.seen0, 0);
    r.seen_last = max(r.seen0 + r.tokens - 1, 0);
    r.tiles = r.tokens > 0 ? max((r.seen_last + kTile - 1) / kTile, 1) : 0;
    return r;
}

// The tiles [begin(c), begin(c + 1)) of CTA c, and the CTA of a tile.
__device__ __forceinline__ long long attn_begin(long long total, int grid, int c) {
    return total * c / grid;
}
__device__ __forceinline__ int attn_cta_of(long long total, int grid, long long tile) {
    return (int)(((tile + 1) * grid - 1) / total);
}

// RP rows in NWG softmax warpgroups of RW = RP / NWG.
template <int D_, int RP_>
struct AttnShape {
    static constexpr int D = D_, RP = RP_;
    static constexpr int NWG = RP > 48 ? 2 : 1;
    static constexpr int RW = RP / NWG;
    static constexpr bool kConcat = RP == 8;            // S columns: hi parts, then lo parts
    static constexpr int kScoreCols = kConcat ? 16 : RP;
    static constexpr int kOutCol = 2 * kScoreCols;
    static constexpr int kCols = kOutCol + 2 * RP;
    static constexpr int kTmem = kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static constexpr int kCtas = RP > 48 ? 1 : 2;       // resident CTAs per SM
    static constexpr int kThreads = NWG * 128 + 64;
    static constexpr int kTileBytes = kTile * D;        // of K, and of V
    static constexpr int kQBytes = 2 * RP * D;
    static constexpr int kPBytes = 2 * RP * kTile;      // one buffer
    static constexpr int kMisc = 1024 + RP * 12 + NWG * 4 * RW * 4 + D * 4 + 256;
    static constexpr int kBudget = (kCtas == 1 ? 227 : 113) * 1024;
    static constexpr int kMost = (kBudget - 1024 - kQBytes - 2 * kPBytes - kMisc) / (2 * kTileBytes);
    static constexpr int kStages = kMost > 6 ? 6 : kMost;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * 2 * kTileBytes + kQBytes + 2 * kPBytes + kMisc;
    static_assert(kStages >= 2, "two tiles in flight");
};

// ---------------------------------------------------------------- device helpers

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1,
                                            int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// Matrix descriptor: start address, leading and stride byte offsets, layout
// (0: no swizzle, 2: 128-byte, 4: 64-byte swizzle), descriptor version 1.
__device__ __forceinline__ uint64_t umma_desc(uint32_t saddr, uint32_t lead, uint32_t stride, uint32_t layout) {
    return (uint64_t)((saddr >> 4) & 0x3fffu) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(stride >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)layout << 61;
}

// Instruction descriptor of kind::f8f6f4, e4m3 x e4m3 -> fp32, M x N; mn = 1:
// both operands have their M / N dimension contiguous in memory.
__host__ __device__ constexpr uint32_t umma_idesc(int m, int n, int mn) {
    return (1u << 4) | (mn ? 3u << 15 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, float* v) {
    uint32_t r[16];
    if constexpr (N == 16) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                     "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                       "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                     : "r"(taddr));
    } else {
        static_assert(N == 8, "8 or 16 columns");
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"r"(taddr), "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])),
                   "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])),
                   "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void fence_proxy_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void group_sync(int id, int threads) {
    asm volatile("barrier.sync.aligned %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Whether `v` holds for any thread of the barrier's.
__device__ __forceinline__ bool group_any(int id, int threads, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %3, 0;\n\t"
        "barrier.red.aligned.or.pred b, %1, %2, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
        : "=r"(r) : "r"(id), "r"(threads), "r"((uint32_t)v) : "memory");
    return r != 0;
}

__device__ __forceinline__ float warp_max_f32(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float log2_fast(float x) {
    float r;
    asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two probabilities -> their e4m3 parts: hi, and the remainder times 16 (low
// half: a).  The fp16 step in between rounds to 2^-11, far below the parts.
__device__ __forceinline__ void split_e4m3(float a, float b, uint32_t& hi, uint32_t& lo) {
    constexpr uint32_t kSixteen = 0x4C004C00u;          // f16x2
    asm("{\n\t"
        ".reg .b16 h, l;\n\t"
        ".reg .b32 x, y, z;\n\t"
        "cvt.rn.f16x2.f32 x, %3, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 h, x;\n\t"
        "cvt.rn.f16x2.e4m3x2 y, h;\n\t"
        "sub.rn.f16x2 z, x, y;\n\t"
        "mul.rn.f16x2 z, z, %4;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 l, z;\n\t"
        "cvt.u32.u16 %0, h;\n\t"
        "cvt.u32.u16 %1, l;\n\t"
        "}"
        : "=r"(hi), "=r"(lo) : "f"(a), "f"(b), "r"(kSixteen));
}

// Sums of v[0..N) over a warp's lanes by halving: afterwards v[0] is the sum
// of value lane_value<N>(lane).
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N], int lane) {
    int off = 16;
#pragma unroll
    for (int n = N; n > 1; n >>= 1, off >>= 1) {
        const bool up = lane & off;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = up ? v[i + n / 2] : v[i], send = up ? v[i] : v[i + n / 2];
            v[i] = keep + __shfl_xor_sync(~0u, send, off);
        }
    }
    for (; off; off >>= 1) v[0] += __shfl_xor_sync(~0u, v[0], off);
}
template <int N>
__device__ __forceinline__ int lane_value(int lane) {
    return lane / (32 / N);
}

// Waits of one CTA: bounded, and short once any of them has given up.
struct CtaWait {
    WaitCtl ctl;
    volatile int* stop;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, unsigned bit) const {
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        const unsigned long long t0 = globaltimer_ns();
#pragma unroll 1
        while (true) {
            if (mbar_try_wait(bar, parity)) return true;
            if (*stop) return false;
            if (globaltimer_ns() - t0 > ctl.limit_ns) {
                atomicOr(ctl.word, bit);
                *stop = 1;
                return false;
            }
        }
    }
};

// The segments of one CTA: the runs of its tiles that belong to one item
// (entry, head).
struct AttnWalk {
    long long at, end, item_begin;      // tiles of the call
    int e, head, tile0, tile1;
    AttnEntry entry;
    __device__ __forceinline__ void item() {
        const long long left = end - at;
        tile1 = left < entry.tiles - tile0 ? tile0 + (int)left : entry.tiles;
        item_begin = at - tile0;
    }
    // `within`: tiles of entry e before `at`
    __device__ __forceinline__ void start(const AttnParams& p, long long at_, long long end_, int e_, long long within) {
        at = at_;
        end = end_;
        e = e_;
        entry = attn_entry(p, e);
        head = (int)(within / entry.tiles);
        tile0 = (int)(within - (long long)head * entry.tiles);
        item();
    }
    __device__ __forceinline__ bool next(const AttnParams& p) {
        at += tile1 - tile0;
        if (at >= end) return false;
        tile0 = 0;
        if (++head == p.kv_heads) {
            head = 0;
            do entry = attn_entry(p, ++e);
            while (entry.tiles == 0);
        }
        item();
        return true;
    }
    __device__ __forceinline__ bool whole() const { return tile0 == 0 && tile1 == entry.tiles; }
};

// ---------------------------------------------------------------- the kernel

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas)
attention_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const __grid_constant__ AttnParams p) {
    constexpr int D = C::D, RP = C::RP, RW = C::RW, NWG = C::NWG, ST = C::kStages;
    constexpr int kProducer = NWG * 4, kMma = NWG * 4 + 1;
    // one accumulator lane per dim: M = 64 leaves 16 rows in each warp's lanes
    constexpr int kDimLanes = D / 4;
    constexpr uint32_t kSwizzle = D == 128 ? 2 : 4;
    // largest exponent of a probability (log2 448 = 8.807), and the one a new maximum gets
    constexpr float kTop = 8.8f, kTarget = 7.5f, kUnset = 1e30f;
    constexpr float kTinyScale = 8.67361737988403547e-19f;       // 2^-60

    extern __shared__ unsigned char smem_raw[];
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    unsigned char* sp = base;                                     // [2 buffers][2 RP / 16][128 tokens][16]
    unsigned char* sq = sp + 2 * C::kPBytes;                      // [2 parts][RP][D]
    unsigned char* tiles = sq + C::kQBytes;                       // [ST][K, V]
    unsigned char* misc = tiles + ST * 2 * C::kTileBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(misc);
    uint64_t *full = bars, *empty = bars + ST, *s_full = empty + ST, *p_full = s_full + 2, *pv_done = p_full + 2,
             *q_full = pv_done + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 1);
    int* s_stop = reinterpret_cast<int*>(tmem_slot + 1);
    long long* s_walk = reinterpret_cast<long long*>(misc + 512);     // total, begin, end, entry, within
    float* s_qs = reinterpret_cast<float*>(misc + 1024);              // [RP] a row's query scale
    float* s_n = s_qs + RP;                                           // [RP] n_r
    int* s_lim = reinterpret_cast<int*>(s_n + RP);                    // [RP] cached tokens a row sees
    float* s_red = reinterpret_cast<float*>(s_lim + RP);              // [NWG][4][RW]
    int* s_nan = reinterpret_cast<int*>(s_red + NWG * 4 * RW);        // [D] first NaN among the new tokens' values

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const CtaWait wait{{p.err_word, p.wait_limit_ns}, s_stop};

    if (warp == kMma) {
        if (lane == 0) {
            for (int i = 0; i < ST; ++i) {
                mbar_init(smem_u32(full + i), 1);
                mbar_init(smem_u32(empty + i), 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_u32(s_full + i), 1);
                mbar_init(smem_u32(p_full + i), NWG * 4);
                mbar_init(smem_u32(pv_done + i), 1);
            }
            mbar_init(smem_u32(q_full), NWG * 4);
            *s_stop = 0;
            fence_mbarrier_init();
        }
        __syncwarp();
        tmem_alloc(smem_u32(tmem_slot), C::kTmem);
    }
    if (warp == kProducer && lane == 0) {
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
    }
    griddep_wait();
    griddep_launch_dependents();
    if (warp == 0) {
        // the CTA's tiles, and the entry in which they begin
        const int entries = p.s.batch * p.row_tiles;
        long long total = 0;
        for (int e = lane; e < entries; e += 32) total += attn_entry(p, e).tiles;
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
        total *= p.kv_heads;
        const int grid = total < gridDim.x ? (int)total : (int)gridDim.x;
        long long begin = 0, end = 0, within = 0;
        int found = -1;
        if ((int)blockIdx.x < grid) {
            begin = attn_begin(total, grid, blockIdx.x);
            end = attn_begin(total, grid, blockIdx.x + 1);
            long long run = 0;
            for (int e0 = 0; e0 < entries && found < 0; e0 += 32) {
                const long long mine = e0 + lane < entries ? (long long)attn_entry(p, e0 + lane).tiles * p.kv_heads : 0;
                long long inc = mine;
                for (int o = 1; o < 32; o <<= 1) {
                    const long long y = __shfl_up_sync(~0u, inc, o);
                    if (lane >= o) inc += y;
                }
                const unsigned hit = __ballot_sync(~0u, run + inc > begin);
                if (hit) {
                    const int src = __ffs(hit) - 1;
                    found = e0 + src;
                    within = begin - run - __shfl_sync(~0u, inc - mine, src);
                }
                run += __shfl_sync(~0u, inc, 31);
            }
        }
        if (lane == 0) {
            s_walk[0] = total;
            s_walk[1] = begin;
            s_walk[2] = found < 0 ? begin : end;
            s_walk[3] = found;
            s_walk[4] = within;
            p.split[blockIdx.x].n = 0;
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const long long total = s_walk[0];
    const bool work = s_walk[2] > s_walk[1];
    AttnWalk w;
    if (work) w.start(p, s_walk[1], s_walk[2], (int)s_walk[3], s_walk[4]);

    if (work && warp == kProducer) {
        // ------------------------------------------------ loads: a page's rows each lane
        const int box = min(p.page_size, kTile), per = kTile / box;
        int it = 0;
        bool ok = true;
        do {
            const int* table = p.s.block_table + (size_t)w.entry.b * p.s.table_cols;
            const int sub = lane & 15;
            auto page_of = [&](int tile) {
                const int j = tile * kTile + sub * box;
                int pg = -1;
                if (sub < per && j < w.entry.seen_last) pg = table[j >> p.page_shift];
                return (unsigned)pg < (unsigned)p.num_pages ? pg : -1;
            };
            int page = page_of(w.tile0);
            for (int tile = w.tile0; tile < w.tile1 && ok; ++tile, ++it) {
                const int next = tile + 1 < w.tile1 ? page_of(tile + 1) : -1;
                const int s = it % ST;
                if (it >= ST) ok = __all_sync(~0u, wait(smem_u32(empty + s), ((it / ST) - 1) & 1, kErrProducerWait));
                if (!ok) break;
                const int copies = __popc(__ballot_sync(~0u, page >= 0));
                const uint32_t bar = smem_u32(full + s);
                if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(copies * box * D));
                __syncwarp();
                if (page >= 0) {
                    const uint32_t dst = smem_u32(tiles + (size_t)s * 2 * C::kTileBytes + (lane >= 16 ? C::kTileBytes : 0) + sub * box * D);
                    tma_load_4d(dst, lane >= 16 ? &tv : &tk, bar, 0, (tile * kTile + sub * box) & (p.page_size - 1),
                                w.head, page);
                }
                page = next;
            }
        } while (ok && w.next(p));
        // after a wait that gave up: no copy of this CTA may still be in flight when it leaves
        if (!ok)
            for (int i = max(it - ST, 0); i < it; ++i)
                mbar_wait_bounded(smem_u32(full + i % ST), (i / ST) & 1, wait.ctl, kErrDrainWait);
    } else if (work && warp == kMma) {
        // ------------------------------------------------ products, issued by one lane
        if (lane == 0) {
            constexpr uint32_t kScoreIdesc = umma_idesc(128, C::kScoreCols, 0);
            constexpr uint32_t kOutIdesc = umma_idesc(D, 2 * RP, 1);
            const uint32_t q0 = smem_u32(sq), p0 = smem_u32(sp);
            int it = 0, seg = 0;
            bool ok = true;
            auto scores = [&](int i) {
                if (!wait(smem_u32(full + i % ST), (i / ST) & 1, kErrConsumerWait)) return false;
                tc_fence_after_sync();
                const uint32_t k0 = smem_u32(tiles + (size_t)(i % ST) * 2 * C::kTileBytes);
                const uint32_t d = tmem + (i & 1) * C::kScoreCols;
#pragma unroll
                for (int part = 0; part < (C::kConcat ? 1 : 2); ++part)
#pragma unroll
                    for (int k = 0; k < D / 32; ++k)
                        umma_e4m3(d, umma_desc(k0 + 32 * k, 16, 8 * D, kSwizzle),
                                  umma_desc(q0 + part * RP * D + 32 * k, 16, 8 * D, kSwizzle), kScoreIdesc,
                                  part > 0 || k > 0);
                umma_commit(smem_u32(s_full + (i & 1)));
                return true;
            };
            do {
                ok = wait(smem_u32(q_full), seg & 1, kErrConsumerWait) && scores(it);
                for (int tile = w.tile0; tile < w.tile1 && ok; ++tile, ++it) {
                    if (tile + 1 < w.tile1 && !(ok = scores(it + 1))) break;
                    if (!(ok = wait(smem_u32(p_full + (it & 1)), (it >> 1) & 1, kErrConsumerWait))) break;
                    tc_fence_after_sync();
                    const uint32_t v0 = smem_u32(tiles + (size_t)(it % ST) * 2 * C::kTileBytes + C::kTileBytes);
#pragma unroll
                    for (int k = 0; k < kTile / 32; ++k)
                        umma_e4m3(tmem + C::kOutCol, umma_desc(v0 + k * 32 * D, 16, 8 * D, kSwizzle),
                                  umma_desc(p0 + (it & 1) * C::kPBytes + k * 32 * 16, 128, kTile * 16, 0), kOutIdesc,
                                  tile > w.tile0 || k > 0);
                    umma_commit(smem_u32(empty + it % ST));
                    umma_commit(smem_u32(pv_done + (it & 1)));
                }
                ++seg;
            } while (ok && w.next(p));
        }
        __syncwarp();
    } else if (work && warp < kProducer) {
        // ------------------------------------------------ softmax: a token each thread
        // (a wait that gives up is not left by: the others of the group are at its barriers)
        const int wg = warp >> 2, wq = warp & 3, tl = tid & 127, bar_id = 1 + wg;
        const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
        const int r0 = wg * RW;
        float* red = s_red + wg * 4 * RW;
        int it = 0;
        int slot = 0;
        do {
            const AttnEntry& en = w.entry;
            const int rows = en.tokens * p.group;
            // scales: the page of a tile's token two tiles ahead, its scales one tile ahead
            const int* table = p.s.block_table + (size_t)en.b * p.s.table_cols;
            auto page_at = [&](int tile) {
                const int j = tile * kTile + tl;
                int pg = -1;
                if (tile < w.tile1 && j < en.seen_last) pg = table[j >> p.page_shift];
                return (unsigned)pg < (unsigned)p.num_pages ? pg : -1;
            };
            auto load_scales = [&](int tile, int pg, float& a, float& b) {
                a = 0.f;
                b = 1.f;
                if (pg >= 0) {
                    const long long o = pg * p.scale_page_stride + w.head * p.scale_head_stride +
                                        (((tile * kTile + tl) & (p.page_size - 1)) >> p.block_shift);
                    a = p.k_scale[o];
                    b = p.v_scale[o];
                }
            };
            int pg0 = page_at(w.tile0), pg1 = page_at(w.tile0 + 1);

            // the row tile's queries as two e4m3 parts, each row scaled to the top of the range
            group_sync(bar_id, 128);
            constexpr int TPR = D / 16;             // threads of a row, 16 elements each
            for (int r = tl / TPR; r < RW; r += 128 / TPR) {
                const int c = tl % TPR, row = r0 + r;
                const int i = row / p.group, g = row - i * p.group;
                uint32_t x[8] = {};
                if (row < rows) {
                    const uint16_t* src = p.q + (size_t)(en.row0 + i) * p.q_stride + (size_t)(w.head * p.group + g) * D + 16 * c;
                    const uint4 a = ldg128(src), b = ldg128(src + 8);
                    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
                    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
                }
                uint32_t top = 0;                   // largest magnitude: bf16 bits order as integers
#pragma unroll
                for (int k = 0; k < 8; ++k) top = max(top, max(x[k] & 0x7fffu, (x[k] >> 16) & 0x7fffu));
#pragma unroll
                for (int o = TPR / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(~0u, top, o));
                // 2^e <= largest < 2^(e+1) becomes [128, 256); a row with an infinity or a NaN answers NaN
                const int e = max((int)(top >> 7), 1) - 127;
                const bool odd = (top >> 7) == 255;
                const float up1 = __uint_as_float((uint32_t)(127 + (7 - e) / 2) << 23);      // 2^(7-e) in two steps: each
                const float up2 = __uint_as_float((uint32_t)(127 + (7 - e) - (7 - e) / 2) << 23);  // one fits fp32
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float f[4], s[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const uint32_t two = x[2 * k + m / 2];
                        f[m] = __uint_as_float(m & 1 ? two & 0xffff0000u : two << 16) * up1 * up2;
                    }
                    hi[k] = f32x2_to_e4m3x2(f[0], f[1]) | f32x2_to_e4m3x2(f[2], f[3]) << 16;
                    uint32_t h01, h23;
                    e4m3x4_to_f16x2x2(hi[k], h01, h23);
                    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
                        : "=f"(s[0]), "=f"(s[1]) : "r"(h01));
                    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
                        : "=f"(s[2]), "=f"(s[3]) : "r"(h23));
                    lo[k] = f32x2_to_e4m3x2(f[0] - s[0], f[1] - s[1]) | f32x2_to_e4m3x2(f[2] - s[2], f[3] - s[3]) << 16;
                }
                const int sw = D == 128 ? (c ^ (row & 7)) : (c ^ ((row >> 1) & 3));
                const int at = row * D + sw * 16;
                // the parts' rows follow one another: RP is a multiple of 8, so both swizzle alike
                sts128(smem_u32(sq + at), hi[0], hi[1], hi[2], hi[3]);
                sts128(smem_u32(sq + RP * D + at), lo[0], lo[1], lo[2], lo[3]);
                if (c == 0) {
                    const float down = __uint_as_float((uint32_t)(127 + (e - 7)/2) << 23) *
                                       __uint_as_float((uint32_t)(127 + (e - 7) - (e - 7) / 2) << 23);
                    s_qs[row] = row < rows ? (odd ? __uint_as_float(0x7fffffffu) : down * p.scale_log2) : 0.f;
                    s_n[row] = kUnset;
                    s_lim[row] = row < rows ? max(en.seen0 + i, 0) : 0;
                }
            }
            if (wg == 0 && tl < D) s_nan[tl] = 0x7fffffff;
            fence_proxy_async_smem();
            group_sync(bar_id, 128);
            if (lane == 0) mbar_arrive(smem_u32(q_full));

            float ks, vs;
            load_scales(w.tile0, pg0, ks, vs);
            float l[RW];
#pragma unroll
            for (int r = 0; r < RW; ++r) l[r] = 0.f;

            for (int tile = w.tile0; tile < w.tile1; ++tile, ++it) {
                const int pg2 = page_at(tile + 2);
                float ks_next, vs_next;
                load_scales(tile + 1, pg1, ks_next, vs_next);
                const bool absent = pg0 < 0;
                const bool tiny = vs < kTinyScale;
                const float vs_used = tiny ? kTinyScale : vs;
                const float lv = log2_fast(vs_used), inv = __frcp_rn(vs_used);
                const float fix = tiny ? vs * (1.f / kTinyScale) : 1.f;

                wait(smem_u32(s_full + (it & 1)), (it >> 1) & 1, kErrConsumerWait);
                tc_fence_after_sync();
                float t[RW];
                const uint32_t sc = lanes + (it & 1) * C::kScoreCols + r0;
                if constexpr (C::kConcat) {
                    float both[16];
                    tmem_ld<16>(sc, both);
                    tmem_wait_ld();
#pragma unroll
                    for (int r = 0; r < 8; ++r) t[r] = both[r] + both[8 + r];
                } else {
#pragma unroll
                    for (int r = 0; r < RW; r += 16) tmem_ld<16>(sc + r, t + r);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int r = 0; r < RW; r += 4) {
                    const float4 qs = *reinterpret_cast<const float4*>(s_qs + r0 + r);
                    t[r] = fmaf(t[r] * qs.x, ks, lv);
                    t[r + 1] = fmaf(t[r + 1] * qs.y, ks, lv);
                    t[r + 2] = fmaf(t[r + 2] * qs.z, ks, lv);
                    t[r + 3] = fmaf(t[r + 3] * qs.w, ks, lv);
                }
                const int j = tile * kTile + tl;
                if ((tile + 1) * kTile > en.seen_first || __any_sync(~0u, absent)) {
#pragma unroll
                    for (int r = 0; r < RW; ++r)
                        if (absent || j >= s_lim[r0 + r]) t[r] = -INFINITY;
                    // values that some row must not see: zeros past the end, and NaN codes of the
                    // new tokens (0 x NaN would reach every row) noted by dim and taken out
                    if (wg == 0) {
                        wait(smem_u32(full + it % ST), (it / ST) & 1, kErrConsumerWait);
                        unsigned char* row = tiles + (size_t)(it % ST) * 2 * C::kTileBytes + C::kTileBytes + tl * D;
                        if (absent) {
#pragma unroll
                            for (int c = 0; c < D; c += 16) sts128(smem_u32(row + c), 0, 0, 0, 0);
                        } else if (j >= en.seen_first) {
                            for (int c = 0; c < D; c += 4) {
                                uint32_t* word = reinterpret_cast<uint32_t*>(row + c);
                                const uint32_t bad = __vcmpeq4(*word & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                if (bad) {
                                    *word &= ~bad;
                                    const int chunk = D == 128 ? (c / 16) ^ (tl & 7) : (c / 16) ^ ((tl >> 1) & 3);
                                    for (int k = 0; k < 4; ++k)
                                        if (bad >> (8 * k) & 1) atomicMin(s_nan + chunk * 16 + c % 16 + k, j);
                                }
                            }
                        }
                    }
                }
                // keep every probability below the top of the e4m3 range
                float top = -INFINITY;
#pragma unroll
                for (int r = 0; r < RW; r += 4) {
                    const float4 n = *reinterpret_cast<const float4*>(s_n + r0 + r);
                    top = fmaxf(top, fmaxf(fmaxf(t[r] + n.x, t[r + 1] + n.y), fmaxf(t[r + 2] + n.z, t[r + 3] + n.w)));
                }
                if (group_any(bar_id, 128, top > kTop)) {
                    float m0 = 0.f;
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        const float m = warp_max_f32(t[r]);
                        if (lane == (r & 31)) m0 = m;
                        if ((r & 31) == 31 || r == RW - 1)
                            if (lane <= (r & 31)) red[wq * RW + (r & ~31) + lane] = m0;
                    }
                    group_sync(bar_id, 128);
                    float factor = 1.f;
                    if (tl < RW) {
                        const float m = fmaxf(fmaxf(red[tl], red[RW + tl]), fmaxf(red[2 * RW + tl], red[3 * RW + tl]));
                        const float n = s_n[r0 + tl];
                        if (m + n > kTop && m > -INFINITY) {
                            factor = exp2_fast(kTarget - m - n);
                            s_n[r0 + tl] = kTarget - m;
                        }
                    }
                    group_sync(bar_id, 128);
                    if (tl < RW) red[tl] = factor;
                    group_sync(bar_id, 128);
#pragma unroll
                    for (int r = 0; r < RW; ++r) l[r] *= red[r];
                    if (tile > w.tile0) {
                        wait(smem_u32(pv_done + ((it - 1) & 1)), ((it - 1) >> 1) & 1, kErrConsumerWait);
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int part = 0; part < 2; ++part)
#pragma unroll 1
                            for (int r = 0; r < RW; r += 8) {
                                float o[8];
                                const uint32_t at = lanes + C::kOutCol + part * RP + r0 + r;
                                tmem_ld<8>(at, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 8; ++k) o[k] *= red[r + k];
                                tmem_st8(at, o);
                            }
                        tmem_wait_st();
                    }
                }
                if (it >= 2) wait(smem_u32(pv_done + (it & 1)), ((it - 2) >> 1) & 1, kErrConsumerWait);
                unsigned char* dst = sp + (it & 1) * C::kPBytes + tl * 16;
                const bool any_tiny = __any_sync(~0u, tiny);
#pragma unroll
                for (int r = 0; r < RW; r += 16) {
                    constexpr int kRows = RW < 16 ? RW : 16;
                    uint32_t hi[kRows / 4], lo[kRows / 4];
#pragma unroll
                    for (int k = 0; k < kRows; k += 4) {
                        const float4 n = *reinterpret_cast<const float4*>(s_n + r0 + r + k);
                        float e[4] = {exp2_fast(t[r + k] + n.x), exp2_fast(t[r + k + 1] + n.y),
                                      exp2_fast(t[r + k + 2] + n.z), exp2_fast(t[r + k + 3] + n.w)};
#pragma unroll
                        for (int m = 0; m < 4; ++m) l[r + k + m] = fmaf(e[m], inv, l[r + k + m]);
                        if (any_tiny)
#pragma unroll
                            for (int m = 0; m < 4; ++m) e[m] *= fix;
                        uint32_t h0, l0, h1, l1;
                        split_e4m3(e[0], e[1], h0, l0);
                        split_e4m3(e[2], e[3], h1, l1);
                        hi[k / 4] = h0 | h1 << 16;
                        lo[k / 4] = l0 | l1 << 16;
                    }
                    if constexpr (RW == 8) {
                        sts128(smem_u32(dst), hi[0], hi[1], lo[0], lo[1]);
                    } else {
                        sts128(smem_u32(dst + (r0 + r) / 16 * (kTile * 16)), hi[0], hi[1], hi[2], hi[3]);
                        sts128(smem_u32(dst + (RP + r0 + r) / 16 * (kTile * 16)), lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(p_full + (it & 1)));
                pg0 = pg1;
                pg1 = pg2;
                ks = ks_next;
                vs = vs_next;
            }

            // ---------------------------------------- the segment's sums
            wait(smem_u32(pv_done + ((it - 1) & 1)), ((it - 1) >> 1) & 1, kErrConsumerWait);
            tc_fence_after_sync();
            group_sync(bar_id, 128);                 // red: the last maxima have been read
#pragma unroll
            for (int r = 0; r < RW; r += 16) {
                constexpr int kRows = RW < 16 ? RW : 16;
                float v[kRows];
#pragma unroll
                for (int k = 0; k < kRows; ++k) v[k] = l[r + k];
                warp_sums<kRows>(v, lane);
                if (lane % (32 / kRows) == 0) red[wq * RW + r + lane_value<kRows>(lane)] = v[0];
            }
            group_sync(bar_id, 128);
            const bool whole = w.whole();
            const int cta_slot = blockIdx.x * 2 + slot;
            const int dim = wq * kDimLanes + lane;
            const int nan_from = lane < kDimLanes ? s_nan[dim] : 0x7fffffff;
            float* po = p.partial + (size_t)cta_slot * RP * D;
            float* ps = p.partial + (size_t)gridDim.x * 2 * RP * D + (size_t)cta_slot * RP * 2;
#pragma unroll 1
            for (int r = 0; r < RW; r += 8) {
                if (r0 + r >= rows) break;
                float a[8], b[8];
                tmem_ld<8>(lanes + C::kOutCol + r0 + r, a);
                tmem_ld<8>(lanes + C::kOutCol + RP + r0 + r, b);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int row = r0 + r + k;
                    if (row >= rows) break;
                    const float sum = (red[r + k] + red[RW + r + k]) + (red[2 * RW + r + k] + red[3 * RW + r + k]);
                    float o = fmaf(b[k], 1.f / 16, a[k]);
                    if (nan_from < s_lim[row]) o = __uint_as_float(0x7fffffffu);
                    const int i = row / p.group, g = row - i * p.group;
                    const size_t at = (size_t)(en.row0 + i) * p.q_heads + w.head * p.group + g;
                    if (whole) {
                        if (lane < kDimLanes) p.out[at * D + dim] = f32_to_bf16_rne(sum == 0.f ? 0.f : o / sum);
                        if (p.lse && tl == 0)
                            p.lse[at] = sum == 0.f ? -INFINITY : (log2f(sum) - s_n[row]) * 0.693147180559945f;
                    } else {
                        if (lane < kDimLanes) po[(size_t)row * D + dim] = o;
                        if (tl == 0) {
                            ps[2 * row] = s_n[row];
                            ps[2 * row + 1] = sum;
                        }
                    }
                }
            }
            if (!whole && w.tile0 == 0 && tid == 0) {
                // this CTA begins a split item
                const int last = attn_cta_of(total, total < gridDim.x ? (int)total : (int)gridDim.x,
                                             w.item_begin + en.tiles - 1);
                p.split[blockIdx.x] = AttnSplit{last - (int)blockIdx.x + 1, slot, en.row0, rows, w.head};
            }
            slot = 1;
        } while (w.next(p));
        tc_fence_before_sync();
    }
    __syncthreads();
    if (warp == kMma) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmem);
    }
}

// Joins the partial sums of split items, CTA by CTA in order: a warp each row.
template <int D>
__global__ void __launch_bounds__(128) attention_combine_kernel(const __grid_constant__ AttnParams p, int rp, int grid) {
    griddep_wait();
    griddep_launch_dependents();
    const int c = blockIdx.x, row = blockIdx.y * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const AttnSplit s = p.split[c];
    if (s.n == 0 || row >= s.rows) return;
    const float* stats = p.partial + (size_t)grid * 2 * rp * D;
    auto slot = [&](int i) { return (size_t)(2 * (c + i) + (i == 0 ? s.slot0 : 0)); };
    float least = 1e30f;
    for (int i = lane; i < s.n; i += 32) least = fminf(least, stats[(slot(i) * rp + row) * 2]);
    least = -warp_max_f32(-least);
    constexpr int V = D / 32;
    float acc[V] = {}, sum = 0.f;
#pragma unroll 4
    for (int i = 0; i < s.n; ++i) {
        const size_t at = slot(i) * rp + row;
        const float2 st = *reinterpret_cast<const float2*>(stats + at * 2);
        const float f = exp2_fast(least - st.x);
        sum = fmaf(f, st.y, sum);
        const float* o = p.partial + at * D + lane * V;
        if constexpr (V == 4) {
            const float4 x = *reinterpret_cast<const float4*>(o);
            acc[0] = fmaf(f, x.x, acc[0]);
            acc[1] = fmaf(f, x.y, acc[1]);
            acc[2] = fmaf(f, x.z, acc[2]);
            acc[3] = fmaf(f, x.w, acc[3]);
        } else {
            const float2 x = *reinterpret_cast<const float2*>(o);
            acc[0] = fmaf(f, x.x, acc[0]);
            acc[1] = fmaf(f, x.y, acc[1]);
        }
    }
    const int i = row / p.group, g = row - i * p.group;
    const size_t at = (size_t)(s.row0 + i) * p.q_heads + s.head * p.group + g;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint32_t packed[V / 2];
#pragma unroll
    for (int k = 0; k < V / 2; ++k)
        packed[k] = sum == 0.f ? 0u
                               : f32_to_bf16_rne(acc[2 * k] * inv) | (uint32_t)f32_to_bf16_rne(acc[2 * k + 1] * inv) << 16;
    uint32_t* out = reinterpret_cast<uint32_t*>(p.out + at * D) + lane * (V / 2);
    if constexpr (V == 4)
        *reinterpret_cast<uint2*>(out) = make_uint2(packed[0], packed[1]);
    else
        *out = packed[0];
    if (p.lse && lane == 0) p.lse[at] = sum == 0.f ? -INFINITY : (log2f(sum) - least) * 0.693147180559945f;
}

// ---------------------------------------------------------------- launch

struct AttnLaunch {
    CUtensorMap tk, tv;
    AttnParams p;
    int grid;
    cudaStream_t stream;
};

// RP, resident CTAs per SM of the instance for `rows` rows.
inline int attn_rows_padded(int rows) {
    for (int rp : {8, 16, 32, 48, 64, 96, 128})
        if (rows <= rp) return rp;
    return 0;
}
inline int attn_ctas_per_sm(int rp) { return rp > 48 ? 1 : 2; }

cudaError_t launch_attention_d64(int rp, const AttnLaunch& a);
cudaError_t launch_attention_d128(int rp, const AttnLaunch& a);

}  // namespace dl
