// Attention over the paged 8-bit cache on the 5th-generation tensor cores.
//
// The mathematics.  For one key/value head and the rows r (a new token and one
// of the query heads that share the key/value head), over the cached tokens j:
//     t_jr = c * ks_j * (q_r . k_j) + log2 vs_j ,   c = scale * log2 e,
//     P_jr = 2^(t_jr + n_r) ,   o_r = sum_j P_jr v_j / sum_j (P_jr / vs_j),
// k_j, v_j the stored codes and ks_j, vs_j the scales of their blocks.  Folding
// vs_j into the exponent makes P_jr the token's true weight on its codes, so n_r
// bounds what is multiplied, and costs nothing per element.  n_r places the
// first tile's largest P (kTarget) and moves only when one passes the top (kTop).
//
// Both products run on the tensor cores with tokens on the TMEM lanes:
//     S^T [128 tokens x rows] = K [128 x D] . Q^T
//     O^T [D x rows]         += V^T [D x 128] . P^T
// S is kind::f8f6f4 on the codes as they lie in the cache.  A bf16 query has 8
// significant bits and an e4m3 number 4, so a query is the sum of two e4m3 parts,
// exact down to 2^-17 of the row's largest element (each row is scaled to the top of
// the range).  O has two forms:
//   up to 16 rows  kind::f8f6f4 on the codes too, P as four e4m3 parts of 16 times
//                  each other's scale, in columns of their own: 11 bits (an fp16
//                  step comes first) down to 2^-13 of the row's largest, 2^-21 of
//                  it absolute below.  Nothing touches a value but the MMA: shared
//                  memory moves 64 KB a tile, half of what the other form moves.
//   more rows      kind::f16: values widened to fp16 (exact), P rounded to fp16:
//                  relative 2^-12, absolute 2^-28 of the row's largest.  The
//                  widening costs the same for any rows, the parts 7
//                  instructions for each probability.
// (Two parts of P would do for even weights, but leave 18 bits of range for both the
// tokens that weigh little and a maximum that grows: moving n_r took most of the time
// at 128 rows.)  Scores, maxima, exponentials, sums and accumulators are fp32.
//
// A CTA runs a contiguous range of 128-token tiles of the whole call (sequence,
// row tile, head, tile), the same number for every CTA to within one: the work
// of a long sequence spreads over the chip, and many short ones pack.  A
// sequence that ends up on several CTAs leaves partial sums in the workspace,
// joined in a fixed order by attention_combine_kernel.
#pragma once

#include <type_traits>

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

// RP rows.  The softmax warpgroups are TG tile groups, which take tiles in turn
// and have accumulators of their own, of CG column groups of RW rows each.  A
// tile's chain of waits and dependent instructions is about as long as its share of
// the memory's time, so two tiles are in work on an SM: two CTAs up to 16 rows, two
// tile groups to 64; beyond, registers leave room for one tile.
template <int D_, int RP_>
struct AttnShape {
    static constexpr int D = D_, RP = RP_;
    static constexpr bool kParts = RP <= 16;            // P as e4m3 parts (else fp16)
    static constexpr int TG = RP > 16 && RP <= 64 ? 2 : 1;
    static constexpr int CG = RP > 64 ? 4 : RP > 48 ? 2 : 1;
    static constexpr int NWG = TG * CG;
    static constexpr int RW = RP / CG;
    static constexpr bool kConcat = kParts;             // S columns: hi parts, then lo parts
    static constexpr int kScoreCols = kConcat ? 2 * RP : RP;
    static constexpr int kOutCol = 2 * kScoreCols;
    static constexpr int kOutCols = kParts ? 4 * RP : RP;
    static constexpr int kCols = kOutCol + TG * kOutCols;
    static constexpr int kTmem = kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static constexpr int kCtas = kParts ? 2 : 1;        // resident CTAs per SM
    static constexpr int kThreads = NWG * 128 + 96;
    static constexpr int kTileBytes = kTile * D;        // codes of K, and of V
    static constexpr int kQBytes = 2 * RP * D;
    static constexpr int kPBytes = kOutCols * kTile * (kParts ? 1 : 2);
    static constexpr int kVBytes = kParts ? 0 : kTile * D * 2;      // widened values
    static constexpr int kPBufs = RP < 96 ? 2 : 1, kVBufs = 2;
    static constexpr int kMisc = 1024 + RP * (8 + 8 * TG) + NWG * 4 * RW * 4 + D * 4 + 256;
    static constexpr int kBudget = (kCtas == 1 ? 227 : 113) * 1024;
    // a tile's slot: its codes, and 16 bytes a token of values made from the scales
    static constexpr int kPairBytes = 2 * kTileBytes + kTile * 16;
    static constexpr int kRoom = kBudget - 1024 - kQBytes - kPBufs * kPBytes - kVBufs * kVBytes - kMisc;
    static constexpr int kKeySlots = kRoom / kPairBytes > 6 ? 6 : kRoom / kPairBytes;
    static constexpr int kMore = kRoom - kKeySlots * kPairBytes >= kTileBytes + kTile * 16 ? 1 : 0;
    static constexpr int kValueSlots = kKeySlots + kMore;
    static constexpr size_t kSmem = 1024 + (size_t)kKeySlots * kTileBytes + (size_t)kValueSlots * (kTileBytes + kTile * 16) +
                                    kQBytes + kPBufs * kPBytes + kVBufs * kVBytes + kMisc;
    static_assert(kKeySlots >= 2, "two tiles in flight");
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

// Instruction descriptor, M x N with an fp32 accumulator: e4m3 x e4m3 for
// kind::f8f6f4, fp16 x fp16 for kind::f16; mn = 1: both operands have their M / N
// dimension contiguous in memory.
__host__ __device__ constexpr uint32_t umma_idesc(int m, int n, int mn) {
    return (1u << 4) | (mn ? 3u << 15 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// D[taddr] (+)= A . B^T for one K step of 16, fp16 operands.
__device__ __forceinline__ void umma_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate) : "memory");
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

// Pairs of fp32 in one 64-bit register: Blackwell's two-wide multiply, add and
// fused multiply-add.
using F2 = unsigned long long;
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack(F2 v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Four floats of shared memory as two pairs.
__device__ __forceinline__ void lds_f2x2(const float* p, F2& a, F2& b) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    a = v.x;
    b = v.y;
}

// Four probabilities -> their four e4m3 parts, each the rest of the one before
// times 16.  The fp16 step in between rounds to 2^-11.
__device__ __forceinline__ void split_e4m3(const float (&e)[4], uint32_t (&part)[4]) {
    constexpr uint32_t kSixteen = 0x4C004C00u;          // f16x2
    uint32_t x = f32x2_to_f16x2(e[0], e[1]), y = f32x2_to_f16x2(e[2], e[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        asm("{\n\t"
            ".reg .b16 a, b;\n\t"
            ".reg .b32 u, v;\n\t"
            "cvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n\t"
            "cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 u, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 v, b;\n\t"
            "sub.rn.f16x2 u, %1, u;\n\t"
            "sub.rn.f16x2 v, %2, v;\n\t"
            "mul.rn.f16x2 %1, u, %3;\n\t"
            "mul.rn.f16x2 %2, v, %3;\n\t"
            "mov.b32 %0, {a, b};\n\t"
            "}"
            : "=r"(part[i]), "+r"(x), "+r"(y) : "r"(kSixteen));
    }
}

// The smaller one; NaN if either is.
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The factor of a row's sums when its n moves by x.  A first n may move up: the sums are still 0.
__device__ __forceinline__ float shrink(float x) { return exp2_fast(fminf(x, 0.f)); }

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

// What the softmax needs of a token, from its scales: c * ks, log2 vs, 1 / vs
// (< 0: the token is absent) and a factor of P, 1 but for scales below 2^-60.
struct __align__(16) TokenScales {
    float key, log_value, inv_value, fix;
};

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas)
attention_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const __grid_constant__ AttnParams p) {
    constexpr int D = C::D, RP = C::RP, RW = C::RW, TG = C::TG, CG = C::CG, NWG = C::NWG;
    constexpr int NK = C::kKeySlots, NV = C::kValueSlots;
    constexpr int kProducer = NWG * 4, kMma = NWG * 4 + 1, kScaler = NWG * 4 + 2;
    constexpr int kAllBar = NWG + 1, kSoftmax = NWG * 128;
    // one accumulator lane per dim: M = 64 leaves 16 rows in each warp's lanes
    constexpr int kDimLanes = D / 4;
    constexpr uint32_t kSwizzle = D == 128 ? 2 : 4;
    // largest exponent of a probability (log2 448 = 8.807; fp16 ends at 2^16), and the one a maximum gets
    constexpr float kTop = C::kParts ? 8.8f : 15.9f, kTarget = C::kParts ? -1.f : 3.f;
    constexpr float kTinyScale = 8.67361737988403547e-19f;       // 2^-60

    extern __shared__ unsigned char smem_raw[];
    unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    unsigned char* sp = base;                                     // P [rows / 16 bytes][128 tokens][16 bytes]
    unsigned char* sq = sp + C::kPBufs * C::kPBytes;              // query parts [2][RP][D]
    unsigned char* sv = sq + C::kQBytes;                          // widened values [dims / 64][128 tokens][64]
    unsigned char* keys = sv + C::kVBufs * C::kVBytes;            // codes, [128 tokens][D] each
    unsigned char* values = keys + NK * C::kTileBytes;
    TokenScales* scales = reinterpret_cast<TokenScales*>(values + NV * C::kTileBytes);   // [NV][128]
    unsigned char* misc = reinterpret_cast<unsigned char*>(scales + NV * kTile);
    uint64_t* bars = reinterpret_cast<uint64_t*>(misc);
    uint64_t *k_full = bars, *k_empty = k_full + NK, *v_full = k_empty + NK, *v_empty = v_full + NV,
             *s_full = v_empty + NV, *p_full = s_full + 2, *pv_done = p_full + 2, *q_full = pv_done + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 1);
    int* s_stop = reinterpret_cast<int*>(tmem_slot + 1);
    long long* s_walk = reinterpret_cast<long long*>(misc + 512);     // total, begin, end, entry, within
    int* s_force = reinterpret_cast<int*>(misc + 576);                // [NWG] a row has no n_r yet
    int* s_flags = reinterpret_cast<int*>(misc + 640);                // [NV] kAbsent: some token is, kTiny: some scale is
    float* s_qs = reinterpret_cast<float*>(misc + 1024);              // [RP] a row's query scale
    int* s_lim = reinterpret_cast<int*>(s_qs + RP);                   // [RP] cached tokens a row sees
    float* s_n = reinterpret_cast<float*>(s_lim + RP);                // [TG][RP] n_r
    float* s_l = s_n + TG * RP;                                       // [TG][RP] sums of P / vs
    float* s_red = s_l + TG * RP;                                     // [NWG][4][RW]
    int* s_nan = reinterpret_cast<int*>(s_red + NWG * 4 * RW);        // [D] first NaN among the new tokens' values
    constexpr int kAbsent = 1, kTiny = 2;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const CtaWait wait{{p.err_word, p.wait_limit_ns}, s_stop};

    if (warp == kMma) {
        if (lane == 0) {
            for (int i = 0; i < NK; ++i) {
                mbar_init(smem_u32(k_full + i), 1);
                mbar_init(smem_u32(k_empty + i), 1);
            }
            for (int i = 0; i < NV; ++i) {
                mbar_init(smem_u32(v_full + i), 2);                    // the codes, the scales
                mbar_init(smem_u32(v_empty + i), C::kParts ? 1 : CG * 4);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_u32(s_full + i), 1);
                mbar_init(smem_u32(p_full + i), CG * 4);
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
        // ------------------------------------------------ loads: a page's rows each lane, keys by
        // lanes 0 to 15, values by the others
        const int box = min(p.page_size, kTile), per = kTile / box;
        const bool is_v = lane >= 16;
        const int sub = lane & 15;
        int it = 0;
        bool ok = true;
        do {
            const int* table = p.s.block_table + (size_t)w.entry.b * p.s.table_cols;
            auto page_of = [&](int tile) {
                const int j = tile * kTile + sub * box;
                int pg = -1;
                if (sub < per && j < w.entry.seen_last) pg = table[j >> p.page_shift];
                return (unsigned)pg < (unsigned)p.num_pages ? pg : -1;
            };
            int page = page_of(w.tile0);
            for (int tile = w.tile0; tile < w.tile1; ++tile, ++it) {
                const int next = tile + 1 < w.tile1 ? page_of(tile + 1) : -1;
                const uint32_t bytes = (uint32_t)(__popc(__ballot_sync(~0u, page >= 0) & 0xffff) * box * D);
                const int at = (tile * kTile + sub * box) & (p.page_size - 1);
                const int ks = it % NK, vs = it % NV;
                if (it >= NK) ok = __all_sync(~0u, wait(smem_u32(k_empty + ks), (it / NK - 1) & 1, kErrProducerWait));
                if (!ok) break;
                if (lane == 0) mbar_arrive_expect_tx(smem_u32(k_full + ks), bytes);
                __syncwarp();
                if (page >= 0 && !is_v)
                    tma_load_4d(smem_u32(keys + ks * C::kTileBytes + sub * box * D), &tk, smem_u32(k_full + ks), 0, at,
                                w.head, page);
                if (it >= NV) ok = __all_sync(~0u, wait(smem_u32(v_empty + vs), (it / NV - 1) & 1, kErrProducerWait));
                if (!ok) {
                    mbar_wait_bounded(smem_u32(k_full + ks), (it / NK) & 1, wait.ctl, kErrDrainWait);
                    break;
                }
                if (lane == 16) mbar_arrive_expect_tx(smem_u32(v_full + vs), bytes);
                __syncwarp();
                if (page >= 0 && is_v)
                    tma_load_4d(smem_u32(values + vs * C::kTileBytes + sub * box * D), &tv, smem_u32(v_full + vs), 0, at,
                                w.head, page);
                page = next;
            }
        } while (ok && w.next(p));
        // after a wait that gave up: no copy of this CTA may still be in flight when it leaves
        if (!ok) {
            for (int i = max(it - NK, 0); i < it; ++i)
                mbar_wait_bounded(smem_u32(k_full + i % NK), (i / NK) & 1, wait.ctl, kErrDrainWait);
            for (int i = max(it - NV, 0); i < it; ++i)
                mbar_wait_bounded(smem_u32(v_full + i % NV), (i / NV) & 1, wait.ctl, kErrDrainWait);
        }
    } else if (work && warp == kScaler) {
        // ------------------------------------------------ scales: four tokens each lane; a tile's
        // pages are read two tiles ahead, its scales one
        int it = 0;
        bool ok = true;
        do {
            const int* table = p.s.block_table + (size_t)w.entry.b * p.s.table_cols;
            auto pages_of = [&](int tile, int (&pg)[4]) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int j = tile * kTile + 32 * k + lane;
                    pg[k] = -1;
                    if (tile < w.tile1 && j < w.entry.seen_last) pg[k] = table[j >> p.page_shift];
                }
            };
            auto load = [&](int tile, const int (&pg)[4], float (&a)[4], float (&b)[4]) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    a[k] = 0.f;
                    b[k] = -1.f;
                    if ((unsigned)pg[k] < (unsigned)p.num_pages) {
                        const int t = (tile * kTile + 32 * k + lane) & (p.page_size - 1);
                        const long long o = pg[k] * p.scale_page_stride + w.head * p.scale_head_stride + (t >> p.block_shift);
                        a[k] = p.k_scale[o];
                        b[k] = p.v_scale[o];
                    }
                }
            };
            int pg[4], next[4];
            float a[4], b[4];
            pages_of(w.tile0, pg);
            pages_of(w.tile0 + 1, next);
            load(w.tile0, pg, a, b);
            for (int tile = w.tile0; tile < w.tile1; ++tile, ++it) {
                float a1[4], b1[4];
                int later[4];
                load(tile + 1, next, a1, b1);
                pages_of(tile + 2, later);
                const int s = it % NV;
                if (it >= NV) ok = __all_sync(~0u, wait(smem_u32(v_empty + s), (it / NV - 1) & 1, kErrProducerWait));
                if (!ok) break;
                int flags = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool absent = (unsigned)pg[k] >= (unsigned)p.num_pages;
                    const bool tiny = !absent && b[k] < kTinyScale;
                    const float used = absent ? 1.f : tiny ? kTinyScale : b[k];
                    flags |= (absent ? kAbsent : 0) | (tiny ? kTiny : 0);
                    scales[s * kTile + 32 * k + lane] =
                        TokenScales{a[k], log2_fast(used), absent ? -1.f : __frcp_rn(used), tiny ? b[k] * (1.f / kTinyScale) : 1.f};
                }
                flags = __reduce_or_sync(~0u, flags);
                if (lane == 0) s_flags[s] = flags;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(v_full + s));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    pg[k] = next[k];
                    next[k] = later[k];
                    a[k] = a1[k];
                    b[k] = b1[k];
                }
            }
        } while (ok && w.next(p));
    } else if (work && warp == kMma) {
        // ------------------------------------------------ products, issued by one lane
        if (lane == 0) {
            constexpr uint32_t kScoreIdesc = umma_idesc(128, C::kScoreCols, 0);
            constexpr uint32_t kOutIdesc = umma_idesc(D, C::kOutCols, 1);
            const uint32_t q0 = smem_u32(sq);
            int it = 0, seg = 0;
            bool ok = true;
            auto scores = [&](int i) {
                if (!wait(smem_u32(k_full + i % NK), (i / NK) & 1, kErrConsumerWait)) return false;
                tc_fence_after_sync();
                const uint32_t k0 = smem_u32(keys + i % NK * C::kTileBytes);
                const uint32_t d = tmem + (i & 1) * C::kScoreCols;
#pragma unroll
                for (int part = 0; part < (C::kConcat ? 1 : 2); ++part)
#pragma unroll
                    for (int k = 0; k < D / 32; ++k)
                        umma_e4m3(d, umma_desc(k0 + 32 * k, 16, 8 * D, kSwizzle),
                                  umma_desc(q0 + part * RP * D + 32 * k, 16, 8 * D, kSwizzle), kScoreIdesc,
                                  part > 0 || k > 0);
                umma_commit(smem_u32(s_full + (i & 1)));
                umma_commit(smem_u32(k_empty + i % NK));
                return true;
            };
            do {
                ok = wait(smem_u32(q_full), seg & 1, kErrConsumerWait) && scores(it);
                for (int tile = w.tile0; tile < w.tile1 && ok; ++tile, ++it) {
                    if (tile + 1 < w.tile1 && !(ok = scores(it + 1))) break;
                    if (!(ok = wait(smem_u32(p_full + (it & 1)), (it >> 1) & 1, kErrConsumerWait))) break;
                    tc_fence_after_sync();
                    const uint32_t p0 = smem_u32(sp + it % C::kPBufs * C::kPBytes);
                    const uint32_t o = tmem + C::kOutCol + (TG == 2 ? (it & 1) * C::kOutCols : 0);
                    const bool more = tile - w.tile0 >= TG;          // this accumulator holds something
                    if constexpr (C::kParts) {
                        const uint32_t v0 = smem_u32(values + it % NV * C::kTileBytes);
#pragma unroll
                        for (int k = 0; k < kTile / 32; ++k)
                            umma_e4m3(o, umma_desc(v0 + k * 32 * D, 16, 8 * D, kSwizzle),
                                      umma_desc(p0 + k * 32 * 16, 128, kTile * 16, 0), kOutIdesc, more || k > 0);
                        umma_commit(smem_u32(v_empty + it % NV));
                    } else {
                        const uint32_t v0 = smem_u32(sv + it % C::kVBufs * C::kVBytes);
#pragma unroll
                        for (int k = 0; k < kTile / 16; ++k)
                            umma_f16(o, umma_desc(v0 + k * 16 * 128, kTile * 128, 1024, 2),
                                     umma_desc(p0 + k * 16 * 16, 128, kTile * 16, 0), kOutIdesc, more || k > 0);
                    }
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
        const int tg = wg / CG, r0 = wg % CG * RW;          // tile group, first row
        const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
        float* red = s_red + wg * 4 * RW;
        float* my_n = s_n + tg * RP + r0;
        int it0 = 0;                                        // the segment's first tile, counted by the CTA
        int slot = 0;
        auto pv_wait = [&](int i) {         // the product of tile i has been made
            if (i >= 0) wait(smem_u32(pv_done + (i & 1)), (i >> 1) & 1, kErrConsumerWait);
        };
        do {
            const AttnEntry& en = w.entry;
            const int rows = en.tokens * p.group, tiles = w.tile1 - w.tile0;

            // the row tile's queries as two e4m3 parts, each row scaled to the top of the range
            group_sync(kAllBar, kSoftmax);
            constexpr int TPR = D / 16;             // threads of a row, 16 elements each
            for (int row = tid / TPR; row < RP; row += kSoftmax / TPR) {
                const int c = tid % TPR;
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
                const unsigned mates = TPR == 8 ? 0xffu << (lane & 24) : 0xfu << (lane & 28);
#pragma unroll
                for (int o = TPR / 2; o; o >>= 1) top = max(top, __shfl_xor_sync(mates, top, o));
                // 2^e <= largest < 2^(e+1) becomes [128, 256); a row with an infinity or a NaN answers NaN
                const int e = max((int)(top >> 7), 1) - 127;
                const bool odd = (top >> 7) == 255;
                // 2^(7-e) in two steps: each one fits fp32
                const float up1 = __uint_as_float((uint32_t)(127 + (7 - e) / 2) << 23);
                const float up2 = __uint_as_float((uint32_t)(127 + (7 - e) - (7 - e) / 2) << 23);
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
                    const float down = __uint_as_float((uint32_t)(127 + (e - 7) / 2) << 23) *
                                       __uint_as_float((uint32_t)(127 + (e - 7) - (e - 7) / 2) << 23);
                    s_qs[row] = row < rows ? (odd ? __uint_as_float(0x7fffffffu) : down * p.scale_log2) : 0.f;
                    s_lim[row] = row < rows ? max(en.seen0 + i, 0) : 0;
                }
            }
            if (tid < D) s_nan[tid] = 0x7fffffff;
            if (tl < RW) my_n[tl] = 0.f;
            if (tl == 0) s_force[wg] = 1;
            fence_proxy_async_smem();
            group_sync(kAllBar, kSoftmax);
            if (lane == 0) mbar_arrive(smem_u32(q_full));

            F2 l[RW / 2];
#pragma unroll
            for (int r = 0; r < RW / 2; ++r) l[r] = 0;
            uint32_t unset = ~0u;            // threads below RW: this row has no n_r yet
            const int t_first = TG == 2 ? (it0 + tg) & 1 : 0;       // the group's tiles have its parity
            for (int t = t_first; t < tiles; t += TG) {
                const int it = it0 + t, tile = w.tile0 + t, j = tile * kTile + tl;
                wait(smem_u32(v_full + it % NV), (it / NV) & 1, kErrConsumerWait);
                const TokenScales ts = scales[it % NV * kTile + tl];
                const int flags = s_flags[it % NV];
                const bool absent = ts.inv_value < 0.f;
                const bool masked = (tile + 1) * kTile > en.seen_first || (flags & kAbsent);

                // exponents t + n
                wait(smem_u32(s_full + (it & 1)), (it >> 1) & 1, kErrConsumerWait);
                tc_fence_after_sync();
                float d[RW];
                const uint32_t sc = lanes + (it & 1) * C::kScoreCols + r0;
                if constexpr (C::kConcat) {
                    float both[2 * RP];
#pragma unroll
                    for (int r = 0; r < 2 * RP; r += 16) tmem_ld<16>(sc + r, both + r);
                    tmem_wait_ld();
#pragma unroll
                    for (int r = 0; r < RW; ++r) d[r] = both[r] + both[RP + r];
                } else {
#pragma unroll
                    for (int r = 0; r + 16 <= RW; r += 16) tmem_ld<16>(sc + r, d + r);
                    if constexpr (RW % 16) tmem_ld<8>(sc + RW - 8, d + RW - 8);
                    tmem_wait_ld();
                }
                const F2 ks2 = f2(ts.key, ts.key), lv2 = f2(ts.log_value, ts.log_value);
#pragma unroll
                for (int r = 0; r < RW; r += 4) {
                    F2 q0, q1, n0, n1;
                    lds_f2x2(s_qs + r0 + r, q0, q1);
                    lds_f2x2(my_n + r, n0, n1);
                    unpack(add2(fma2(mul2(f2(d[r], d[r + 1]), q0), ks2, lv2), n0), d[r], d[r + 1]);
                    unpack(add2(fma2(mul2(f2(d[r + 2], d[r + 3]), q1), ks2, lv2), n1), d[r + 2], d[r + 3]);
                }
                if (masked) {
#pragma unroll
                    for (int r = 0; r < RW; ++r)
                        if (absent || j >= s_lim[r0 + r]) d[r] = -INFINITY;
                }
                float top = -INFINITY;
#pragma unroll
                for (int r = 0; r < RW; r += 2) top = max3(top, d[r], d[r + 1]);
                // a row passes the top, or has no n_r yet: its n_r moves, and its sums follow
                if (group_any(bar_id, 128, top > kTop || (tl == 0 && s_force[wg]))) {
                    float m0 = 0.f;
#pragma unroll
                    for (int r = 0; r < RW; ++r) {
                        const float m = warp_max_f32(d[r]);
                        if (lane == (r & 31)) m0 = m;
                        if ((r & 31) == 31 || r == RW - 1)
                            if (lane <= (r & 31)) red[wq * RW + (r & ~31) + lane] = m0;
                    }
                    group_sync(bar_id, 128);
                    float move = 0.f;
                    if (tl < RW) {
                        const float m = fmaxf(fmaxf(red[tl], red[RW + tl]), fmaxf(red[2 * RW + tl], red[3 * RW + tl]));
                        if (m > -INFINITY && (m > kTop || unset)) {
                            move = kTarget - m;
                            my_n[tl] += move;
                            unset = 0;
                        }
                    }
                    const bool more = group_any(bar_id, 128, tl < RW && unset && r0 + tl < rows);
                    if (tl < RW) red[tl] = move;
                    if (tl == 0) s_force[wg] = more;
                    group_sync(bar_id, 128);
#pragma unroll
                    for (int r = 0; r < RW; r += 4) {
                        const float4 x = *reinterpret_cast<const float4*>(red + r);
                        d[r] = min_nan(d[r] + x.x, kTop);
                        d[r + 1] = min_nan(d[r + 1] + x.y, kTop);
                        d[r + 2] = min_nan(d[r + 2] + x.z, kTop);
                        d[r + 3] = min_nan(d[r + 3] + x.w, kTop);
                        l[r / 2] = mul2(l[r / 2], f2(shrink(x.x), shrink(x.y)));
                        l[r / 2 + 1] = mul2(l[r / 2 + 1], f2(shrink(x.z), shrink(x.w)));
                    }
                    if (t >= TG) {
                        pv_wait(it - TG);
                        tc_fence_after_sync();
#pragma unroll 1
                        for (int r = 0; r < RW; r += 8) {
                            float f[8], o[8];
                            bool same = true;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                f[k] = red[r + k];
                                same &= f[k] == 0.f;
                            }
                            if (same) continue;
#pragma unroll 1
                            for (int part = 0; part < (C::kParts ? 4 : 1); ++part) {
                                const uint32_t at = lanes + C::kOutCol + tg * C::kOutCols + part * RP + r0 + r;
                                tmem_ld<8>(at, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 8; ++k) o[k] *= shrink(f[k]);
                                tmem_st8(at, o);
                            }
                        }
                        tmem_wait_st();
                    }
                }

                // this token's values: what some row must not see is taken out -- all of an absent
                // token, and NaN codes of the new tokens (0 x NaN would reach every row), which
                // are noted by dim -- and, for fp16 products, they are widened
                unsigned char* codes = values + it % NV * C::kTileBytes + tl * D;
                constexpr int kChunks = D / 16 / CG;
                const int c0 = wg % CG * kChunks;
                auto at_chunk = [&](int c) {
                    return reinterpret_cast<uint4*>(codes + (D == 128 ? (c ^ (tl & 7)) : (c ^ ((tl >> 1) & 3))) * 16);
                };
                if (!C::kParts || masked) {
                    if (!C::kParts) pv_wait(it - C::kVBufs);
                    constexpr int kBatch = kChunks < 4 ? kChunks : 4;   // loads before the first store
                    unsigned char* wide = C::kParts ? nullptr : sv + it % C::kVBufs * C::kVBytes + tl * 128;
#pragma unroll
                    for (int i0 = 0; i0 < kChunks; i0 += kBatch) {
                        uint4 x[kBatch];
#pragma unroll
                        for (int i = 0; i < kBatch; ++i) x[i] = *at_chunk(c0 + i0 + i);
                        if (masked) {
#pragma unroll
                            for (int i = 0; i < kBatch; ++i) {
                                const int c = c0 + i0 + i;
                                if (absent) {
                                    x[i] = make_uint4(0, 0, 0, 0);
                                } else if (j >= en.seen_first) {
                                    uint32_t* word = &x[i].x;
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        const uint32_t bad = __vcmpeq4(word[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                        word[k] &= ~bad;
                                        for (int m = 0; bad && m < 4; ++m)
                                            if (bad >> (8 * m) & 1) atomicMin(s_nan + 16 * c + 4 * k + m, j);
                                    }
                                }
                                if (C::kParts) *at_chunk(c) = x[i];
                            }
                        }
                        if constexpr (!C::kParts) {
#pragma unroll
                            for (int i = 0; i < kBatch; ++i) {
                                const int c = c0 + i0 + i, q = c % 4 * 2;
                                uint32_t h[8];
                                e4m3x4_to_f16x2x2(x[i].x, h[0], h[1]);
                                e4m3x4_to_f16x2x2(x[i].y, h[2], h[3]);
                                e4m3x4_to_f16x2x2(x[i].z, h[4], h[5]);
                                e4m3x4_to_f16x2x2(x[i].w, h[6], h[7]);
                                unsigned char* to = wide + c / 4 * (kTile * 128);
                                sts128(smem_u32(to + ((q ^ (tl & 7)) * 16)), h[0], h[1], h[2], h[3]);
                                sts128(smem_u32(to + (((q + 1) ^ (tl & 7)) * 16)), h[4], h[5], h[6], h[7]);
                            }
                        }
                    }
                    if constexpr (!C::kParts) {
                        __syncwarp();
                        if (lane == 0) mbar_arrive(smem_u32(v_empty + it % NV));
                    }
                }

                // probabilities
                if (C::kParts || C::kPBufs < C::kVBufs) pv_wait(it - C::kPBufs);
                unsigned char* dst = sp + it % C::kPBufs * C::kPBytes + tl * 16;
                const F2 inv2 = f2(ts.inv_value, ts.inv_value);
#pragma unroll
                for (int r = 0; r < RW; r += 8) {
                    float e[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) e[k] = exp2_fast(d[r + k]);
#pragma unroll
                    for (int k = 0; k < 8; k += 2) l[(r + k) / 2] = fma2(f2(e[k], e[k + 1]), inv2, l[(r + k) / 2]);
                    if (flags & kTiny)
#pragma unroll
                        for (int k = 0; k < 8; ++k) e[k] *= ts.fix;
                    if constexpr (C::kParts) {
                        // columns: RP of each part, 16 to a chunk of 2 KB
                        uint32_t a[4], b[4];
                        split_e4m3({e[0], e[1], e[2], e[3]}, a);
                        split_e4m3({e[4], e[5], e[6], e[7]}, b);
                        if constexpr (RP == 8) {
                            sts128(smem_u32(dst), a[0], b[0], a[1], b[1]);
                            sts128(smem_u32(dst + kTile * 16), a[2], b[2], a[3], b[3]);
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                *reinterpret_cast<uint2*>(dst + k * (kTile * 16) + r) = make_uint2(a[k], b[k]);
                        }
                    } else {
                        sts128(smem_u32(dst + (r0 + r) / 8 * (kTile * 16)), f32x2_to_f16x2(e[0], e[1]), f32x2_to_f16x2(e[2], e[3]),
                               f32x2_to_f16x2(e[4], e[5]), f32x2_to_f16x2(e[6], e[7]));
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(p_full + (it & 1)));
            }

            // ---------------------------------------- the segment's sums
#pragma unroll
            for (int r = 0; r < RW; r += 8) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; k += 2) unpack(l[(r + k) / 2], v[k], v[k + 1]);
                warp_sums<8>(v, lane);
                if (r == 0) group_sync(bar_id, 128);         // red: the last moves have been read
                if (lane % 4 == 0) red[wq * RW + r + lane_value<8>(lane)] = v[0];
            }
            group_sync(bar_id, 128);
            if (tl < RW)
                s_l[tg * RP + r0 + tl] = (red[tl] + red[RW + tl]) + (red[2 * RW + tl] + red[3 * RW + tl]);
            it0 += tiles;
            pv_wait(it0 - 1);
            if (TG == 2) pv_wait(it0 - 2);
            tc_fence_after_sync();
            group_sync(kAllBar, kSoftmax);
            const bool whole = w.whole();
            const int cta_slot = blockIdx.x * 2 + slot;
            const int dim = wq * kDimLanes + lane;
            const int nan_from = lane < kDimLanes ? s_nan[dim] : 0x7fffffff;
            float* po = p.partial + (size_t)cta_slot * RP * D;
            float* ps = p.partial + (size_t)gridDim.x * 2 * RP * D + (size_t)cta_slot * RP * 2;
#pragma unroll 1
            for (int r = wg * 8; r < rows; r += NWG * 8) {
                float a[8], b[8] = {};
                tmem_ld<8>(lanes + C::kOutCol + r, a);
                if constexpr (C::kParts) {
                    float c[8], e[8];
                    tmem_ld<8>(lanes + C::kOutCol + RP + r, b);
                    tmem_ld<8>(lanes + C::kOutCol + 2 * RP + r, c);
                    tmem_ld<8>(lanes + C::kOutCol + 3 * RP + r, e);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        a[k] = fmaf(fmaf(fmaf(e[k], 1.f / 16, c[k]), 1.f / 16, b[k]), 1.f / 16, a[k]);
                } else {
                    if (TG == 2) tmem_ld<8>(lanes + C::kOutCol + C::kOutCols + r, b);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int row = r + k;
                    if (row >= rows) break;
                    float sum = s_l[row], n = s_n[row], o = a[k];
                    if (TG == 2) {
                        // a group whose sum is 0 saw nothing (or had no tile: its accumulator is stale)
                        const float l0 = sum, l1 = s_l[RP + row], n1 = s_n[RP + row];
                        const float least = fminf(l0 == 0.f ? n1 : n, l1 == 0.f ? n : n1);
                        const float f0 = l0 == 0.f ? 0.f : exp2_fast(least - n), f1 = l1 == 0.f ? 0.f : exp2_fast(least - n1);
                        o = (l0 == 0.f ? 0.f : a[k] * f0) + (l1 == 0.f ? 0.f : b[k] * f1);
                        sum = l0 * f0 + l1 * f1;
                        n = least;
                    }
                    if (nan_from < s_lim[row]) o = __uint_as_float(0x7fffffffu);
                    const int i = row / p.group, g = row - i * p.group;
                    const size_t at = (size_t)(en.row0 + i) * p.q_heads + w.head * p.group + g;
                    if (whole) {
                        if (lane < kDimLanes) p.out[at * D + dim] = f32_to_bf16_rne(sum == 0.f ? 0.f : o / sum);
                        if (p.lse && wq == 0 && lane == 0)
                            p.lse[at] = sum == 0.f ? -INFINITY : (log2f(sum) - n) * 0.693147180559945f;
                    } else {
                        if (lane < kDimLanes) po[(size_t)row * D + dim] = o;
                        if (wq == 0 && lane == 0) {
                            ps[2 * row] = sum == 0.f ? INFINITY : n;           // nothing seen here
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

// Joins the partial sums of split items, CTA by CTA in order.  W warps take a row: 4
// where few items may be split over many CTAs each (their loads would follow one
// another), else 1.
template <int D, int W>
__global__ void __launch_bounds__(128) attention_combine_kernel(const __grid_constant__ AttnParams p, int rp, int grid) {
    constexpr int V = D / 32;
    __shared__ float s_acc[4][D], s_sum[4];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x, row = W == 4 ? blockIdx.y : blockIdx.y * 4 + warp, first = W == 4 ? warp : 0;
    const AttnSplit s = p.split[c];
    if (s.n == 0 || row >= s.rows) return;
    const float* stats = p.partial + (size_t)grid * 2 * rp * D;
    auto slot = [&](int i) { return (size_t)(2 * (c + i) + (i == 0 ? s.slot0 : 0)); };
    float least = INFINITY;
    for (int i = lane; i < s.n; i += 32) least = fminf(least, stats[(slot(i) * rp + row) * 2]);
    least = -warp_max_f32(-least);
    float acc[V] = {}, sum = 0.f;
#pragma unroll 5
    for (int i = first; i < s.n; i += W) {
        const size_t at = slot(i) * rp + row;
        const float2 st = *reinterpret_cast<const float2*>(stats + at * 2);
        const float f = st.x == INFINITY ? 0.f : exp2_fast(least - st.x);
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
    if constexpr (W == 4) {
#pragma unroll
        for (int k = 0; k < V; ++k) s_acc[warp][lane * V + k] = acc[k];
        if (lane == 0) s_sum[warp] = sum;
        __syncthreads();
        if (warp > 0) return;
#pragma unroll
        for (int k = 0; k < V; ++k)
            acc[k] = (s_acc[0][lane * V + k] + s_acc[1][lane * V + k]) + (s_acc[2][lane * V + k] + s_acc[3][lane * V + k]);
        sum = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
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
inline int attn_ctas_per_sm(int rp) { return rp > 16 ? 1 : 2; }

cudaError_t launch_attention_d64(int rp, const AttnLaunch& a);
cudaError_t launch_attention_d128(int rp, const AttnLaunch& a);

}  // namespace dl
