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
// Both products run as tcgen05.mma kind::f8f6f4 on the codes exactly as they
// lie in the cache, tokens on the TMEM lanes; nothing converts keys or values:
//     S^T [128 tokens x rows] = K [128 x D] . Q^T
//     O^T [D x rows]         += V^T [D x 128] . P^T
// The 16-bit side goes in as sums of 8-bit numbers.  A bf16 query has 8 significant
// bits and is the sum of two e4m3 parts of 4: exact for elements from 2^-9 of the
// row's largest on (each row is scaled to the top of the range), to 2^-17 of it absolute
// below.  P is rounded to fp16 and cut into three e5m2 parts of 16 times each
// other's scale, each in accumulator columns of its own.  A part has 3 significant bits
// and a sign, so three hold fp16's 11 exactly, and with e5m2's range down to its
// smallest number, 2^-24.  The row's largest P is at 2^9 at least: a weight loses no
// more than 11 bits' rounding down to 2^-23 of the largest, 2^-34 of it absolute
// below, so that a tail of many small ones counts beside a token that takes nearly all
// weight.  The maximum may grow by 2^5.8 before n_r has to move.
// (e4m3 parts end at 2^-21 of the largest, three or four of them: 32768 tokens of 2^-22
// were lost, 0.8 % of the weight.  Two e4m3 parts have 18 bits of range for both, and moving
// n_r took most of the time at 128 rows; fp16 products need the values widened in
// shared memory, which then moves twice the bytes and bounds the kernel at 48 rows.)
// Scores, maxima, exponentials, sums and accumulators are fp32.
//
// A CTA runs a contiguous range of 128-token tiles of the whole call (sequence,
// row tile, head, tile), the same number for every CTA to within one: the work
// of a long sequence spreads over the chip, and many short ones pack.  A
// sequence that ends up on several CTAs leaves partial sums in the workspace,
// joined in a fixed order by attention_combine_kernel.
//
// What bounds it, with 64 query heads on 8 heads of 128, and what a call measured
// with the join: up to 16 rows the read of the cache (64 sequences of up to 16384
// tokens, 1.6 GB: 243 to 246 us, 6.6 TB/s, 0.97 of a copy's rate; 32 of up to 4096: 40 us, 5.1 TB/s),
// or, where there is little of it, a chain of latencies (one sequence of 500 tokens
// 7.5 us, of 30011 tokens 18 us).  Beyond, the softmax's instructions, about 610 a
// warp and tile at 64 rows (4 x 32768 tokens, 16 new ones each: 126.7 us, 2.1 TB/s;
// 16 x up to 8192 with 6: 59 us, 3.5 TB/s).
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
    int num_pages, q_heads;
    int kv_heads, head_parts, group;    // key/value heads times parts of their query heads; heads of a part
    int page_size, page_shift, block_shift;
    int tile_tokens, row_tiles;         // new tokens of a row tile, row tiles of max_q
    float scale_log2;                   // scale * log2(e)
    Sequences s;
    float* partial;                     // [grid][2][RP][D] then [grid][2][RP][2]
    struct AttnSplit* split;            // [grid]
    unsigned* err_word;
    unsigned long long wait_limit_ns;
    int withhold;                       // k: CTA 0 never copies its k-th tile's keys (0: none)
};

// A split item, at the index of the CTA that begins it (n = 0: none).
struct AttnSplit {
    int n;                              // CTAs that share it, consecutive
    int slot0;                          // which of the first CTA's two slots it uses
    int row0, rows, head;               // first token row, rows, head (part)
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

// The tiles of the call dealt to `grid` CTAs in runs of equal length, the first
// `more` of them one longer.
struct AttnShare {
    long long each;
    int more;
    __device__ __forceinline__ AttnShare(long long total, int grid) {
        if (total >> 31) {
            each = total / grid;
            more = (int)(total % grid);
        } else {                        // 32-bit division is several times faster
            const unsigned q = (unsigned)total / (unsigned)grid;
            each = q;
            more = (int)((unsigned)total - q * (unsigned)grid);
        }
    }
    __device__ __forceinline__ long long begin(int c) const { return c * each + min(c, more); }
    __device__ __forceinline__ int cta_of(long long tile) const {
        const long long head = more * (each + 1);
        const bool longer = tile < head;
        const long long at = longer ? tile : tile - head, run = longer ? each + 1 : each;
        return (longer ? 0 : more) + ((at | run) >> 31 ? (int)(at / run) : (int)((unsigned)at / (unsigned)run));
    }
};

// RP rows.  A tile's chain of waits and dependent instructions is longer than its
// share of the memory's time, so several tiles are in work on an SM: two CTAs up to
// 16 rows (three with heads of 64, whose tiles are half as long: 32 sequences of
// 4096 tokens, 8 rows, 28.1 -> 26.1 us), beyond that one CTA whose two tile groups
// (TG) take tiles in turn, with accumulators of their own, and share the pipeline's
// slots.  A tile group beyond 32 rows is two warpgroups (CG) of RW rows each: more
// warps to hide one another's latencies (64 rows at 4 x 32768 tokens: 200 -> 159 us
// when it was built).  With heads of 64, 17 to 32 rows are better off as two CTAs of one tile
// group of two warpgroups (64 x 2048 tokens, 32 rows: 63.0 -> 49.6 us; 24 x 2049, 24
// rows: 29.9 -> 24.2), with heads of 128 only where sequences are short (256 x 512: 128
// -> 93 us, but 16 x 8192: 49 -> 58), which the host cannot know; 48 rows as two CTAs of heads
// of 64 gain 2 % there and lose 10 % on one long sequence.
template <int D_, int RP_>
struct AttnShape {
    static constexpr int D = D_, RP = RP_;
    static constexpr int kParts = 3;
    static constexpr int TG = RP > 32 || (RP > 16 && D == 128) ? 2 : 1;
    static constexpr int CG = RP > 32 || (RP > 16 && D == 64) ? 2 : 1;
    static constexpr int RW = RP / CG;
    static constexpr bool kConcat = RP <= 32;           // S columns: hi parts, then lo parts (else summed by the MMA)
    static constexpr int kScoreCols = kConcat ? 2 * RP : RP;
    static constexpr int kOutCol = 2 * kScoreCols;
    static constexpr int kOutCols = (kParts * RP + 15) / 16 * 16;    // P's columns come in chunks of 16
    static constexpr int kCols = kOutCol + TG * kOutCols;
    static constexpr int kTmem = kCols <= 32 ? 32 : kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
    static constexpr int kCtas = TG == 2 ? 1 : D == 64 && RP <= 16 ? 3 : 2;      // resident CTAs per SM
    static constexpr int kThreads = TG * CG * 128 + 96;
    static constexpr int kTileBytes = kTile * D;        // codes of K, and of V
    static constexpr int kQBytes = 2 * RP * D;
    static constexpr int kPBytes = kOutCols * kTile;    // one of two buffers
    // segment descriptors: one more than tiles can be in flight, and the one in work
    static constexpr int kSegments = 10;
    static constexpr int kMisc = 1024 + kSegments * 36 + 8 + RP * 32 * TG + TG * 4 * RP * 4 + TG * D * 4 + 256;
    static constexpr int kBudget = (kCtas == 1 ? 227 : kCtas == 2 ? 113 : 75) * 1024;
    // a tile's slots: its codes, and 8 bytes of scales for each token
    static constexpr int kScaleBytes = kTile * 8;
    static constexpr int kRoom = kBudget - 1024 - kQBytes - 2 * kPBytes - kMisc;
    static constexpr int kFit = kRoom / (2 * kTileBytes + kScaleBytes);
    static constexpr int kKeySlots = kFit > 6 ? 6 : kFit;
    static constexpr int kValueSlots = kKeySlots + (kRoom - kKeySlots * (2 * kTileBytes + kScaleBytes) >= kTileBytes + kScaleBytes);
    static constexpr size_t kSmem = 1024 + (size_t)kKeySlots * kTileBytes + (size_t)kValueSlots * (kTileBytes + kScaleBytes) +
                                    kQBytes + 2 * kPBytes + kMisc;
    static_assert(kValueSlots + 2 <= kSegments && kKeySlots >= 2 && kCols <= 512 && kCols * kCtas <= 512 && kOutCols <= 256, "fits an SM");
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

// Instruction descriptors of kind::f8f6f4 -> fp32, M x N, A in e4m3: B in e4m3, both
// operands with their K dimension contiguous in memory; and B in e5m2, M and N contiguous.
__host__ __device__ constexpr uint32_t umma_idesc_k(int m, int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__host__ __device__ constexpr uint32_t umma_idesc_mn_e5m2(int m, int n) {
    return umma_idesc_k(m, n) | (1u << 10) | (3u << 15);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
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
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
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

// Four probabilities -> their e5m2 parts, each the rest of the one before times 16.
// The fp16 step in between rounds to 2^-11, and is all that is lost of numbers below 2^15.
template <int N>
__device__ __forceinline__ void split_e5m2(float e0, float e1, float e2, float e3, uint32_t (&part)[N]) {
    constexpr uint32_t kSixteen = 0x4C004C00u;          // f16x2
    uint32_t x = f32x2_to_f16x2(e0, e1), y = f32x2_to_f16x2(e2, e3);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        if (i + 1 < N) {
            uint32_t u, v;
            asm("{\n\t"
                ".reg .b16 a, b;\n\t"
                "cvt.rn.satfinite.e5m2x2.f16x2 a, %3;\n\t"
                "cvt.rn.satfinite.e5m2x2.f16x2 b, %4;\n\t"
                "cvt.rn.f16x2.e5m2x2 %1, a;\n\t"
                "cvt.rn.f16x2.e5m2x2 %2, b;\n\t"
                "mov.b32 %0, {a, b};\n\t"
                "}"
                : "=r"(part[i]), "=r"(u), "=r"(v) : "r"(x), "r"(y));
            asm("{\n\t"
                "sub.rn.f16x2 %0, %0, %2;\n\t"
                "sub.rn.f16x2 %1, %1, %3;\n\t"
                "mul.rn.f16x2 %0, %0, %4;\n\t"
                "mul.rn.f16x2 %1, %1, %4;\n\t"
                "}"
                : "+r"(x), "+r"(y) : "r"(u), "r"(v), "r"(kSixteen));
        } else {
            asm("{\n\t"
                ".reg .b16 a, b;\n\t"
                "cvt.rn.satfinite.e5m2x2.f16x2 a, %1;\n\t"
                "cvt.rn.satfinite.e5m2x2.f16x2 b, %2;\n\t"
                "mov.b32 %0, {a, b};\n\t"
                "}"
                : "=r"(part[i]) : "r"(x), "r"(y));
        }
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

// A ring's slot and the parity of its current round.
template <int N>
struct Ring {
    int slot = 0;
    uint32_t round = 0;
    __device__ __forceinline__ void step(int n = 1) {
        slot += n;
        if (slot >= N) {
            slot -= N;
            round ^= 1;
        }
    }
};

__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}

// Waits of one CTA: bounded, and short once any of them has given up.
struct CtaWait {
    WaitCtl ctl;
    volatile int* stop;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t parity, unsigned bit) const {
        // a test answers in a third of the time of a wait that may suspend
        return after(mbar_test(bar, parity), bar, parity, bit);
    }
    // `done`: what a test made before has said
    __device__ __forceinline__ bool after(bool done, uint32_t bar, uint32_t parity, unsigned bit) const {
        if (__builtin_expect(done, 1)) return true;
        if (*stop) return false;
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
    __device__ __forceinline__ void start(const AttnEntry& entry_, long long at_, long long end_, int e_, int within) {
        at = at_;
        end = end_;
        e = e_;
        entry = entry_;
        head = (int)((unsigned)within / (unsigned)entry.tiles);
        tile0 = (int)within - head * entry.tiles;
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

// What the softmax needs of a segment, made by the warp that walks ahead.
struct __align__(16) AttnSegment {
    int row0, rows, seen0, head;        // first token row, rows, cached tokens the first sees, head (part)
    int tile0, tiles;
    int whole, last;                    // a whole item; the CTA's last segment
};

// The scales of a token's blocks; value < 0: the token is absent.
struct __align__(8) TokenScales {
    float key, value;
};

// After a wait that gave up: no copy and no product of the CTA may still be in flight when it
// leaves.  One limit for all copies, which have been under way together.
template <int NK, int NV>
__device__ __forceinline__ void attn_drain_copies(uint32_t k_full, uint32_t v_full, int keys, int values, WaitCtl ctl) {
    bool landed = true;
    for (int i = max(keys - NK, 0); i < keys && landed; ++i)
        landed = mbar_wait_bounded(k_full + 8 * (i % NK), (i / NK) & 1, ctl, kErrDrainWait);
    for (int i = max(values - NV, 0); i < values && landed; ++i)
        landed = mbar_wait_bounded(v_full + 8 * (i % NV), (i / NV) & 1, ctl, kErrDrainWait);
}
// By the warp that issued them.
__device__ __forceinline__ void attn_drain_products(uint32_t all_done, WaitCtl ctl) {
    if (elect_one()) umma_commit(all_done);
    __syncwarp();
    mbar_wait_bounded(all_done, 0, ctl, kErrDrainWait);
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kCtas)
attention_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const __grid_constant__ AttnParams p) {
    constexpr int D = C::D, RP = C::RP, RW = C::RW, TG = C::TG, CG = C::CG, NWG = TG * CG;
    constexpr int NK = C::kKeySlots, NV = C::kValueSlots, NS = C::kSegments;
    constexpr int kProducer = NWG * 4, kMma = NWG * 4 + 1, kScaler = NWG * 4 + 2;
    constexpr int kAllBar = NWG + 1, kSoftmax = NWG * 128;
    // one accumulator lane per dim: M = 64 leaves 16 rows in each warp's lanes
    constexpr int kDimLanes = D / 4;
    constexpr uint32_t kSwizzle = D == 128 ? 2 : 4;
    // largest exponent of a probability (its parts hold numbers below 2^15), and the one a maximum
    // gets: the rest is its room to grow.  (A maximum at 2^5, with 2^9.8 to grow: the same times up to
    // 16 rows, 125.7 -> 124.8 us at 4 x 32768 tokens with 16 new ones; small weights would end at 2^-30.)
    constexpr float kTop = 14.8f, kTarget = 9.f;
    // rows that a softmax thread works on at a time, and columns of a load: as registers allow
    constexpr int kHalf = RW > 24 && C::CG == 2 ? RW / 2 : RW, kStep = kHalf % 16 ? 8 : 16;
    constexpr float kTinyScale = 8.67361737988403547e-19f;       // 2^-60

    extern __shared__ unsigned char smem_raw[];
    // (an offset, not a rounded pointer: the compiler keeps seeing shared memory)
    unsigned char* base = smem_raw + (-smem_u32(smem_raw) & 1023);
    unsigned char* sp = base;                                     // [2] P [columns / 16][128 tokens][16]
    unsigned char* sq = sp + 2 * C::kPBytes;                      // query parts [2][RP][D]
    unsigned char* keys = sq + C::kQBytes;                        // codes, [128 tokens][D] each
    unsigned char* values = keys + NK * C::kTileBytes;
    TokenScales* scales = reinterpret_cast<TokenScales*>(values + NV * C::kTileBytes);   // [NV][128]
    unsigned char* misc = reinterpret_cast<unsigned char*>(scales + NV * kTile);
    uint64_t* bars = reinterpret_cast<uint64_t*>(misc);
    uint64_t *k_full = bars, *k_empty = k_full + NK, *v_full = k_empty + NK, *v_empty = v_full + NV,
             *s_full = v_empty + NV, *s_read = s_full + 2, *p_full = s_read + 2, *pv_done = p_full + 2, *q_full = pv_done + 2,
             *seg_full = q_full + 1, *all_done = seg_full + NS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(all_done + 1);
    int* s_stop = reinterpret_cast<int*>(tmem_slot + 1);
    long long* s_walk = reinterpret_cast<long long*>(misc + 512);     // total, begin, end
    int* s_start = reinterpret_cast<int*>(misc + 536);                // first entry, tiles of it before `begin`
    AttnEntry* s_entry = reinterpret_cast<AttnEntry*>(misc + 544);
    int* s_copied = reinterpret_cast<int*>(misc + 592);               // tiles whose keys, and whose values, were copied
    volatile int* s_quit = s_copied + 2;                              // a softmax thread has waited for a segment in vain
    int* s_flags = reinterpret_cast<int*>(misc + 640);                // [NV] some token is absent, or its scale tiny
    AttnSegment* s_seg = reinterpret_cast<AttnSegment*>(misc + 1024); // [NS]
    int* s_share = reinterpret_cast<int*>(s_seg + NS);                // [NS] CTAs that share an item begun here, or 0
    // [TG] of what belongs to a segment's rows: with two tile groups the next one's is made early
    float* s_qs = reinterpret_cast<float*>(s_share + (NS + 3) / 4 * 4);   // [TG][RP] a row's query scale
    int* s_lim = reinterpret_cast<int*>(s_qs + TG * RP);              // [TG][RP] cached tokens a row sees
    long long* s_out = reinterpret_cast<long long*>(s_lim + TG * RP); // [TG][RP] where a row's output begins
    float* s_n = reinterpret_cast<float*>(s_out + TG * RP);           // [TG][RP] n_r
    float* s_l = s_n + TG * RP;                                       // [TG][RP] sums of P / vs
    float* s_f = s_l + TG * RP;                                       // [TG][RP] factors of the accumulators
    float* s_red = s_f + TG * RP;                                     // [NWG][4][RW]
    int* s_nan = reinterpret_cast<int*>(s_red + TG * 4 * RP);         // [TG][D] first NaN among the new tokens' values

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
                mbar_init(smem_u32(v_empty + i), 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(smem_u32(s_full + i), 1);
                mbar_init(smem_u32(s_read + i), CG * 4);
                mbar_init(smem_u32(p_full + i), CG * 4);
                mbar_init(smem_u32(pv_done + i), 1);
            }
            mbar_init(smem_u32(q_full), CG * 4);
            for (int i = 0; i < NS; ++i) mbar_init(smem_u32(seg_full + i), 1);
            mbar_init(smem_u32(all_done), 1);
            *s_stop = 0;
            s_copied[0] = s_copied[1] = *s_quit = 0;
            for (int i = 0; i < NS; ++i) s_share[i] = 0;       // may be read before it is written, after a wait that gave up
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
        // the CTA's tiles, and the entry in which they begin: entries 32 at a time
        const int entries = p.s.batch * p.row_tiles;
        AttnEntry held;
        held.tiles = 0;
        if (lane < entries) held = attn_entry(p, lane);
        long long total = 0, begin = 0, end = 0;
        int grid = gridDim.x;
        bool found = false;
        auto hit = [&](const AttnEntry& en, int e, long long before) {
            s_start[0] = e;
            s_start[1] = (int)(begin - before);
            *s_entry = en;
        };
        if (entries <= 32 && __all_sync(~0u, held.tiles < (1 << 25) / p.kv_heads)) {
            // one round, in 32 bits
            const int mine = held.tiles * p.kv_heads;
            int inc = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(~0u, inc, o);
                if (lane >= o) inc += y;
            }
            total = __shfl_sync(~0u, inc, 31);
            grid = min(grid, (int)total);
            if ((int)blockIdx.x < grid) {
                const AttnShare share(total, grid);
                begin = share.begin(blockIdx.x);
                end = share.begin(blockIdx.x + 1);
                found = true;
                if (inc > begin && inc - mine <= begin) hit(held, lane, inc - mine);
            }
        } else {
            total = held.tiles;
            for (int e = 32 + lane; e < entries; e += 32) total += attn_entry(p, e).tiles;
            for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(~0u, total, o);
            total *= p.kv_heads;
            if (total < grid) grid = (int)total;
            if ((int)blockIdx.x < grid) {
                const AttnShare share(total, grid);
                begin = share.begin(blockIdx.x);
                end = share.begin(blockIdx.x + 1);
                long long run = 0;
#pragma unroll 1
                for (int e0 = 0; e0 < entries && !found; e0 += 32) {
                    AttnEntry en = held;
                    if (e0 > 0) {
                        en.tiles = 0;
                        if (e0 + lane < entries) en = attn_entry(p, e0 + lane);
                    }
                    const long long mine = (long long)en.tiles * p.kv_heads;
                    long long inc = mine;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const long long y = __shfl_up_sync(~0u, inc, o);
                        if (lane >= o) inc += y;
                    }
                    const unsigned which = __ballot_sync(~0u, run + inc > begin);
                    if (which) {
                        found = true;
                        if (lane == __ffs(which) - 1) hit(en, e0 + lane, run + inc - mine);
                    }
                    run += __shfl_sync(~0u, inc, 31);
                }
            }
        }
        if (lane == 0) {
            s_walk[0] = total;
            s_walk[1] = begin;
            s_walk[2] = found ? end : begin;
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
    if (work) w.start(*s_entry, s_walk[1], s_walk[2], s_start[0], s_start[1]);

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
                if (page >= 0 && !is_v && !(it + 1 == p.withhold && blockIdx.x == 0))
                    tma_load_4d(smem_u32(keys + ks * C::kTileBytes + sub * box * D), &tk, smem_u32(k_full + ks), 0, at,
                                w.head / p.head_parts, page);
                if (it >= NV) ok = __all_sync(~0u, wait(smem_u32(v_empty + vs), (it / NV - 1) & 1, kErrProducerWait));
                if (!ok) {
                    if (lane == 0) s_copied[0] = 1;             // the keys of one tile more
                    break;
                }
                if (lane == 16) mbar_arrive_expect_tx(smem_u32(v_full + vs), bytes);
                __syncwarp();
                if (page >= 0 && is_v)
                    tma_load_4d(smem_u32(values + vs * C::kTileBytes + sub * box * D), &tv, smem_u32(v_full + vs), 0, at,
                                w.head / p.head_parts, page);
                page = next;
            }
        } while (ok && w.next(p));
        if (lane == 0) {
            s_copied[0] += it;
            s_copied[1] = it;
        }
    } else if (work && warp == kScaler) {
        // ------------------------------------------------ scales: four tokens each lane; a tile's
        // pages are read two tiles ahead, its scales one.  And what the softmax needs of a segment: a
        // descriptor's slot comes round again after more segments than tiles can be in flight.
        int it = 0, seg = 0;
        bool ok = true;
        do {
            if (lane == 0) {
                s_seg[seg % NS] = AttnSegment{w.entry.row0, w.entry.tokens * p.group, w.entry.seen0, w.head, w.tile0,
                                              w.tile1 - w.tile0, w.whole(), w.at + (w.tile1 - w.tile0) >= w.end};
                mbar_arrive(smem_u32(seg_full + seg % NS));
            }
            __syncwarp();
            const int* table = p.s.block_table + (size_t)w.entry.b * p.s.table_cols;
            const int head = w.head / p.head_parts;
            // four consecutive tokens are on one page, and share a block of four or more
            auto page_of = [&](int tile) {
                const int j = tile * kTile + 4 * lane;
                return tile < w.tile1 && j < w.entry.seen_last ? table[j >> p.page_shift] : -1;
            };
            auto load = [&](int tile, int pg, float (&a)[4], float (&b)[4]) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    a[k] = 0.f;
                    b[k] = -1.f;
                }
                if ((unsigned)pg >= (unsigned)p.num_pages) return;
                const int j = tile * kTile + 4 * lane, t = j & (p.page_size - 1);
                const long long o = pg * p.scale_page_stride + head * p.scale_head_stride + (t >> p.block_shift);
                a[0] = p.k_scale[o];
                b[0] = p.v_scale[o];
#pragma unroll
                for (int k = 1; k < 4; ++k) {
                    const int more = k >> p.block_shift;
                    a[k] = more ? p.k_scale[o + more] : a[0];
                    b[k] = more ? p.v_scale[o + more] : b[0];
                    if (j + k >= w.entry.seen_last) b[k] = -1.f;
                }
            };
            float a[4], b[4];
            int next = page_of(w.tile0);
            load(w.tile0, next, a, b);
            next = page_of(w.tile0 + 1);
            if (lane == 0) {
                // read after the segment's last tile, so nobody waits for the divisions
                int share = 0;
                if (w.tile0 == 0 && !w.whole()) {
                    const AttnShare dealt(total, total < gridDim.x ? (int)total : (int)gridDim.x);
                    share = dealt.cta_of(w.item_begin + w.entry.tiles - 1) - (int)blockIdx.x + 1;
                }
                s_share[seg % NS] = share;
            }
            ++seg;
            for (int tile = w.tile0; tile < w.tile1; ++tile, ++it) {
                float a1[4], b1[4];
                load(tile + 1, next, a1, b1);
                next = page_of(tile + 2);
                const int s = it % NV;
                if (it >= NV) ok = __all_sync(~0u, wait(smem_u32(v_empty + s), (it / NV - 1) & 1, kErrProducerWait));
                if (!ok) break;
                int flags = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) flags |= b[k] < kTinyScale;         // -1 where absent
                float4* to = reinterpret_cast<float4*>(scales + s * kTile + 4 * lane);
                to[0] = make_float4(a[0], b[0], a[1], b[1]);
                to[1] = make_float4(a[2], b[2], a[3], b[3]);
                flags = __reduce_or_sync(~0u, flags);
                if (lane == 0) s_flags[s] = flags;
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(v_full + s));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    a[k] = a1[k];
                    b[k] = b1[k];
                }
            }
        } while (ok && w.next(p));
    } else if (work && warp == kMma) {
        // ------------------------------------------------ products: the warp waits, one lane issues
        constexpr uint32_t kScoreIdesc = umma_idesc_k(128, C::kScoreCols);
        constexpr uint32_t kOutIdesc = umma_idesc_mn_e5m2(D, C::kOutCols);
        const bool leader = elect_one();
        const uint64_t q_desc = umma_desc(smem_u32(sq), 16, 8 * D, kSwizzle);
        const uint64_t k_desc = umma_desc(smem_u32(keys), 16, 8 * D, kSwizzle);
        const uint64_t v_desc = umma_desc(smem_u32(values), 16, 8 * D, kSwizzle);
        const uint64_t p_desc = umma_desc(smem_u32(sp), 128, kTile * 16, 0);
        int it = 0, seg = 0;
        bool ok = true;
        Ring<NK> kr;
        Ring<NV> vr;
        auto scores = [&](int i) {
            if (!__all_sync(~0u, wait(smem_u32(k_full + kr.slot), kr.round, kErrConsumerWait))) return false;
            tc_fence_after_sync();
            const uint64_t a = k_desc + (uint32_t)(kr.slot * C::kTileBytes >> 4);
            const uint32_t d = tmem + (i & 1) * C::kScoreCols;
            if (leader) {
#pragma unroll
                for (int part = 0; part < (C::kConcat ? 1 : 2); ++part)
#pragma unroll
                    for (int k = 0; k < D / 32; ++k)
                        umma_e4m3(d, a + 2 * k, q_desc + (part * RP * D >> 4) + 2 * k, kScoreIdesc, part > 0 || k > 0);
                umma_commit(smem_u32(s_full + (i & 1)));
                umma_commit(smem_u32(k_empty + kr.slot));
            }
            __syncwarp();
            kr.step();
            return true;
        };
        // the scores of tile i are read: their buffer is free
        auto read = [&](int i) {
            return i < 0 || __all_sync(~0u, wait(smem_u32(s_read + (i & 1)), (i >> 1) & 1, kErrConsumerWait));
        };
        do {
            // scores run two tiles ahead: as soon as those of the tile before in their buffer are read
            ok = __all_sync(~0u, wait(smem_u32(q_full), seg & 1, kErrConsumerWait)) && read(it - 2) && scores(it) &&
                 (w.tile0 + 1 >= w.tile1 || (read(it - 1) && scores(it + 1)));
            for (int tile = w.tile0; tile < w.tile1 && ok; ++tile, ++it) {
                if (tile + 2 < w.tile1 && !(ok = read(it) && scores(it + 2))) break;
                if (!(ok = __all_sync(~0u, wait(smem_u32(p_full + (it & 1)), (it >> 1) & 1, kErrConsumerWait)))) break;
                tc_fence_after_sync();
                const uint64_t a = v_desc + (uint32_t)(vr.slot * C::kTileBytes >> 4);
                const uint64_t b = p_desc + (uint32_t)((it & 1) * C::kPBytes >> 4);
                const uint32_t o = tmem + C::kOutCol + (TG == 2 ? (it & 1) * C::kOutCols : 0);
                const uint32_t more = tile - w.tile0 >= TG;      // this accumulator holds something
                if (leader) {
#pragma unroll
                    for (int k = 0; k < kTile / 32; ++k)
                        umma_e4m3(o, a + k * (32 * D >> 4), b + k * 32, kOutIdesc, k > 0 ? 1u : more);
                    umma_commit(smem_u32(pv_done + (it & 1)));
                    umma_commit(smem_u32(v_empty + vr.slot));
                }
                __syncwarp();
                vr.step();
            }
            ++seg;
        } while (ok && w.next(p));
    } else if (work && warp < kProducer) {
        // ------------------------------------------------ softmax: a token each thread
        // (a wait that gives up is not left by: the others of the group are at its barriers.  All leave together
        // at a segment's end, once one of them has waited for the next one's descriptor in vain: s_quit is
        // written before and read after a barrier of all)
        const int wg = warp >> 2, wq = warp & 3, tl = tid & 127, bar_id = 1 + wg;
        const int tg = wg / CG, r0 = wg % CG * RW;          // tile group, first row
        const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
        const uint32_t out_at = lanes + C::kOutCol + tg * C::kOutCols + r0;
        float* red = s_red + wg * 4 * RW;
        float* my_n = s_n + tg * RP + r0;
        int it0 = 0;                                        // the segment's first tile, counted by the CTA
        Ring<NV> vr;                                        // its slot of values and scales
        int slot = 0;
        auto pv_wait = [&](int i) {         // the product of tile i has been made
            if (i >= 0) wait(smem_u32(pv_done + (i & 1)), (i >> 1) & 1, kErrConsumerWait);
        };
        // a segment's queries: 16 elements each thread, read before the segment before it is finished
        constexpr int TPR = D / 16;                         // threads of a row
        static_assert(RP * TPR <= kSoftmax, "16 dims each thread");
        // a thread's 16 dims of a row of a segment's queries
        auto load_query = [&](const AttnSegment& sg, int t, uint4 (&v)[2]) {
            const int row = t / TPR, token = row / p.group;
            v[0] = v[1] = make_uint4(0, 0, 0, 0);
            if (row < sg.rows) {
                const uint16_t* src = p.q + (size_t)(sg.row0 + token) * p.q_stride +
                                      (size_t)(sg.head * p.group + row - token * p.group) * D + t % TPR * 16;
                v[0] = ldg128(src);
                v[1] = ldg128(src + 8);
            }
        };
        // ... as two e4m3 parts, each row scaled to the top of the range; `buf`: where the segment's rows are noted
        auto store_query = [&](const AttnSegment& sg, int buf, int t, const uint4 (&v)[2]) {
            const int c = t % TPR, row = t / TPR;
            const uint32_t x[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
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
                s_qs[buf * RP + row] = row < sg.rows ? (odd ? __uint_as_float(0x7fffffffu) : down * p.scale_log2) : 0.f;
                const int token = row / p.group;
                s_lim[buf * RP + row] = row < sg.rows ? max(sg.seen0 + token, 0) : 0;
                s_out[buf * RP + row] =
                    ((long long)(sg.row0 + token) * p.q_heads + sg.head * p.group + row - token * p.group) * D;
            }
        };
        uint4 query[2];
        // this segment's descriptor is there: the scales' warp writes no more once it has given up, and those
        // in the ring are then old ones
        bool ready = __all_sync(~0u, wait(smem_u32(seg_full), 0, kErrConsumerWait));
        if (!ready) *s_quit = 1;
        if (ready && tid < RP * TPR) load_query(s_seg[0], tid, query);
        int seg = 0;
        bool last = false;
        do {
            const AttnSegment* sg = s_seg + seg % NS;
            const int tile_first = sg->tile0, tiles = sg->tiles, seen0 = sg->seen0, seen_first = max(seen0, 0);
            const int buf = TG == 2 ? seg & 1 : 0;
            const float* my_qs = s_qs + buf * RP + r0;

            // the accumulators and the rows' notes of the segment before have been read
            if (tl < RW) my_n[tl] = 0.f;
            tc_fence_before_sync();
            group_sync(kAllBar, kSoftmax);
            if (TG == 1 || seg == 0) {
                if (tid < RP * TPR) store_query(*sg, 0, tid, query);
                if (tid < D) s_nan[tid] = 0x7fffffff;
                fence_proxy_async_smem();
                group_sync(kAllBar, kSoftmax);
                if (tg == 0 && lane == 0) mbar_arrive(smem_u32(q_full));
                if (seg == 0 && *s_quit) break;
            }

            F2 l[RW / 2];
#pragma unroll
            for (int r = 0; r < RW / 2; ++r) l[r] = 0;
            uint32_t unset = ~0u;            // threads below RW: this row has no n_r yet
            const int t_first = TG == 2 ? (it0 + tg) & 1 : 0;       // the group's tiles have its parity
            Ring<NV> vt = vr;
            if (t_first) vt.step();
            bool force = true;               // some row has no n_r yet
            for (int t = t_first; t < tiles; t += TG) {
                const int it = it0 + t, tile = tile_first + t, j = tile * kTile + tl;
                // tests together, so that their answers' times overlap
                const bool v_ok = mbar_test(smem_u32(v_full + vt.slot), vt.round);
                const bool s_ok = mbar_test(smem_u32(s_full + (it & 1)), (it >> 1) & 1);
                wait.after(v_ok, smem_u32(v_full + vt.slot), vt.round, kErrConsumerWait);
                const TokenScales ts = scales[vt.slot * kTile + tl];
                const int flags = s_flags[vt.slot];
                const bool absent = ts.value < 0.f;
                // a scale below the smallest that counts is a zero: the token weighs, its values do not.  Its P is
                // that of the smallest scale, so that n_r is placed by tokens whose values count (were its
                // scale taken as 1, scales of 2^-18 would be left with three bits beside it, of 2^-22 with none)
                const bool empty = absent || ts.value < kTinyScale;
                const float value = absent ? 1.f : empty ? kTinyScale : ts.value;
                const float lv = log2_fast(value), inv = rcp_fast(value);
                const bool masked = (tile + 1) * kTile > seen_first || flags;

                wait.after(s_ok, smem_u32(s_full + (it & 1)), (it >> 1) & 1, kErrConsumerWait);
                tc_fence_after_sync();
                // values that do not count are taken out: all of an absent token, those of a zero scale that
                // are not NaN, and NaN codes of the new tokens (0 x NaN would reach every row), which are noted by dim
                if (__builtin_expect(masked && (empty || j >= seen_first), 0)) {
                    unsigned char* codes = values + vt.slot * C::kTileBytes + tl * D;
#pragma unroll 1
                    for (int c = wg % CG; c < D / 16; c += CG) {
                        uint4* at = reinterpret_cast<uint4*>(codes + c * 16);
                        if (absent) {
                            *at = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        uint4 x = *at;
                        uint32_t* word = &x.x;
                        uint32_t any = 0;
#pragma unroll
                        for (int k = 0; k < 4; ++k) any |= (word[k] & 0x7f7f7f7fu) + 0x01010101u;
                        if (!(any & 0x80808080u)) {
                            if (empty) *at = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        const int dims = (D == 128 ? (c ^ (tl & 7)) : (c ^ ((tl >> 1) & 3))) * 16;
#pragma unroll 1
                        for (int k = 0; k < 16; ++k) {
                            unsigned char* byte = codes + c * 16 + k;
                            const bool nan = (*byte & 0x7f) == 0x7f;
                            if (nan && j >= seen_first) atomicMin(s_nan + buf * D + dims + k, j);
                            if (nan ? j >= seen_first : empty) *byte = 0;
                        }
                    }
                }

                const uint32_t sc = lanes + (it & 1) * C::kScoreCols + r0;
                const F2 ks2 = f2(ts.key, ts.key), lv2 = f2(lv, lv), inv2 = f2(inv, inv);
                unsigned char* dst = sp + (it & 1) * C::kPBytes + tl * 16;
                // new token i, rows i * group on, sees cache indexes below seen0 + i: rows before `from` do not see this one
                const int from = absent ? RP : max(min(j - seen0 + 1, RP), 0) * p.group - r0;
                bool still = false;
#pragma unroll
                for (int h = 0; h < RW; h += kHalf) {
                    // exponents t + n of kHalf rows
                    float d[kHalf];
                    {
                        float lo[kHalf];
#pragma unroll
                        for (int r = 0; r < kHalf; r += kStep) {
                            tmem_ld<kStep>(sc + h + r, d + r);
                            if (C::kConcat) tmem_ld<kStep>(sc + RP + h + r, lo + r);
                        }
                        tmem_wait_ld();
                        if (h + kHalf == RW) {
                            tc_fence_before_sync();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(smem_u32(s_read + (it & 1)));
                        }
#pragma unroll
                        for (int r = 0; r < kHalf; r += 4) {
                            F2 q0, q1, n0, n1, x0 = f2(d[r], d[r + 1]), x1 = f2(d[r + 2], d[r + 3]);
                            lds_f2x2(my_qs + h + r, q0, q1);
                            lds_f2x2(my_n + h + r, n0, n1);
                            if (C::kConcat) {
                                x0 = add2(x0, f2(lo[r], lo[r + 1]));
                                x1 = add2(x1, f2(lo[r + 2], lo[r + 3]));
                            }
                            unpack(add2(fma2(mul2(x0, q0), ks2, lv2), n0), d[r], d[r + 1]);
                            unpack(add2(fma2(mul2(x1, q1), ks2, lv2), n1), d[r + 2], d[r + 3]);
                        }
                    }
                    if (masked) {
#pragma unroll
                        for (int r = 0; r < kHalf; ++r)
                            if (h + r < from) d[r] = -INFINITY;
                    }
                    float top = -INFINITY;
#pragma unroll
                    for (int r = 0; r < kHalf; r += 2) top = max3(top, d[r], d[r + 1]);
                    // the buffer that P goes to: asked for ahead of the vote, which takes longer
                    const bool pv_ok = h > 0 || it < 2 || mbar_test(smem_u32(pv_done + (it & 1)), ((it >> 1) - 1) & 1);
                    // a row passes the top, or has no n_r yet: its n_r moves, and its sums follow
                    if (__builtin_expect(group_any(bar_id, 128, top > kTop || force), 0)) {
                        float m0 = 0.f;
#pragma unroll
                        for (int r = 0; r < kHalf; ++r) {
                            const float m = warp_max_f32(d[r]);
                            if (lane == r) m0 = m;
                        }
                        if (lane < kHalf) red[wq * kHalf + lane] = m0;
                        group_sync(bar_id, 128);
                        float move = 0.f;
                        const uint32_t bit = 1u << (h / kHalf);
                        if (tl < kHalf) {
                            const float m = fmaxf(fmaxf(red[tl], red[kHalf + tl]), fmaxf(red[2 * kHalf + tl], red[3 * kHalf + tl]));
                            if (m > -INFINITY && (m > kTop || (unset & bit))) {
                                move = kTarget - m;
                                my_n[h + tl] += move;
                                unset &= ~bit;
                            }
                        }
                        const bool more = group_any(bar_id, 128, tl < kHalf && (unset & bit) && r0 + h + tl < sg->rows);
                        still |= more;
                        if (tl < kHalf) red[tl] = move;
                        group_sync(bar_id, 128);
#pragma unroll
                        for (int r = 0; r < kHalf; r += 4) {
                            const float4 x = *reinterpret_cast<const float4*>(red + r);
                            d[r] = min_nan(d[r] + x.x, kTop);
                            d[r + 1] = min_nan(d[r + 1] + x.y, kTop);
                            d[r + 2] = min_nan(d[r + 2] + x.z, kTop);
                            d[r + 3] = min_nan(d[r + 3] + x.w, kTop);
                            l[(h + r) / 2] = mul2(l[(h + r) / 2], f2(shrink(x.x), shrink(x.y)));
                            l[(h + r) / 2 + 1] = mul2(l[(h + r) / 2 + 1], f2(shrink(x.z), shrink(x.w)));
                        }
                        if (t >= TG) {
                            pv_wait(it - TG);
                            tc_fence_after_sync();
#pragma unroll 1
                            for (int r = 0; r < kHalf; r += 8) {
                                float f[8], o[8];
                                bool same = true;
#pragma unroll
                                for (int k = 0; k < 8; ++k) {
                                    f[k] = red[r + k];
                                    same &= f[k] == 0.f;
                                }
                                if (same) continue;
#pragma unroll 1
                                for (int part = 0; part < C::kParts; ++part) {
                                    tmem_ld<8>(out_at + part * RP + h + r, o);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int k = 0; k < 8; ++k) o[k] *= shrink(f[k]);
                                    tmem_st8(out_at + part * RP + h + r, o);
                                }
                            }
                            tmem_wait_st();
                        }
                        group_sync(bar_id, 128);         // red has been read
                    }

                    // probabilities, cut into parts: columns of part i, then row, 16 to a chunk of 2 KB
                    if (h == 0) wait.after(pv_ok, smem_u32(pv_done + (it & 1)), ((it >> 1) - 1) & 1, kErrConsumerWait);
#pragma unroll
                    for (int r = 0; r < kHalf; r += kStep) {
                        uint32_t part[kStep / 4][C::kParts];
#pragma unroll
                        for (int k = 0; k < kStep; k += 4) {
                            float e[4];
#pragma unroll
                            for (int m = 0; m < 4; ++m) e[m] = exp2_fast(d[r + k + m]);
                            const int at = (h + r + k) / 2;
                            l[at] = fma2(f2(e[0], e[1]), inv2, l[at]);
                            l[at + 1] = fma2(f2(e[2], e[3]), inv2, l[at + 1]);
                            split_e5m2<C::kParts>(e[0], e[1], e[2], e[3], part[k / 4]);
                        }
                        if constexpr (RP == 8) {
                            sts128(smem_u32(dst), part[0][0], part[1][0], part[0][1], part[1][1]);
                            sts128(smem_u32(dst + kTile * 16), part[0][2], part[1][2], 0, 0);   // columns that fill the chunk
                        } else {
#pragma unroll
                            for (int i = 0; i < C::kParts; ++i) {
                                const int col = i * RP + r0 + h + r;
                                unsigned char* to = dst + col / 16 * (kTile * 16);
                                if constexpr (kStep == 16)
                                    sts128(smem_u32(to), part[0][i], part[1][i], part[2][i], part[3][i]);
                                else
                                    *reinterpret_cast<uint2*>(to + col % 16) = make_uint2(part[0][i], part[1][i]);
                            }
                        }
                    }
                }
                fence_proxy_async_smem();
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(p_full + (it & 1)));
                if (force) force = still;
                vt.step(TG);
            }

            // with one tile group the next segment's queries are on their way while this one's sums are made
            const int rows = sg->rows;
            const bool whole = sg->whole;
            last = sg->last;
            if (!last) {
                ready = __all_sync(~0u, wait(smem_u32(seg_full + (seg + 1) % NS), ((seg + 1) / NS) & 1, kErrConsumerWait));
                if (!ready) *s_quit = 1;
                if (TG == 1 && ready && tid < RP * TPR) load_query(s_seg[(seg + 1) % NS], tid, query);
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
            if (tl < RW) s_l[tg * RP + r0 + tl] = (red[tl] + red[RW + tl]) + (red[2 * RW + tl] + red[3 * RW + tl]);
            it0 += tiles;
            // with two, the one that is ready first makes them while the other takes the last tile: the
            // next scores are then there when that one is done (the last scores of this segment
            // are what read these queries last)
            if (TG == 2 && !last && ready && tg != ((it0 - 1) & 1)) {
                wait(smem_u32(s_full + ((it0 - 1) & 1)), ((it0 - 1) >> 1) & 1, kErrConsumerWait);
                const AttnSegment& after = s_seg[(seg + 1) % NS];
                const int t0 = (wg % CG) * 128 + tl;
                constexpr int kGroupThreads = CG * 128;
#pragma unroll 1
                for (int t = t0; t < RP * TPR; t += kGroupThreads) {
                    uint4 v[2];
                    load_query(after, t, v);
                    store_query(after, buf ^ 1, t, v);
                }
                for (int d = t0; d < D; d += kGroupThreads) s_nan[(buf ^ 1) * D + d] = 0x7fffffff;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(q_full));
            }
            {
                const int rounds = (vr.slot + tiles) / NV;
                vr.slot += tiles - rounds * NV;
                vr.round ^= rounds & 1;
            }
            if (NWG > 1) group_sync(kAllBar, kSoftmax);
            const int cta_slot = blockIdx.x * 2 + slot;
            if (tid < RP) {
                // a row's sum over the tile groups, and what its accumulators count for: -1 for a group whose sum
                // is 0, which saw nothing (or had no tile: its accumulator is stale); a factor of 0 counts (a NaN stays)
                float sum = s_l[tid], n = s_n[tid], f0 = sum == 0.f ? -1.f : 1.f, f1 = -1.f;
                if (TG == 2) {
                    const float l0 = sum, l1 = s_l[RP + tid], n1 = s_n[RP + tid];
                    const float least = l0 == 0.f ? n1 : l1 == 0.f ? n : fminf(n, n1);
                    f0 = l0 == 0.f ? -1.f : exp2_fast(least - n);
                    f1 = l1 == 0.f ? -1.f : exp2_fast(least - n1);
                    sum = (l0 == 0.f ? 0.f : l0 * f0) + (l1 == 0.f ? 0.f : l1 * f1);
                    n = least;
                }
                if (whole) {
                    const float scale = 1.f / sum;
                    if (!(f0 < 0.f)) f0 *= scale;
                    if (!(f1 < 0.f)) f1 *= scale;
                    if (p.lse && tid < rows) p.lse[s_out[buf * RP + tid] / D] = sum == 0.f ? -INFINITY : (log2f(sum) - n) * 0.693147180559945f;
                } else {
                    float* ps = p.partial + (size_t)gridDim.x * 2 * RP * D + ((size_t)cta_slot * RP + tid) * 2;
                    ps[0] = sum == 0.f ? INFINITY : n;           // nothing seen here
                    ps[1] = sum;
                }
                s_f[tid] = f0;
                if (TG == 2) s_f[RP + tid] = f1;
            }
            pv_wait(it0 - 1);
            if (TG == 2) pv_wait(it0 - 2);
            tc_fence_after_sync();
            group_sync(kAllBar, kSoftmax);
            last |= *s_quit;
            const int dim = wq * kDimLanes + lane;
            const int nan_from = lane < kDimLanes ? s_nan[buf * D + dim] : 0x7fffffff;
            const bool nan_any = __any_sync(~0u, nan_from != 0x7fffffff);
#pragma unroll 1
            for (int r = wg * 8; r < rows; r += NWG * 8) {
                float o[8] = {};
#pragma unroll
                for (int g = 0; g < TG; ++g) {
                    float x[C::kParts][8], f[8];
#pragma unroll
                    for (int i = 0; i < C::kParts; ++i) tmem_ld<8>(lanes + C::kOutCol + g * C::kOutCols + i * RP + r, x[i]);
#pragma unroll
                    for (int k = 0; k < 8; k += 4) {
                        const float4 y = *reinterpret_cast<const float4*>(s_f + g * RP + r + k);
                        f[k] = y.x; f[k + 1] = y.y; f[k + 2] = y.z; f[k + 3] = y.w;
                    }
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 8; k += 2) {
                        F2 y = f2(x[C::kParts - 1][k], x[C::kParts - 1][k + 1]);
#pragma unroll
                        for (int i = C::kParts - 2; i >= 0; --i) y = fma2(y, f2(1.f / 16, 1.f / 16), f2(x[i][k], x[i][k + 1]));
                        float y0, y1;
                        unpack(y, y0, y1);
                        if (!(f[k] < 0.f)) o[k] = fmaf(y0, f[k], o[k]);
                        if (!(f[k + 1] < 0.f)) o[k + 1] = fmaf(y1, f[k + 1], o[k + 1]);
                    }
                }
                if (nan_any) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (nan_from < s_lim[buf * RP + r + k]) o[k] = __uint_as_float(0x7fffffffu);
                }
                if (lane < kDimLanes) {
                    if (whole) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (r + k < rows) p.out[s_out[buf * RP + r + k] + dim] = f32_to_bf16_rne(o[k]);
                    } else {
                        float* to = p.partial + ((size_t)cta_slot * RP + r) * D + dim;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (r + k < rows) to[k * D] = o[k];
                    }
                }
            }
            if (tid == 0 && s_share[seg % NS] > 0)
                p.split[blockIdx.x] = AttnSplit{s_share[seg % NS], slot, sg->row0, rows, sg->head};
            slot = 1;
            ++seg;
        } while (!last);
        tc_fence_before_sync();
    }
    __syncthreads();
    // (in line, as the branch not expected: as calls they took 64 rows from 126.6 to 128.8 us at 4 x 32768 tokens)
    if (__builtin_expect(*s_stop, 0)) {
        if (warp == kProducer) attn_drain_copies<NK, NV>(smem_u32(k_full), smem_u32(v_full), s_copied[0], s_copied[1], wait.ctl);
        if (warp == kMma) attn_drain_products(smem_u32(all_done), wait.ctl);
    }
    if (warp == kMma) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, C::kTmem);
    }
}

// Joins the partial sums of split items, CTA by CTA in order.  Latency bounds it: the
// descriptor, then all partial sums of a row at once.  W warps take a row: 4 where few
// items may be split over many CTAs each (one sequence of 30011 tokens, 8 heads: 20.3 ->
// 19.1 us), else 1 (32 sequences of 4096, 256 items: 42.4 -> 39.6 us).  A CTA looks after
// G of the descriptors.  Of few items most descriptors are empty, and a CTA for each would
// be more CTAs than fit beside the kernel before: 4 instead of 1 there take 19.1 to 18.0 us
// (500 tokens: 8.8 to 7.4; 8 take 8.3), but 2 where most are in use 39.8 to 40.8 us.
template <int D, int W, int G>
__global__ void __launch_bounds__(128) attention_combine_kernel(const __grid_constant__ AttnParams p, int rp, int grid) {
    constexpr int V = D / 32;
    __shared__ float s_acc[4][D];
    __shared__ float2 s_stat[4];
    griddep_wait();
    griddep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = W == 4 ? blockIdx.y : blockIdx.y * 4 + warp, first = W == 4 ? warp : 0;
    AttnSplit held = {};
    if (lane < G && blockIdx.x * G + lane < grid) held = p.split[blockIdx.x * G + lane];
    const float* stats = p.partial + (size_t)grid * 2 * rp * D;
    for (unsigned todo = __ballot_sync(~0u, held.n != 0 && row < held.rows); todo; todo &= todo - 1) {
        const int from = __ffs(todo) - 1, c = blockIdx.x * G + from;
        const AttnSplit s = {__shfl_sync(~0u, held.n, from), __shfl_sync(~0u, held.slot0, from),
                             __shfl_sync(~0u, held.row0, from), 0, __shfl_sync(~0u, held.head, from)};
        auto slot = [&](int i) { return (size_t)(2 * (c + i) + (i == 0 ? s.slot0 : 0)) * rp + row; };
        float acc[V] = {}, sum = 0.f, least = INFINITY;
        // this warp's pieces first + W k, kAhead of them at a time: all loads before their first use
        constexpr int kAhead = 10;
        for (int i0 = first; i0 < s.n; i0 += W * kAhead) {
            float x[kAhead][V];
            float2 st[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int i = i0 + W * k;
                st[k] = make_float2(INFINITY, 0.f);
                if (i < s.n) {
                    const float* at = p.partial + slot(i) * D + lane * V;
                    st[k] = *reinterpret_cast<const float2*>(stats + slot(i) * 2);
                    if constexpr (V == 4) {
                        const float4 y = *reinterpret_cast<const float4*>(at);
                        x[k][0] = y.x; x[k][1] = y.y; x[k][2] = y.z; x[k][3] = y.w;
                    } else {
                        const float2 y = *reinterpret_cast<const float2*>(at);
                        x[k][0] = y.x; x[k][1] = y.y;
                    }
                }
            }
            float now = least;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) now = fminf(now, st[k].x);
            const float fix = least == INFINITY ? 0.f : exp2_fast(now - least);
            sum *= fix;
#pragma unroll
            for (int v = 0; v < V; ++v) acc[v] *= fix;
            least = now;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (st[k].x == INFINITY) continue;              // nothing seen there, or no such piece
                const float f = exp2_fast(least - st[k].x);
                sum = fmaf(f, st[k].y, sum);
#pragma unroll
                for (int v = 0; v < V; ++v) acc[v] = fmaf(f, x[k][v], acc[v]);
            }
        }
        if constexpr (W == 4) {
#pragma unroll
            for (int k = 0; k < V; ++k) s_acc[warp][lane * V + k] = acc[k];
            if (lane == 0) s_stat[warp] = make_float2(least, sum);
            __syncthreads();
            if (warp > 0) {
                __syncthreads();
                continue;
            }
            float2 st[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                st[w] = s_stat[w];
                least = fminf(least, st[w].x);
            }
            sum = 0.f;
#pragma unroll
            for (int k = 0; k < V; ++k) acc[k] = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                if (st[w].x == INFINITY) continue;
                const float f = exp2_fast(least - st[w].x);
                sum = fmaf(f, st[w].y, sum);
#pragma unroll
                for (int k = 0; k < V; ++k) acc[k] = fmaf(f, s_acc[w][lane * V + k], acc[k]);
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
        if constexpr (W == 4) __syncthreads();          // the next descriptor's pieces take their place
    }
}

// ---------------------------------------------------------------- launch

struct AttnLaunch {
    CUtensorMap tk, tv;
    AttnParams p;
    int grid;
    cudaStream_t stream;
};

// RP and resident CTAs per SM of the instance for `rows` rows (at most kMaxRows).
constexpr int kMaxRows = 64;
inline int attn_rows_padded(int rows) { return rows <= 8 ? 8 : rows <= 48 ? (rows + 15) / 16 * 16 : 64; }
inline int attn_ctas_per_sm(int rp, int dim) {
    return dim == 128 ? (rp > 16 ? 1 : 2) : rp > 32 ? 1 : rp > 16 ? 2 : 3;
}

cudaError_t launch_attention_d64(int rp, const AttnLaunch& a);
cudaError_t launch_attention_d128(int rp, const AttnLaunch& a);

}  // namespace dl
