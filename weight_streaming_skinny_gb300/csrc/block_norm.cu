// The end of one block and the start of the next: norms, gate, residual scale (dl_block_norm).
#include "dl_device.cuh"
#include "dl_host.h"
#include "rows.cuh"

namespace dl {

struct NormSide {
    const void *weight, *bias;
    float eps, offset;
    int kind;
    bool f32;            // of weight and bias
};

struct BlockNormParams {
    Rows y, h, gate, r, x;
    NormSide post, pre;
    float scale, h_scale;
    int rows, dim, gate_kind;
    bool sigmoid;
    int lanes;           // of a row's team inside a warp, or 0: the CTA is the team
};

// What bounds it: the bytes of y, h and the two outputs; every element is read once, held in
// registers over both norms' sums and written once.  A row belongs to one team of threads, a part of a
// warp for short rows and a CTA for long ones, so that a sum is a few shuffles, with one barrier where
// the team is a CTA.  CTAs go over many rows, the next row's loads ahead of this one's sums.  One row of 8192
// takes 3.3 us, 16 with both norms and a gate 4.0: launch, load, sums.
//
// Sums of squares run over centred values in fp32: for the centred norm a first mean is taken
// off, then what the centred values still sum to (its rounding error), so that a mean far
// larger than the spread costs no digits.  Squares that leave fp32's range (beyond 1e37, or
// below 1e-30 where eps does not cover them) are summed again with the values scaled by a power
// of two.
template <bool CTA>
struct Team {
    float2* red;         // CTA teams: two buffers of 32 pairs, used in turn
    int lanes;           // of a team inside a warp
    int threads = 0;     // of a CTA team (all of the CTA's, or its first ones)
    int turn = 0;

    // The team's lanes: teams of one warp may go different ways.
    __device__ unsigned mask() const {
        return CTA || lanes == 32 ? ~0u : ((1u << lanes) - 1) << (threadIdx.x & 31 & ~(lanes - 1));
    }
    __device__ float sum(float v) {
        const unsigned m = mask();
        for (int o = CTA ? 16 : lanes >> 1; o; o >>= 1) v += __shfl_xor_sync(m, v, o);
        if (!CTA) return v;
        v = across(make_float2(v, 0.f), 0.f).x;
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
        return v;
    }
    __device__ float2 sum(float2 v) {
        const unsigned m = mask();
        for (int o = CTA ? 16 : lanes >> 1; o; o >>= 1) {
            v.x += __shfl_xor_sync(m, v.x, o);
            v.y += __shfl_xor_sync(m, v.y, o);
        }
        if (!CTA) return v;
        v = across(v, 0.f);
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            v.x += __shfl_xor_sync(~0u, v.x, o);
            v.y += __shfl_xor_sync(~0u, v.y, o);
        }
        return v;
    }
    __device__ float max(float v) {      // of values >= 0
        const unsigned m = mask();
        for (int o = CTA ? 16 : lanes >> 1; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(m, v, o));
        if (!CTA) return v;
        v = across(make_float2(v, 0.f), 0.f).x;
#pragma unroll
        for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
        return v;
    }
    // The CTA's warps' values, a lane each, the same in every warp.  The two buffers take turns: whoever writes
    // one has passed the barrier after its last readers' reads.
    __device__ float2 across(float2 v, float none) {
        float2* buf = red + 32 * (turn ^= 1);
        const int lane = threadIdx.x & 31;
        if (lane == 0) buf[threadIdx.x >> 5] = v;
        asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
        return lane < threads >> 5 ? buf[lane] : make_float2(none, none);
    }
};

// Eight consecutive elements of a row anywhere (aligned to their type), the first n of them its own: read as the
// aligned pieces of 16 bytes that hold them, as far as these lie in the whole array [lo, hi), and moved by what the address
// is off when they are used; at the array's ends element by element.
struct Piece {
    uint4 a, b, c;
    bool moved;              // a, b (and c) hold the group, to be moved; or a (and b) the group itself
};
struct Bounds {
    const char *lo, *hi;
};
template <bool WIDE>
__device__ __forceinline__ void any_load(Piece& p, const char* row, bool f32, int e, int n, const Bounds& in) {
    const bool wide = WIDE && f32;
    const char* at = row + (wide ? 4LL : 2LL) * e;
    const int off = (int)((uintptr_t)at & 15);
    const char* from = at - off;
    p.moved = from >= in.lo && from + (wide ? 48 : 32) <= in.hi;
    if (p.moved) {
        p.a = ldg128(from);
        p.b = ldg128(from + 16);
        if (wide) p.c = ldg128(from + 32);
    } else if (wide) {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(at);
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = k < n ? q[k] : 0;
        p.a = make_uint4(w[0], w[1], w[2], w[3]);
        p.b = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(at);
        uint32_t w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) w[k] = k < n ? q[k] : 0;
        p.a = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
}
template <bool WIDE>
__device__ __forceinline__ void any_get(const Piece& p, const char* row, bool f32, int e, int n, float* v) {
    const int off = p.moved ? (int)((uintptr_t)(row + (WIDE && f32 ? 4LL : 2LL) * e) & 15) : 0;
    uint32_t t[12] = {p.a.x, p.a.y, p.a.z, p.a.w, p.b.x, p.b.y, p.b.z, p.b.w, p.c.x, p.c.y, p.c.z, p.c.w};
    if (WIDE && f32) {
#pragma unroll
        for (int k = 0; k < 10; ++k) t[k] = off & 8 ? t[k + 2] : t[k];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(off & 4 ? t[k + 1] : t[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 6; ++k) t[k] = off & 8 ? t[k + 2] : t[k];
#pragma unroll
        for (int k = 0; k < 5; ++k) t[k] = off & 4 ? t[k + 1] : t[k];
#pragma unroll
        for (int k = 0; k < 4; ++k) bf16x2_to_f32(__funnelshift_r(t[k], t[k + 1], (off & 2) * 8), v[2 * k], v[2 * k + 1]);
    }
    if (n < 8) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k >= n) v[k] = 0.f;
    }
}
// Eight values to a row anywhere, the first n of them.
__device__ __forceinline__ void any_store(char* row, bool f32, int e, int n, const float* v) {
    if (f32) {
        float* q = reinterpret_cast<float*>(row) + e;
        if (n < 8) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (k < n) q[k] = v[k];
        } else if ((uintptr_t)q & 4) {
            q[0] = v[0];
#pragma unroll
            for (int k = 1; k < 7; k += 2) *reinterpret_cast<float2*>(q + k) = make_float2(v[k], v[k + 1]);
            q[7] = v[7];
        } else {
#pragma unroll
            for (int k = 0; k < 8; k += 2) *reinterpret_cast<float2*>(q + k) = make_float2(v[k], v[k + 1]);
        }
        return;
    }
    uint16_t* q = reinterpret_cast<uint16_t*>(row) + e;
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = f32x2_to_bf16x2(v[2 * k], v[2 * k + 1]);
    if (n < 8) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < n) q[k] = (uint16_t)(w[k >> 1] >> 16 * (k & 1));
    } else if ((uintptr_t)q & 2) {
        q[0] = (uint16_t)w[0];
        uint32_t* two = reinterpret_cast<uint32_t*>(q + 1);
#pragma unroll
        for (int k = 0; k < 3; ++k) two[k] = __funnelshift_r(w[k], w[k + 1], 16);
        q[7] = (uint16_t)(w[3] >> 16);
    } else {
        uint32_t* two = reinterpret_cast<uint32_t*>(q);
#pragma unroll
        for (int k = 0; k < 4; ++k) two[k] = w[k];
    }
}

// How a thread of a team holds its elements of a row: every size-th one; groups of 8 consecutive ones, whole and
// aligned; the same of rows that are not.
constexpr int kSingle = 0, kGroups = 1, kMoved = 2;
template <int E, int M>
struct Slots {
    int first, step, count, n, dim;      // elements or groups: the thread's first, from one to the next, how many; its elements

    __device__ Slots(int rank, int size, int dim_) : first(rank), step(size), dim(dim_) {
        const int all = M == kSingle ? dim : (dim + 7) / 8;
        count = rank < all ? (all - rank + size - 1) / size : 0;
        n = M == kSingle ? count : M == kGroups ? 8 * count : count ? 8 * (count - 1) + min(8, dim - 8 * (rank + (count - 1) * size)) : 0;
    }
    __device__ __forceinline__ bool has(int i) const { return i < n; }
    // of a row of an array
    __device__ __forceinline__ void load(const void* p, bool f32, float (&v)[E], const Bounds& in) const {
        if constexpr (M == kSingle) {
            if (f32) {
                const float* q = static_cast<const float*>(p) + first;
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = i < count ? q[i * step] : 0.f;
            } else {
                const uint16_t* q = static_cast<const uint16_t*>(p) + first;
#pragma unroll
                for (int i = 0; i < E; ++i) v[i] = i < count ? bf16_bits_to_f32(q[i * step]) : 0.f;
            }
        } else {
#pragma unroll
            for (int i = 0; i < E / 8; ++i) {
                const int e = (first + i * step) * 8;
                if (i >= count) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[8 * i + k] = 0.f;
                } else if (M == kGroups) {
                    row_load8(p, f32, e, v + 8 * i);
                } else {
                    Piece t = {};
                    any_load<true>(t, static_cast<const char*>(p), f32, e, min(n - 8 * i, 8), in);
                    any_get<true>(t, static_cast<const char*>(p), f32, e, min(n - 8 * i, 8), v + 8 * i);
                }
            }
        }
    }
    // of a row by itself
    __device__ __forceinline__ void load(const void* p, bool f32, float (&v)[E]) const {
        const char* at = static_cast<const char*>(p);
        load(p, f32, v, Bounds{at, at + (size_t)dim * (f32 ? 4 : 2)});
    }
    __device__ __forceinline__ void store(void* p, bool f32, const float (&v)[E]) const {
        if constexpr (M == kSingle) {
            if (f32) {
                float* q = static_cast<float*>(p) + first;
#pragma unroll
                for (int i = 0; i < E; ++i)
                    if (i < count) q[i * step] = v[i];
            } else {
                uint16_t* q = static_cast<uint16_t*>(p) + first;
#pragma unroll
                for (int i = 0; i < E; ++i)
                    if (i < count) q[i * step] = f32_to_bf16_rne(v[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < E / 8; ++i) {
                if (i >= count) continue;
                const int e = (first + i * step) * 8;
                if (M == kGroups)
                    row_store8(p, f32, e, v + 8 * i);
                else
                    any_store(static_cast<char*>(p), f32, e, min(n - 8 * i, 8), v + 8 * i);
            }
        }
    }
};

// Pairs of a thread's elements: v = v * s, v = v * w, sums of squares.
template <int E>
__device__ __forceinline__ void times(float (&v)[E], float s) {
#pragma unroll
    for (int i = 0; i < E; i += 2) unpack(mul2(f2(v[i], v[i + 1]), f2(s, s)), v[i], v[i + 1]);
}
template <int E>
__device__ __forceinline__ void times(float (&v)[E], const float (&w)[E]) {
#pragma unroll
    for (int i = 0; i < E; i += 2) unpack(mul2(f2(v[i], v[i + 1]), f2(w[i], w[i + 1])), v[i], v[i + 1]);
}
template <int E>
__device__ __forceinline__ float squares(const float (&v)[E]) {
    F2 s = f2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < E; i += 2) {
        const F2 x = f2(v[i], v[i + 1]);
        s = fma2(x, x, s);
    }
    float a, b;
    unpack(s, a, b);
    return a + b;
}

// v = N(v): the elements of one row, zeros past its end.
template <int E, int M, bool CTA>
__device__ __forceinline__ void normalise(float (&v)[E], const NormSide& n, Team<CTA>& team, const Slots<E, M>& slots, int dim) {
    const float inv_dim = 1.f / dim;
    float ss;
    if (n.kind == DL_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(v[i], inv_dim, s);
        const float mean = team.sum(s);
        float2 t = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < E; ++i) {
            v[i] = slots.has(i) ? v[i] - mean : 0.f;
            t.x = fmaf(v[i], inv_dim, t.x);
        }
        t.y = squares(v);
        t = team.sum(t);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = slots.has(i) ? v[i] - t.x : 0.f;
        ss = t.y <= 1e37f ? fmaxf(fmaf(-dim * t.x, t.x, t.y), 0.f) : t.y;
    } else {
        ss = team.sum(squares(v));
    }
    float inv = 1.f / sqrtf(fmaf(ss, inv_dim, n.eps));
    if (ss > 1e37f || (ss < 1e-30f && n.eps < 1e-30f)) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) m = fmaxf(m, fabsf(v[i]));
        m = team.max(m);
        if (m > 0.f && m <= 3.4028235e38f) {
            const float up = ldexpf(1.f, -max(ilogbf(m), -100));
            times(v, up);
            ss = team.sum(squares(v));
            inv = 1.f / sqrtf(fmaf(ss, inv_dim, n.eps * up * up));
        }
    }
    times(v, inv);
    float w[E];
    if (n.weight) {
        slots.load(n.weight, n.f32, w);
        if (n.offset != 0.f) {
#pragma unroll
            for (int i = 0; i < E; ++i) w[i] += n.offset;
        }
        times(v, w);
    }
    if (n.bias) {
        slots.load(n.bias, n.f32, w);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] += w[i];
    }
}

// What is read of a row ahead of its turn: up to 16 elements of y and h a thread (up to 8 where they are not
// aligned), of 16 bits, or of 32.
template <int E, int M, bool WIDE>
struct Ahead {
    static constexpr bool kOn = M == kGroups && E <= 16, kPieces = M == kMoved && E == 8;
    uint4 v[kOn ? E / 8 : 1][WIDE ? 2 : 1];
    Piece piece;

    __device__ __forceinline__ void load(const Slots<E, M>& s, const char* p, bool f32, const Bounds& in) {
        if constexpr (kOn) {
#pragma unroll
            for (int i = 0; i < E / 8; ++i) {
                if (i >= s.count) continue;
                const int e = (s.first + i * s.step) * 8;
                if (WIDE && f32) {
                    v[i][0] = ldg128(p + 4 * e);
                    v[i][WIDE] = ldg128(p + 4 * e + 16);
                } else {
                    v[i][0] = ldg128(p + 2 * e);
                }
            }
        } else if constexpr (kPieces) {
            if (s.count) any_load<WIDE>(piece, p, f32, 8 * s.first, s.n, in);
        }
    }
    __device__ __forceinline__ void get(const Slots<E, M>& s, const char* p, bool f32, float (&x)[E], const Bounds& in) const {
        if constexpr (kOn) {
#pragma unroll
            for (int i = 0; i < E / 8; ++i) {
                float* t = x + 8 * i;
                const uint4 a = v[i][0], b = v[i][WIDE];
                if (i >= s.count) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) t[k] = 0.f;
                } else if (WIDE && f32) {
                    t[0] = __uint_as_float(a.x); t[1] = __uint_as_float(a.y); t[2] = __uint_as_float(a.z); t[3] = __uint_as_float(a.w);
                    t[4] = __uint_as_float(b.x); t[5] = __uint_as_float(b.y); t[6] = __uint_as_float(b.z); t[7] = __uint_as_float(b.w);
                } else {
                    bf16x2_to_f32(a.x, t[0], t[1]);
                    bf16x2_to_f32(a.y, t[2], t[3]);
                    bf16x2_to_f32(a.z, t[4], t[5]);
                    bf16x2_to_f32(a.w, t[6], t[7]);
                }
            }
        } else if constexpr (kPieces) {
            if (s.count) {
                any_get<WIDE>(piece, p, f32, 8 * s.first, s.n, x);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) x[k] = 0.f;
            }
        } else {
            s.load(p, f32, x, in);
        }
    }
};

// 1 / (1 + exp(-x)), by an exponential that is at most 1: the quick quotient takes divisors below 2^126 only.
__device__ __forceinline__ float sigmoid(float x) {
    const float e = expf(-fabsf(x)), q = __fdividef(1.f, 1.f + e);
    return x < 0.f ? e * q : q;
}

__device__ __forceinline__ Bounds bounds_of(const Rows& r, int rows, int dim) {
    return Bounds{r.ptr, row_ptr(r, rows - 1) + (size_t)dim * (r.f32 ? 4 : 2)};
}

// v = h_scale h + scale act(gate) post(v), of what there is.
template <int E, int M, bool CTA>
__device__ __forceinline__ void join(float (&v)[E], const float (&h)[E], const BlockNormParams& p, long long row, Team<CTA>& team,
                                     const Slots<E, M>& slots) {
    if (p.y.ptr) {
        if (p.post.kind != DL_NORM_NONE) normalise<E, M, CTA>(v, p.post, team, slots, p.dim);
        if (p.gate_kind != DL_GATE_NONE) {
            float g[E];
            if (p.gate_kind == DL_GATE_ROW) {
                const float one = row_load1(row_ptr(p.gate, row), p.gate.f32, 0);
#pragma unroll
                for (int i = 0; i < E; ++i) g[i] = one;
            } else {
                if (p.gate_kind == DL_GATE_FULL)
                    slots.load(row_ptr(p.gate, row), p.gate.f32, g, bounds_of(p.gate, p.rows, p.dim));
                else
                    slots.load(p.gate.ptr, p.gate.f32, g);
            }
            if (p.sigmoid) {
#pragma unroll
                for (int i = 0; i < E; ++i) g[i] = sigmoid(g[i]);
            }
            times(v, g);
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (!slots.has(i)) v[i] = 0.f;       // (an infinite gate times an absent element)
        }
        if (p.scale != 1.f) times(v, p.scale);
        if (p.h.ptr) {
#pragma unroll
            for (int i = 0; i < E; i += 2)
                unpack(fma2(f2(h[i], h[i + 1]), f2(p.h_scale, p.h_scale), f2(v[i], v[i + 1])), v[i], v[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = p.h_scale * h[i];
    }
}

// WIDE: y or h is fp32; T: the most threads of a CTA
template <int E, int M, bool CTA, bool WIDE, int T>
__global__ void __launch_bounds__(T, T == 128 ? 4 : 1024 / T) block_norm_kernel(const __grid_constant__ BlockNormParams p) {
    __shared__ float2 red[CTA ? 64 : 1];
    Team<CTA> team{red, p.lanes, (int)blockDim.x};
    const int size = CTA ? blockDim.x : p.lanes, rank = CTA ? threadIdx.x : threadIdx.x & (p.lanes - 1);
    long long row = CTA ? blockIdx.x : ((long long)blockIdx.x * blockDim.x + threadIdx.x) / p.lanes;
    const long long step = CTA ? gridDim.x : (long long)gridDim.x * blockDim.x / p.lanes;
    const Slots<E, M> slots(rank, size, p.dim);
    griddep_wait();
    griddep_launch_dependents();
    Ahead<E, M, WIDE> next_y = {}, next_h = {};
    const Bounds in_y = bounds_of(p.y, p.rows, p.dim), in_h = bounds_of(p.h, p.rows, p.dim);
    if (row < p.rows) {
        if (p.y.ptr) next_y.load(slots, row_ptr(p.y, row), p.y.f32, in_y);
        if (p.h.ptr) next_h.load(slots, row_ptr(p.h, row), p.h.f32, in_h);
    }
    for (; row < p.rows; row += step) {  // (teams of a warp may leave at different times: their shuffles are their own)
        float v[E], h[E];
        if (p.y.ptr) next_y.get(slots, row_ptr(p.y, row), p.y.f32, v, in_y);
        if (p.h.ptr) next_h.get(slots, row_ptr(p.h, row), p.h.f32, h, in_h);
        if (row + step < p.rows) {
            if (p.y.ptr) next_y.load(slots, row_ptr(p.y, row + step), p.y.f32, in_y);
            if (p.h.ptr) next_h.load(slots, row_ptr(p.h, row + step), p.h.f32, in_h);
        }
        join(v, h, p, row, team, slots);
        if (p.r.ptr) slots.store(row_ptr(p.r, row), p.r.f32, v);
        if (p.x.ptr) {
            if (p.pre.kind != DL_NORM_NONE) normalise<E, M, CTA>(v, p.pre, team, slots, p.dim);
            slots.store(row_ptr(p.x, row), p.x.f32, v);
        }
    }
}

// Many long rows, all streams there and in 16-byte pieces: rows come into a ring of shared memory by bulk copies,
// stages ahead, and what is made of them goes back from the same place: r over h, x over y.  One warp has the
// copies made both ways; the others wait for a row, and, once, for its sum.  16384 x 8192 in bf16: 173 us, 6.2 TB/s
// (with the next row in registers instead 234, elements singly instead of in pairs 196).
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

struct RingParams {
    BlockNormParams n;
    int stages, y_bytes, h_bytes;        // of a row
    WaitCtl wait;
    int withhold;                        // test hook: CTA 0 never copies its k-th row (0: none)
};

// Eight values as pairs, and back.
__device__ __forceinline__ void pairs_bf16(uint4 a, F2 (&t)[4]) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = f2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
}
template <bool F32>
__device__ __forceinline__ void pairs_shared(uint32_t p, F2 (&t)[4]) {
    if (F32) {
        const uint4 a = lds128(p), b = lds128(p + 16);
        t[0] = f2(__uint_as_float(a.x), __uint_as_float(a.y));
        t[1] = f2(__uint_as_float(a.z), __uint_as_float(a.w));
        t[2] = f2(__uint_as_float(b.x), __uint_as_float(b.y));
        t[3] = f2(__uint_as_float(b.z), __uint_as_float(b.w));
    } else {
        pairs_bf16(lds128(p), t);
    }
}
template <bool F32>
__device__ __forceinline__ void put_pairs_shared(uint32_t p, const F2* t) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) unpack(t[k], v[2 * k], v[2 * k + 1]);
    if (F32) {
        sts128(p, __float_as_int(v[0]), __float_as_int(v[1]), __float_as_int(v[2]), __float_as_int(v[3]));
        sts128(p + 16, __float_as_int(v[4]), __float_as_int(v[5]), __float_as_int(v[6]), __float_as_int(v[7]));
    } else {
        sts128(p, f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]), f32x2_to_bf16x2(v[6], v[7]));
    }
}
__device__ __forceinline__ void pairs_global(const void* p, bool f32, int e, F2 (&t)[4]) {
    float v[8];
    row_load8(p, f32, e, v);
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = f2(v[2 * k], v[2 * k + 1]);
}

template <int N>
__device__ __forceinline__ float pair_squares(const F2 (&v)[N]) {
    F2 s = f2(0.f, 0.f), t = s;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        s = fma2(v[i], v[i], s);
        t = fma2(v[i + 1], v[i + 1], t);
    }
    float a, b;
    unpack(add2(s, t), a, b);
    return a + b;
}
template <int N>
__device__ __forceinline__ float pair_sum(const F2 (&v)[N], float scale) {
    F2 s = f2(0.f, 0.f);
    const F2 w = f2(scale, scale);
#pragma unroll
    for (int i = 0; i < N; ++i) s = fma2(v[i], w, s);
    float a, b;
    unpack(s, a, b);
    return a + b;
}

// As normalise(), for a row that the team's threads hold to the last element: the centred (and, beyond
// fp32's range, scaled) values stay in v, what they are to be multiplied with is returned.
template <int N>
__device__ __forceinline__ float centred(F2 (&v)[N], const NormSide& n, Team<true>& team, int dim) {
    const float inv_dim = 1.f / dim;
    float ss;
    if (n.kind == DL_NORM_LAYER) {
        const float mean = team.sum(pair_sum(v, inv_dim));
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = add2(v[i], f2(-mean, -mean));
        const float2 t = team.sum(make_float2(pair_sum(v, inv_dim), pair_squares(v)));
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = add2(v[i], f2(-t.x, -t.x));
        ss = t.y <= 1e37f ? fmaxf(fmaf(-dim * t.x, t.x, t.y), 0.f) : t.y;
    } else {
        ss = team.sum(pair_squares(v));
    }
    float inv = 1.f / sqrtf(fmaf(ss, inv_dim, n.eps));
    if (ss > 1e37f || (ss < 1e-30f && n.eps < 1e-30f)) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float a, b;
            unpack(v[i], a, b);
            m = fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
        }
        m = team.max(m);
        if (m > 0.f && m <= 3.4028235e38f) {
            const float up = ldexpf(1.f, -max(ilogbf(m), -100));
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = mul2(v[i], f2(up, up));
            ss = team.sum(pair_squares(v));
            inv = 1.f / sqrtf(fmaf(ss, inv_dim, n.eps * up * up));
        }
    }
    return inv;
}

// Eight values of N(v): v inv w + b.
__device__ __forceinline__ void finish8(F2* v, float inv, const NormSide& n, int e) {
    F2 w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = mul2(v[k], f2(inv, inv));
    if (n.weight) {
        pairs_global(n.weight, n.f32, e, w);
        if (n.offset != 0.f) {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = add2(w[k], f2(n.offset, n.offset));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = mul2(v[k], w[k]);
    }
    if (n.bias) {
        pairs_global(n.bias, n.f32, e, w);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = add2(v[k], w[k]);
    }
}

// The threads that compute hold E elements of a row each, all of it; a warp more copies.  YF, HF, XF: y, h and r, x
// are fp32.
template <int E, bool YF, bool HF, bool XF>
__global__ void __launch_bounds__(256 + 32, 2) block_norm_ring_kernel(const __grid_constant__ RingParams q) {
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ float2 red[64];
    __shared__ __align__(8) unsigned long long bars[16];         // rows in place, rows made
    __shared__ volatile int dead;        // a wait gave up: nobody waits any more, nothing is copied
    const BlockNormParams& p = q.n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = (blockDim.x >> 5) - 1, S = q.stages;
    const uint32_t full = smem_u32(bars), made = full + 64, ring = smem_u32(smem);
    const int stage_bytes = q.y_bytes + q.h_bytes;
    if (tid == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(full + 8 * i, 1);
            mbar_init(made + 8 * i, warps);
        }
        fence_mbarrier_init();
        dead = 0;
    }
    __syncthreads();
    griddep_wait();
    griddep_launch_dependents();
    const int n = (int)((p.rows - 1 - (int)blockIdx.x) / (int)gridDim.x) + 1;       // rows of this CTA
    auto row_of = [&](int i) { return (long long)blockIdx.x + (long long)i * gridDim.x; };
    if (warp == warps) {
        if (lane == 0) {
            auto load = [&](int i, int stage) {
                const uint32_t to = ring + stage * stage_bytes, bar = full + 8 * stage;
                mbar_arrive_expect_tx(bar, stage_bytes);
                if (blockIdx.x == 0 && i + 1 == q.withhold) return;
                bulk_load(to, row_ptr(p.y, row_of(i)), q.y_bytes, bar);
                bulk_load(to + q.y_bytes, row_ptr(p.h, row_of(i)), q.h_bytes, bar);
            };
            int loaded = 0, stage = 0, turn = 0;
            for (; loaded < min(S, n); ++loaded) load(loaded, loaded);
            for (int i = 0; i < n && !dead; ++i) {
                if (!mbar_wait_bounded(made + 8 * stage, turn & 1, q.wait, kErrProducerWait)) {
                    dead = 1;
                    break;
                }
                if (dead) break;
                const uint32_t from = ring + stage * stage_bytes;
                bulk_store(row_ptr(p.x, row_of(i)), from, p.dim * (XF ? 4 : 2));
                bulk_store(row_ptr(p.r, row_of(i)), from + q.y_bytes, q.h_bytes);
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                if (loaded < n) {
                    asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                    load(loaded++, stage);
                }
                if (++stage == S) stage = 0, ++turn;
            }
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
            if (dead)                    // what is on its way arrives before the CTA leaves
                for (int i = max(loaded - S, 0); i < loaded; ++i)
                    mbar_wait_bounded(full + 8 * (i % S), (i / S) & 1, q.wait, kErrDrainWait);
        }
        return;
    }
    Team<true> team{red, 0, 32 * warps};
    const int size = 256 * warps;        // elements from one of a thread's groups of 8 to the next
    int stage = 0, turn = 0;
    for (int i = 0; i < n; ++i) {
        if (!dead && !mbar_wait_bounded(full + 8 * stage, turn & 1, q.wait, kErrConsumerWait)) dead = 1;
        __syncwarp();
        const uint32_t at = ring + stage * stage_bytes, at_y = at + tid * (YF ? 32 : 16), at_h = at + q.y_bytes + tid * (HF ? 32 : 16);
        F2 v[E / 2];
#pragma unroll
        for (int k = 0; k < E / 8; ++k) {
            F2 t[4];
            pairs_shared<YF>(at_y + k * size * (YF ? 4 : 2), t);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * k + j] = t[j];
        }
        if (p.post.kind != DL_NORM_NONE) {
            const float inv = centred(v, p.post, team, p.dim);
#pragma unroll
            for (int k = 0; k < E / 8; ++k) finish8(v + 4 * k, inv, p.post, tid * 8 + k * size);
        }
        if (p.gate_kind != DL_GATE_NONE) {
            const float one = p.gate_kind == DL_GATE_ROW ? row_load1(row_ptr(p.gate, row_of(i)), p.gate.f32, 0) : 0.f;
#pragma unroll
            for (int k = 0; k < E / 8; ++k) {
                float g[8], a, b;
                if (p.gate_kind == DL_GATE_ROW) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) g[j] = one;
                } else {
                    row_load8(p.gate.ptr, p.gate.f32, tid * 8 + k * size, g);
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    a = g[2 * j];
                    b = g[2 * j + 1];
                    if (p.sigmoid) {
                        a = sigmoid(a);
                        b = sigmoid(b);
                    }
                    v[4 * k + j] = mul2(v[4 * k + j], f2(a, b));
                }
            }
        }
        const F2 scale = f2(p.scale, p.scale), h_scale = f2(p.h_scale, p.h_scale);
#pragma unroll
        for (int k = 0; k < E / 8; ++k) {
            F2 t[4];
            pairs_shared<HF>(at_h + k * size * (HF ? 4 : 2), t);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[4 * k + j] = fma2(t[j], h_scale, mul2(v[4 * k + j], scale));
            put_pairs_shared<HF>(at_h + k * size * (HF ? 4 : 2), v + 4 * k);
        }
        const float inv = centred(v, p.pre, team, p.dim);
#pragma unroll
        for (int k = 0; k < E / 8; ++k) {
            finish8(v + 4 * k, inv, p.pre, tid * 8 + k * size);
            // (all have read y: the norm's sum came after it)
            put_pairs_shared<XF>(at + (tid * 8 + k * size) * (XF ? 4 : 2), v + 4 * k);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(made + 8 * stage);
        if (++stage == S) stage = 0, ++turn;
    }
}

constexpr int kMaxDim = 32768;

template <int E, int M, bool CTA, int T>
cudaError_t launch_norm(const BlockNormParams& p, long long grid, int threads, cudaStream_t stream) {
    constexpr bool kWide = M == kGroups && E <= 16;
    return kWide && (p.y.f32 || p.h.f32)
               ? launch_dependent(block_norm_kernel<E, M, CTA, kWide, T>, dim3((unsigned)grid), dim3(threads), 0, stream, p)
               : launch_dependent(block_norm_kernel<E, M, CTA, false, T>, dim3((unsigned)grid), dim3(threads), 0, stream, p);
}

template <int E, bool YF, bool HF, bool XF>
cudaError_t launch_ring_kernel(RingParams& q, int sm_count, cudaStream_t stream) {
    const int threads = q.n.dim / E, stage = q.y_bytes + q.h_bytes;
    // CTAs of an SM: 512 threads' worth, with two rows each at least
    constexpr int kSm = 220 * 1024;
    int ctas = 512 / threads;
    while (ctas > 1 && kSm / (ctas * stage) < 2) --ctas;
    q.stages = kSm / (ctas * stage);
    if (q.stages > 4) q.stages = 4;
    const size_t smem = (size_t)q.stages * stage;
    const cudaError_t e = raise_smem<block_norm_ring_kernel<E, YF, HF, XF>>(kSm);
    if (e != cudaSuccess) return e;
    const int most = ctas * sm_count;
    return launch_dependent(block_norm_ring_kernel<E, YF, HF, XF>, dim3(q.n.rows < most ? q.n.rows : most), dim3(threads + 32),
                            smem, stream, q);
}

template <int E, bool HF>
cudaError_t launch_ring_types(RingParams& q, int sm_count, cudaStream_t stream) {
    if (!q.n.y.f32) return launch_ring_kernel<E, false, HF, false>(q, sm_count, stream);
    return q.n.x.f32 ? launch_ring_kernel<E, true, HF, true>(q, sm_count, stream)
                     : launch_ring_kernel<E, true, HF, false>(q, sm_count, stream);
}

// Many long rows through the ring: where all streams are there, r has h's type, x is no wider than y, and
// whole warps of threads hold a row: 16 elements each up to 4096, 32 up to 8192.  Rows of up to 4096 with h in bf16
// have enough of them in registers (4000 x 4096: 24 us both, with a norm of y 35 and 33; with h in fp32 37 and 47), and
// a gate for each element would not come through it (4000 x 8192: 81 and 74 us; without 47 and 46, with a norm of y 49
// and 69).
static bool launch_ring(const BlockNormParams& p, int sm_count, const WaitCtl& wait, int withhold, cudaStream_t stream, cudaError_t& e) {
    if (!p.y.ptr || !p.h.ptr || !p.r.ptr || !p.x.ptr || p.pre.kind == DL_NORM_NONE || p.r.f32 != p.h.f32 ||
        (p.x.f32 && !p.y.f32) || p.gate_kind == DL_GATE_FULL || (p.dim <= 4096 && !p.h.f32) || p.rows < 4 * sm_count ||
        p.dim > 8192 || p.dim % (p.dim <= 4096 ? 512 : 1024))
        return false;
    RingParams q = {p, 0, p.dim * (p.y.f32 ? 4 : 2), p.dim * (p.h.f32 ? 4 : 2), wait, withhold};
    e = p.dim <= 4096  ? launch_ring_types<16, true>(q, sm_count, stream)
        : p.h.f32 ? launch_ring_types<32, true>(q, sm_count, stream)
                  : launch_ring_types<32, false>(q, sm_count, stream);
    return true;
}

template <int M>
cudaError_t launch_norm_rows(BlockNormParams& p, int sm_count, const WaitCtl& wait, int withhold, cudaStream_t stream) {
    const int groups = (p.dim + 7) / 8;
    if (groups <= 64) {                     // teams inside a warp, two groups a thread at most
        int lanes = 8;
        while (lanes < 32 && lanes < groups) lanes *= 2;
        const int threads = 128;
        const long long all = ((long long)p.rows * lanes + threads - 1) / threads, most = 16LL * sm_count;
        const long long grid = all < most ? all : most;
        p.lanes = lanes;
        return groups <= lanes ? launch_norm<8, M, false, 128>(p, grid, threads, stream)
                               : launch_norm<16, M, false, 128>(p, grid, threads, stream);
    }
    cudaError_t e;
    if (M == kGroups && launch_ring(p, sm_count, wait, withhold, stream, e)) return e;
    // A CTA each, as few groups a thread as 1024 threads allow: one up to 8192 (8000 rows of 1000, 2000, 3000, 8000: 11, 23, 38,
    // 88 us; two 20, 29, 44, 118 us; rows of 1000 by a warp 26), single elements too (999 rows of 1537: 13 us; two 30)
    const int per = groups <= 1024 ? 1 : groups <= 2048 ? 2 : 4, threads = ((groups + per - 1) / per + 31) / 32 * 32;
    const long long fit = 1024 / threads, most = fit * sm_count, grid = p.rows < most ? p.rows : most;
    if (per == 1)
        return threads <= 256 ? launch_norm<8, M, true, 256>(p, grid, threads, stream)
                              : launch_norm<8, M, true, 1024>(p, grid, threads, stream);
    return per == 2 ? launch_norm<16, M, true, 1024>(p, grid, threads, stream)
                    : launch_norm<32, M, true, 1024>(p, grid, threads, stream);
}

static dl_status check_norm(const dl_norm* n, const char* name, NormSide& out) {
    out = NormSide{};
    if (!n || n->kind == DL_NORM_NONE) return DL_OK;
    if (n->kind != DL_NORM_RMS && n->kind != DL_NORM_LAYER)
        return host_fail(DL_ERR_INVALID_ARG, "%s: unknown kind %d", name, n->kind);
    if (n->dtype != DL_ROWS_BF16 && n->dtype != DL_ROWS_F32)
        return host_fail(DL_ERR_INVALID_ARG, "%s: unknown dtype %d", name, n->dtype);
    if (!(n->eps >= 0.f) || !(n->eps <= 3.4028235e38f) || !(n->offset - n->offset == 0.f))
        return host_fail(DL_ERR_INVALID_ARG, "%s: eps must be finite and >= 0, offset finite", name);
    const uintptr_t el = n->dtype == DL_ROWS_F32 ? 3 : 1;
    if (((uintptr_t)n->weight | (uintptr_t)n->bias) & el)
        return host_fail(DL_ERR_MISALIGNED, "%s: weight and bias must be aligned to their type", name);
    out = NormSide{n->weight, n->bias, n->eps, n->offset, n->kind, n->dtype == DL_ROWS_F32};
    return DL_OK;
}

}  // namespace dl

extern "C" dl_status dl_block_norm(const dl_rows* y, const dl_norm* post, const dl_rows* gate, int gate_kind, int gate_act,
                                   float scale, const dl_rows* h, float h_scale, const dl_norm* pre,
                                   const dl_rows* h_out, const dl_rows* x_out, int rows, int dim, void* stream) {
    using namespace dl;
    BlockNormParams p = {};
    if (rows < 0) return host_fail(DL_ERR_INVALID_ARG, "rows=%d must be >= 0", rows);
    if (dim < 1 || dim > kMaxDim) return host_fail(DL_ERR_UNSUPPORTED_SHAPE, "dim=%d is outside [1, %d]", dim, kMaxDim);
    if (gate_kind < DL_GATE_NONE || gate_kind > DL_GATE_FULL)
        return host_fail(DL_ERR_INVALID_ARG, "unknown gate kind %d", gate_kind);
    if (gate_act != DL_GATE_PLAIN && gate_act != DL_GATE_SIGMOID)
        return host_fail(DL_ERR_INVALID_ARG, "unknown gate_act %d", gate_act);
    const bool has_y = y && y->data, has_h = h && h->data, has_gate = gate_kind != DL_GATE_NONE;
    if (rows > 0) {
        if (!has_y && !has_h) return host_fail(DL_ERR_INVALID_ARG, "y and h are both NULL");
        if (has_gate && (!gate || !gate->data)) return host_fail(DL_ERR_INVALID_ARG, "the gate is NULL");
        if (!(h_out && h_out->data) && !(x_out && x_out->data))
            return host_fail(DL_ERR_INVALID_ARG, "h_out and x_out are both NULL");
    }
    if (!has_y && rows > 0 && (has_gate || (post && post->kind != DL_NORM_NONE)))
        return host_fail(DL_ERR_INVALID_ARG, "a gate or a norm of y needs y");
    if (pre && pre->kind != DL_NORM_NONE && rows > 0 && !(x_out && x_out->data))
        return host_fail(DL_ERR_INVALID_ARG, "pre needs x_out");
    dl_status s;
    if ((s = check_norm(post, "post", p.post)) != DL_OK || (s = check_norm(pre, "pre", p.pre)) != DL_OK) return s;
    if (!(scale - scale == 0.f) || !(h_scale - h_scale == 0.f))
        return host_fail(DL_ERR_INVALID_ARG, "scale and h_scale must be finite");
    const int gate_dim = gate_kind == DL_GATE_ROW ? 1 : dim, gate_rows = gate_kind == DL_GATE_CHANNEL ? 1 : rows;
    if ((s = check_rows(y, "y", rows, dim, p.y)) != DL_OK || (s = check_rows(h, "h", rows, dim, p.h)) != DL_OK ||
        (has_gate && (s = check_rows(gate, "gate", gate_rows, gate_dim, p.gate)) != DL_OK) ||
        (s = check_rows(h_out, "h_out", rows, dim, p.r)) != DL_OK ||
        (s = check_rows(x_out, "x_out", rows, dim, p.x)) != DL_OK)
        return s;
    // an output may lie in the place of y or h, row for row; no other overlap
    for (const Rows* out : {&p.r, &p.x}) {
        const char* name = out == &p.r ? "h_out" : "x_out";
        for (const Rows* in : {&p.y, &p.h})
            if (!same_rows(*out, *in) && rows_meet(*out, rows, dim, *in, rows, dim))
                return host_fail(DL_ERR_INVALID_ARG, "%s overlaps y or h in another layout", name);
        if (rows_meet(*out, rows, dim, p.gate, gate_rows, gate_dim))
            return host_fail(DL_ERR_INVALID_ARG, "%s overlaps the gate", name);
        for (const NormSide* n : {&p.post, &p.pre})
            for (const void* w : {n->weight, n->bias})
                if (rows_meet(*out, rows, dim, Rows{(char*)w, 0, n->f32}, 1, dim))
                    return host_fail(DL_ERR_INVALID_ARG, "%s overlaps a norm's weight or bias", name);
    }
    if (rows_meet(p.r, rows, dim, p.x, rows, dim)) return host_fail(DL_ERR_INVALID_ARG, "h_out and x_out overlap");
    if (rows == 0) return host_ok();
    p.scale = scale;
    p.h_scale = h_scale;
    p.rows = rows;
    p.dim = dim;
    p.gate_kind = gate_kind;
    p.sigmoid = gate_act == DL_GATE_SIGMOID;
    // groups of 8 elements need every row and weight on a 16-byte boundary
    bool vec = dim % 8 == 0;
    for (const Rows* t : {&p.y, &p.h, &p.r, &p.x}) vec = vec && rows_aligned16(*t, rows);
    if (gate_kind >= DL_GATE_CHANNEL) vec = vec && rows_aligned16(p.gate, gate_rows);
    for (const NormSide* n : {&p.post, &p.pre}) vec = vec && !(((uintptr_t)n->weight | (uintptr_t)n->bias) & 15);
    HostDevice dev;
    if ((s = host_device(dev)) != DL_OK) return s;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const WaitCtl wait = {dev.err_word, dev.wait_limit_ns};
    // Rows that are not aligned: of bf16 and more than 64 elements in groups, moved, others singly.  Many rows gain by it
    // (moved and singly: 8000 x 1001 22.7 and 26.1 us, 2999 83.5 and 102; 4000 x 16383 246 and 451; 30000 x 100 13.6 and 14.5),
    // and so do few beyond 8192 (16 x 9001 6.8 and 13.0); few shorter ones, and those next to the limit, lose (400 x 2999 7.3
    // and 6.4, 5001 9.6 and 8.9; 16384 x 65 9.3 and 8.9), as they would up to it (16384 x 41 6.2 and 5.8) and in fp32
    // (8000 x 2999, gated, 152 and 131).
    const int hold = vec ? kGroups : dim > 64 && !p.y.f32 && !p.h.f32 ? kMoved : kSingle;
    const cudaError_t e = hold == kGroups  ? launch_norm_rows<kGroups>(p, dev.sm_count, wait, dev.withhold_stage, st)
                          : hold == kMoved ? launch_norm_rows<kMoved>(p, dev.sm_count, wait, dev.withhold_stage, st)
                                           : launch_norm_rows<kSingle>(p, dev.sm_count, wait, dev.withhold_stage, st);
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "block_norm launch: %s", cudaGetErrorString(e));
    return host_ok();
}
