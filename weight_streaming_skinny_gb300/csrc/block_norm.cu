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
// the team is a CTA.
//
// Sums of squares run over centred values in fp32: for the centred norm a first mean is taken
// off, then what the centred values still sum to (its rounding error), so that a mean far
// larger than the spread costs no digits.  Squares that leave fp32's range (beyond 1e37, or
// below 1e-30 where eps does not cover them) are summed again with the values scaled by a power
// of two.
template <int E, bool VEC, bool CTA>
struct Team {
    float2* red;         // CTA teams: two buffers of 32 pairs, used in turn
    int lanes, turn = 0;

    // The team's lanes: teams of one warp may go different ways.
    __device__ unsigned mask() const {
        return CTA || lanes == 32 ? ~0u : ((1u << lanes) - 1) << (threadIdx.x & 31 & ~(lanes - 1));
    }

    __device__ float2 sum(float2 v) {
        if (CTA) {
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                v.x += __shfl_xor_sync(~0u, v.x, o);
                v.y += __shfl_xor_sync(~0u, v.y, o);
            }
            return across(v, [](float2 a, float2 b) { return make_float2(a.x + b.x, a.y + b.y); });
        }
        const unsigned m = mask();
        for (int o = lanes >> 1; o; o >>= 1) {
            v.x += __shfl_xor_sync(m, v.x, o);
            v.y += __shfl_xor_sync(m, v.y, o);
        }
        return v;
    }
    __device__ float sum(float v) { return sum(make_float2(v, 0.f)).x; }
    __device__ float max(float v) {
        const unsigned m = mask();
        for (int o = CTA ? 16 : lanes >> 1; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(m, v, o));
        if (!CTA) return v;
        return across(make_float2(v, 0.f), [](float2 a, float2 b) { return make_float2(fmaxf(a.x, b.x), 0.f); }).x;
    }
    // Join the warps' values of a CTA, the same way in every warp.  The two buffers take turns:
    // whoever writes one has passed the barrier after its last readers' reads.
    template <class F>
    __device__ float2 across(float2 v, F join) {
        float2* buf = red + 32 * (turn ^= 1);
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        if (lane == 0) buf[threadIdx.x >> 5] = v;
        __syncthreads();
        v = lane < warps ? buf[lane] : make_float2(0.f, 0.f);
#pragma unroll
        for (int o = 16; o; o >>= 1)
            v = join(v, make_float2(__shfl_xor_sync(~0u, v.x, o), __shfl_xor_sync(~0u, v.y, o)));
        return v;
    }
};

// Elements that a thread of a team of `size` holds: groups of 8 consecutive ones, or single ones
// where rows or weights are not aligned for groups.
template <int E, bool VEC, class F>
__device__ __forceinline__ void each_group(int rank, int size, F f) {
#pragma unroll
    for (int i = 0; i < E / 8; ++i) {
        if (VEC)
            f(i, (rank + i * size) * 8, 1);
        else
            f(i, rank + i * 8 * size, size);
    }
}

// Eight values, `step` apart from element e on; zeros from `dim` on.
template <bool VEC>
__device__ __forceinline__ void load8(const void* p, bool f32, int e, int step, int dim, float* v) {
    if (VEC) {
        if (e < dim) {
            row_load8(p, f32, e, v);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = 0.f;
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = e + k * step < dim ? row_load1(p, f32, e + k * step) : 0.f;
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(void* p, bool f32, int e, int step, int dim, const float* v) {
    if (VEC) {
        if (e < dim) row_store8(p, f32, e, v);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (e + k * step < dim) row_store1(p, f32, e + k * step, v[k]);
    }
}

// v = N(v): the elements of one row, zeros past its end.
template <int E, bool VEC, bool CTA>
__device__ __forceinline__ void normalise(float (&v)[E], const NormSide& n, Team<E, VEC, CTA>& team, int rank, int size,
                                          int dim) {
    const float inv_dim = 1.f / dim;
    float ss = 0.f;
    if (n.kind == DL_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s = fmaf(v[i], inv_dim, s);
        const float mean = team.sum(s);
        float2 t = {0.f, 0.f};
        each_group<E, VEC>(rank, size, [&](int i, int e, int step) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float& x = v[8 * i + k];
                x = e + k * step < dim ? x - mean : 0.f;
                t.x = fmaf(x, inv_dim, t.x);
                t.y = fmaf(x, x, t.y);
            }
        });
        t = team.sum(t);
        const float rest = t.x;
        ss = t.y <= 1e37f ? fmaxf(fmaf(-dim * rest, rest, t.y), 0.f) : t.y;
        each_group<E, VEC>(rank, size, [&](int i, int e, int step) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (e + k * step < dim) v[8 * i + k] -= rest;
        });
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) ss = fmaf(v[i], v[i], ss);
        ss = team.sum(ss);
    }
    float up = 1.f, inv = 1.f / sqrtf(fmaf(ss, inv_dim, n.eps));
    if (ss > 1e37f || (ss < 1e-30f && n.eps < 1e-30f)) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) m = fmaxf(m, fabsf(v[i]));
        m = team.max(m);
        if (m > 0.f && m <= 3.4028235e38f) {
            up = ldexpf(1.f, -max(ilogbf(m), -100));
            ss = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) ss = fmaf(v[i] * up, v[i] * up, ss);
            ss = team.sum(ss);
            inv = 1.f / sqrtf(fmaf(ss, inv_dim, n.eps * up * up));
        }
    }
    each_group<E, VEC>(rank, size, [&](int i, int e, int step) {
        float w[8], b[8];
        if (n.weight) load8<VEC>(n.weight, n.f32, e, step, dim, w);
        if (n.bias) load8<VEC>(n.bias, n.f32, e, step, dim, b);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float x = v[8 * i + k] * up * inv;
            if (n.weight) x *= w[k] + n.offset;
            v[8 * i + k] = n.bias ? x + b[k] : x;
        }
    });
}

template <int E, bool VEC, bool CTA>
__global__ void __launch_bounds__(1024) block_norm_kernel(const __grid_constant__ BlockNormParams p) {
    __shared__ float2 red[CTA ? 64 : 1];
    Team<E, VEC, CTA> team{red, p.lanes};
    const int size = CTA ? blockDim.x : p.lanes, rank = CTA ? threadIdx.x : threadIdx.x & (p.lanes - 1);
    const long long row = CTA ? blockIdx.x : ((long long)blockIdx.x * blockDim.x + threadIdx.x) / p.lanes;
    const bool mine = row < p.rows;         // a warp's teams stay together for their shuffles
    const int dim = mine ? p.dim : 0;
    griddep_wait();
    griddep_launch_dependents();
    const long long at = mine ? row : 0;
    float v[E], h[E];
    const char *py = row_ptr(p.y, at), *ph = row_ptr(p.h, at);
    each_group<E, VEC>(rank, size, [&](int i, int e, int step) {
        if (p.y.ptr) load8<VEC>(py, p.y.f32, e, step, dim, v + 8 * i);
        if (p.h.ptr) load8<VEC>(ph, p.h.f32, e, step, dim, h + 8 * i);
    });
    if (p.y.ptr) {
        if (p.post.kind != DL_NORM_NONE) normalise<E, VEC, CTA>(v, p.post, team, rank, size, dim);
        const float row_gate = p.gate_kind == DL_GATE_ROW ? row_load1(row_ptr(p.gate, at), p.gate.f32, 0) : 1.f;
        const char* pg = p.gate_kind == DL_GATE_FULL ? row_ptr(p.gate, at) : static_cast<const char*>(p.gate.ptr);
        each_group<E, VEC>(rank, size, [&](int i, int e, int step) {
            float g[8];
            if (p.gate_kind >= DL_GATE_CHANNEL) load8<VEC>(pg, p.gate.f32, e, step, dim, g);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float& x = v[8 * i + k];
                if (p.gate_kind != DL_GATE_NONE) {
                    const float t = p.gate_kind == DL_GATE_ROW ? row_gate : g[k];
                    x *= p.sigmoid ? 1.f / (1.f + expf(-t)) : t;
                }
                x *= p.scale;
                if (p.h.ptr) x = fmaf(p.h_scale, h[8 * i + k], x);
                if (e + k * step >= dim) x = 0.f;      // a gate of infinity times an absent element
            }
        });
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = p.h_scale * h[i];
    }
    if (p.r.ptr) {
        char* pr = row_ptr(p.r, at);
        each_group<E, VEC>(rank, size, [&](int i, int e, int step) { store8<VEC>(pr, p.r.f32, e, step, dim, v + 8 * i); });
    }
    if (p.x.ptr) {
        if (p.pre.kind != DL_NORM_NONE) normalise<E, VEC, CTA>(v, p.pre, team, rank, size, dim);
        char* px = row_ptr(p.x, at);
        each_group<E, VEC>(rank, size, [&](int i, int e, int step) { store8<VEC>(px, p.x.f32, e, step, dim, v + 8 * i); });
    }
}

constexpr int kMaxDim = 32768;

template <int E, bool VEC, bool CTA>
cudaError_t launch_norm(const BlockNormParams& p, long long grid, int threads, cudaStream_t stream) {
    return launch_dependent(block_norm_kernel<E, VEC, CTA>, dim3((unsigned)grid), dim3(threads), 0, stream, p);
}

template <bool VEC>
cudaError_t launch_norm_rows(BlockNormParams& p, int sm_count, cudaStream_t stream) {
    const int groups = (p.dim + 7) / 8;
    if (groups <= 128) {                    // teams inside a warp, at most 32 elements a thread
        int lanes = 8;
        while (lanes < 32 && lanes * 4 < groups) lanes *= 2;
        const int per = (groups + lanes - 1) / lanes, threads = 128;
        const long long grid = ((long long)p.rows * lanes + threads - 1) / threads;
        p.lanes = lanes;
        if (per <= 1) return launch_norm<8, VEC, false>(p, grid, threads, stream);
        if (per <= 2) return launch_norm<16, VEC, false>(p, grid, threads, stream);
        return launch_norm<32, VEC, false>(p, grid, threads, stream);
    }
    // A CTA each: one group a thread where there are few rows, so that a row is loaded at once, two
    // where there are many
    const int want = p.rows <= 2 * sm_count ? 1 : 2;
    int per = want;
    while ((groups + per - 1) / per > 1024) per *= 2;
    const int threads = ((groups + per - 1) / per + 31) / 32 * 32;
    if (per == 1) return launch_norm<8, VEC, true>(p, p.rows, threads, stream);
    if (per == 2) return launch_norm<16, VEC, true>(p, p.rows, threads, stream);
    return launch_norm<32, VEC, true>(p, p.rows, threads, stream);
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
    const cudaError_t e = vec ? launch_norm_rows<true>(p, dev.sm_count, st) : launch_norm_rows<false>(p, dev.sm_count, st);
    if (e != cudaSuccess) return host_fail(DL_ERR_CUDA, "block_norm launch: %s", cudaGetErrorString(e));
    return host_ok();
}
