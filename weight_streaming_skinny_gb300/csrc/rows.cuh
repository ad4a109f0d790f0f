// Rows of bf16 or fp32 elements that the kernels between the linears read and write, and the host
// checks of them.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "dl_device.cuh"
#include "dl_host.h"

namespace dl {

struct Rows {
    char* ptr;
    long long stride;      // bytes from one row to the next
    bool f32;
};

__device__ __forceinline__ char* row_ptr(const Rows& r, long long i) { return r.ptr + i * r.stride; }

__device__ __forceinline__ float row_load1(const void* p, bool f32, int e) {
    return f32 ? static_cast<const float*>(p)[e] : bf16_bits_to_f32(static_cast<const uint16_t*>(p)[e]);
}
__device__ __forceinline__ void row_store1(void* p, bool f32, int e, float v) {
    if (f32)
        static_cast<float*>(p)[e] = v;
    else
        static_cast<uint16_t*>(p)[e] = f32_to_bf16_rne(v);
}
__device__ __forceinline__ void bf16x2_to_f32(uint32_t two, float& a, float& b) {
    a = __uint_as_float(two << 16);
    b = __uint_as_float(two & 0xffff0000u);
}
__device__ __forceinline__ uint32_t f32x2_to_bf16x2(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Eight consecutive elements from e on, 16-byte aligned.
__device__ __forceinline__ void row_load8(const void* p, bool f32, int e, float* v) {
    if (f32) {
        const uint4 a = ldg128(static_cast<const float*>(p) + e), b = ldg128(static_cast<const float*>(p) + e + 4);
        v[0] = __uint_as_float(a.x); v[1] = __uint_as_float(a.y); v[2] = __uint_as_float(a.z); v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x); v[5] = __uint_as_float(b.y); v[6] = __uint_as_float(b.z); v[7] = __uint_as_float(b.w);
    } else {
        const uint4 a = ldg128(static_cast<const uint16_t*>(p) + e);
        bf16x2_to_f32(a.x, v[0], v[1]);
        bf16x2_to_f32(a.y, v[2], v[3]);
        bf16x2_to_f32(a.z, v[4], v[5]);
        bf16x2_to_f32(a.w, v[6], v[7]);
    }
}
__device__ __forceinline__ void row_store8(void* p, bool f32, int e, const float* v) {
    if (f32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + e);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + e) =
            make_uint4(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                       f32x2_to_bf16x2(v[6], v[7]));
    }
}

// Sums of counts over the threads up to each one of a CTA of 1024; `total`: over all.  Calls take turns with the two halves
// of `warp_sum`, so one barrier is enough: who writes a half has passed the barrier after its last reads.
struct Scan {
    int (*warp_sum)[32];     // [2][32] shared
    int half = 0;

    __device__ __forceinline__ int operator()(int v, int& total) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(~0u, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) warp_sum[half][warp] = v;
        __syncthreads();
        const int mine = warp_sum[half][lane];
        half ^= 1;
        total = (int)__reduce_add_sync(~0u, (unsigned)mine);
        return v + (int)__reduce_add_sync(~0u, lane < warp ? (unsigned)mine : 0u);
    }
};

// ---------------------------------------------------------------- host

// The checked form of an argument (NULL, or without data: none).
inline dl_status check_rows(const dl_rows* r, const char* name, long long rows, long long dim, Rows& out) {
    out = Rows{};
    if (!r || !r->data) return DL_OK;
    if (r->dtype != DL_ROWS_BF16 && r->dtype != DL_ROWS_F32)
        return host_fail(DL_ERR_INVALID_ARG, "%s: unknown dtype %d", name, r->dtype);
    const bool f32 = r->dtype == DL_ROWS_F32;
    const long long el = f32 ? 4 : 2;
    if ((uintptr_t)r->data & (el - 1)) return host_fail(DL_ERR_MISALIGNED, "%s must be aligned to its type", name);
    if (rows > 1 && (r->stride < dim || r->stride > (1LL << 40)))
        return host_fail(DL_ERR_INVALID_ARG, "%s: rows are %lld elements apart, a row has %lld", name, r->stride, dim);
    out = Rows{static_cast<char*>(r->data), rows > 1 ? r->stride * el : dim * el, f32};
    return DL_OK;
}

inline bool same_rows(const Rows& a, const Rows& b) { return a.ptr == b.ptr && a.stride == b.stride && a.f32 == b.f32; }

inline bool rows_aligned16(const Rows& r, long long rows) {
    return !((uintptr_t)r.ptr & 15) && (rows <= 1 || r.stride % 16 == 0);
}

// Whether two sets of rows may share a byte.  Side by side in one wider row they do not.
inline bool rows_meet(const Rows& a, long long na, long long da, const Rows& b, long long nb, long long db) {
    if (!a.ptr || !b.ptr || na < 1 || nb < 1 || da < 1 || db < 1) return false;
    const long long wa = da * (a.f32 ? 4 : 2), wb = db * (b.f32 ? 4 : 2);
    const uintptr_t pa = (uintptr_t)a.ptr, pb = (uintptr_t)b.ptr;
    const uintptr_t ea = pa + (na - 1) * a.stride + wa, eb = pb + (nb - 1) * b.stride + wb;
    if (ea <= pb || eb <= pa) return false;
    const long long stride = na > 1 ? a.stride : b.stride;
    if ((na > 1 && nb > 1 && a.stride != b.stride) || stride < 1) return true;
    const long long off = (long long)((pb >= pa ? pb - pa : (uintptr_t)stride - (pa - pb) % stride) % stride);
    return !(off >= wa && stride - off >= wb);
}

// Lets a kernel have up to `most` bytes of dynamic shared memory, the most that any of its launches asks for.  Once a
// device and never changed again: the limit is the process's, and a thread that set it to what its own call
// needs would take it from under another thread's launch.
template <auto Kernel>
cudaError_t raise_smem(size_t most) {
    static std::atomic<bool> raised[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (raised[dev].load()) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e == cudaSuccess) raised[dev].store(true);
    return e;
}

// Launch that may start while the kernel before it on the stream still runs (it waits in
// griddep_wait before it touches anything that kernel may write).
template <class... P>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, const P&... p) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p...);
}

}  // namespace dl
