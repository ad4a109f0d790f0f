// Instantiation of the attention kernels for one head dimension.
#pragma once

#include <atomic>

#include "dl_kernel.cuh"
#include "kv_attention.cuh"

namespace dl {

// Tensor memory that a linear of the tensor-memory family finds taken.  It lets the next launch start
// before it allocates, and an attention CTA allocates before it waits for the linear: were there
// too few columns left, each would wait for the other.  As many CTAs of C as fit into an SM's
// shared memory beside a linear's smallest CTA (two stages) leave the columns that it takes.
template <class C, int MT>
constexpr bool leaves_tmem_to_linear() {
    constexpr int sm_bytes = 228 * 1024, reserved = 1024;           // of shared memory, per CTA
    constexpr int linear = smem_layout(kFP8, kTC, MT, 2).total + 1024 + reserved;
    constexpr int beside = (sm_bytes - linear) / ((int)C::kSmem + reserved);
    return (beside < C::kCtas ? beside : C::kCtas) * C::kTmem + TcShape<MT>::cols <= 512;
}

template <class C>
cudaError_t launch_attention_instance(const AttnLaunch& a) {
    static_assert(leaves_tmem_to_linear<C, 8>() && leaves_tmem_to_linear<C, 16>(), "columns for a linear on the same SM");
    static std::atomic<bool> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev].load()) {
        e = cudaFuncSetAttribute(attention_kernel<C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::kSmem);
        if (e != cudaSuccess) return e;
        ready[dev].store(true);
    }
    // Both kernels may start while the one before drains; they wait for it
    // before they touch memory.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.grid);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    cfg.stream = a.stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, attention_kernel<C>, a.tk, a.tv, a.p)) != cudaSuccess) return e;
    const int rows = a.p.tile_tokens * a.p.group;
    const bool wide = (long long)a.p.s.batch * a.p.row_tiles * a.p.kv_heads * 8 <= a.grid;
    cfg.gridDim = wide ? dim3((a.grid + 3) / 4, rows) : dim3(a.grid, (rows + 3) / 4);
    cfg.blockDim = dim3(128);
    cfg.dynamicSmemBytes = 0;
    return wide ? cudaLaunchKernelEx(&cfg, attention_combine_kernel<C::D, 4, 4>, a.p, C::RP, a.grid)
                : cudaLaunchKernelEx(&cfg, attention_combine_kernel<C::D, 1, 1>, a.p, C::RP, a.grid);
}

template <int D>
cudaError_t launch_attention_dim(int rp, const AttnLaunch& a) {
    switch (rp) {
        case 8: return launch_attention_instance<AttnShape<D, 8>>(a);
        case 16: return launch_attention_instance<AttnShape<D, 16>>(a);
        case 32: return launch_attention_instance<AttnShape<D, 32>>(a);
        case 48: return launch_attention_instance<AttnShape<D, 48>>(a);
        case 64: return launch_attention_instance<AttnShape<D, 64>>(a);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace dl
