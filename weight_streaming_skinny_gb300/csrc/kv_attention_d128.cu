// Attention kernels for heads of 128.
#include "kv_attention_launch.cuh"

namespace dl {
cudaError_t launch_attention_d128(int rp, const AttnLaunch& a) { return launch_attention_dim<128>(rp, a); }
}  // namespace dl
