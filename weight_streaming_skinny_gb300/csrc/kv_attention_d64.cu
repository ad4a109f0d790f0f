// Attention kernels for heads of 64.
#include "kv_attention_launch.cuh"

namespace dl {
cudaError_t launch_attention_d64(int rp, const AttnLaunch& a) { return launch_attention_dim<64>(rp, a); }
}  // namespace dl
