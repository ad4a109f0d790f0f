// Host-side services that dl_api.cu shares with the other entry points'
// translation units (internal, not part of the ABI).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "dl_linear.h"

namespace dl {

// Set the calling thread's error message and return `s`.
dl_status host_fail(dl_status s, const char* fmt, ...);
// Clear the message and return DL_OK.
dl_status host_ok();

struct HostDevice {
    int sm_count;
    unsigned* err_word;                   // the device error word
    unsigned long long wait_limit_ns;     // of every device-side wait
    int withhold_stage;                   // dl_set_wait_test's (0: none)
};
// The current device's (cached) description.
dl_status host_device(HostDevice& out);

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
dl_status host_encode(EncodeTiled& fn);

// The argument checks that the cached-attention entry points share.
dl_status check_cache(const dl_kv_cache* c);
dl_status check_sequences(const int* block_table, int table_cols, const int* seq_lens,
                          const int* q_start, int batch, int tokens, int max_q);

}  // namespace dl
