// The paged 8-bit cache as the kernels see it, and where a call's sequences lie.
#pragma once

#include <stdint.h>

#include "dl_device.cuh"
#include "dl_linear.h"

namespace dl {

// A call's sequences (device arrays).
struct Sequences {
    const int* block_table;    // [batch][table_cols]
    const int* seq_lens;       // [batch]
    const int* q_start;        // [batch + 1]
    int table_cols, batch, tokens, max_q;
};

// Sequence b: its first row, its new tokens (all of them, and those worked on)
// and its cached tokens, with out-of-range values contained.
struct SequenceView {
    int row0, n, n_work, len;
};

__device__ __forceinline__ SequenceView sequence_view(const Sequences& s, int b, int page_size) {
    SequenceView r;
    r.row0 = min(max(s.q_start[b], 0), s.tokens);
    r.n = min(max(s.q_start[b + 1], r.row0), s.tokens) - r.row0;
    r.n_work = min(r.n, s.max_q);
    const long long room = (long long)s.table_cols * page_size;
    const int len = max(s.seq_lens[b], 0);
    r.len = (long long)len > room ? (int)room : len;
    return r;
}

}  // namespace dl
