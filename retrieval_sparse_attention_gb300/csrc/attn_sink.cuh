// attn_sink.cuh -- what the kernels of the windowed attention with sinks share:
// the paged-cache bookkeeping of one sequence and of one cached token.
#pragma once

#include <stdint.h>

#include "common.cuh"
#include "gca.h"

namespace gca {

// Device arrays of a paged call (all null for dense sequences).
struct PagedArgs {
    const int32_t* cu_q;      // [B + 1]
    const int32_t* kv_len;    // [B]
    const int32_t* table;     // [B, width]
    int T, max_q;
    int page_log2, n_pages, width;
};

// One sequence: its new tokens are rows row0 .. row0 + n - 1 of the token tensors, at
// positions pos0 .. pos0 + n - 1 (pos0 < 0: the first ones see nothing).
struct SeqInfo {
    int row0, n, pos0;
};

// Sequence b of a paged call; n = 0 and GCA_ERR_DEVICE_INDEX for entries that contradict
// each other, so nothing out of range is ever addressed.
__device__ __forceinline__ SeqInfo paged_seq(const PagedArgs& a, int b, int* status) {
    const int c0 = a.cu_q[b], c1 = a.cu_q[b + 1], kv = a.kv_len[b];
    SeqInfo s{c0, c1 - c0, kv - (c1 - c0)};
    if (c0 < 0 || c1 < c0 || c1 > a.T || c1 - c0 > a.max_q || kv < 0 ||
        kv > (a.width << a.page_log2)) {
        set_status(status, GCA_ERR_DEVICE_INDEX);
        s = SeqInfo{0, 0, 0};
    }
    return s;
}

}  // namespace gca
