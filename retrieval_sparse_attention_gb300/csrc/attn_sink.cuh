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

// ---------------------------------------------------------------------------
// Units of the forward and of the query-major gradients: the query rows of one
// key head are packed into 128-row tiles, token-major (row r of a tile is token
// r / G, query head r % G of the group), so a key tile is read once for the
// whole group; keys come in tiles of 128.
// ---------------------------------------------------------------------------
struct SinkSched {
    int B, L;            // sequences; dense: their length
    int H, Hkv, G;       // G = H / Hkv
    int W, ns;
    int TM;              // tokens per query tile: min(128 / G, longest sequence)
    int nMT;             // query tiles of the longest sequence
    int paged;
    PagedArgs p;
};

__device__ __forceinline__ SeqInfo sink_seq(const SinkSched& a, int b, int* status) {
    if (!a.paged) return SeqInfo{b * a.L, a.L, 0};
    return paged_seq(a.p, b, status);
}

// The key tiles that query tile mt of a sequence sees: nsk tiles of sinks from tile 0
// on, then tiles k0 .. of the window.  nt = 0: no such query tile.  A query tile
// that sees no key at all (negative positions) has one, fully masked.
struct KeyTiles {
    int p0, p1;          // positions of its first and last token
    int k0, nsk, nt;
    __device__ __forceinline__ int tile(int j) const { return j < nsk ? j : k0 + j - nsk; }
};
__device__ __forceinline__ KeyTiles key_tiles(const SinkSched& a, const SeqInfo& s, int mt) {
    KeyTiles k;
    const int t0 = mt * a.TM;
    k.p0 = s.pos0 + t0;
    k.p1 = s.pos0 + min(s.n, t0 + a.TM) - 1;
    const int lo = max(0, k.p0 - a.W + 1);
    k.k0 = lo >> 7;
    k.nsk = min((a.ns + 127) >> 7, k.k0);
    k.nt = t0 >= s.n ? 0 : k.nsk + (max(k.p1, 0) >> 7) - k.k0 + 1;
    if (k.p1 < 0) { k.k0 = 0; k.nsk = 0; k.nt = t0 >= s.n ? 0 : 1; }
    return k;
}

// Position in the stream of all (sequence, query tile, key head, key tile), in that
// order: where a worker's share of the stream begins, and how long it is.
struct StreamPos {
    int b, mt, h, j;
    int left;
};

}  // namespace gca
