// attn_sink.cuh -- what the kernels of the windowed attention with sinks share: a paged
// call's sequences, the units of work and their equal shares, bounded waits, the way of
// an accumulator's rows to global memory, and their launches.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "common.cuh"
#include "gca.h"
#include "kernels.h"
#include "tc_common.cuh"
#include "tc_ptx.cuh"

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

// Sum over i = 1 .. n of min(cap, step i + 1): the tiles of a row's n query tiles, of which the i-th
// ends in tile step i at most and sees no more than cap.
constexpr double kMaxSteps = 2.1e9;              // a stream's end plus one share (1/152 of it) stays below 2^31
inline double causal_sum(double n, double step, double cap) {
    const double m = std::min(n, std::max(0.0, std::floor((cap - 1) / step)));
    return step * m * (m + 1) / 2 + m + (n - m) * cap;
}

// The first of this thread's sequences whose cu_q decreases, or B.  Asked at the kernel's start and
// looked at behind its set-up, with kv_len on its way into L1 too: free for 48 and 64 sequences, where a
// check at once took 0.5 and 1 us of 52 and 38; 0.3 us of 13 for 3 sequences.
template <int THREADS>
__device__ __forceinline__ int first_decrease(const PagedArgs& a, int B) {
    int first = B;
#pragma unroll 1
    for (int b = B > 1 ? threadIdx.x : B; b < B; b += THREADS) {
        asm volatile("prefetch.global.L1 [%0];" ::"l"(a.kv_len + b));
        if (a.cu_q[b + 1] < a.cu_q[b]) first = min(first, b);
    }
    return first;
}

// The sequences before the first whose cu_q decreases: those behind it could claim their rows, and the
// stream could be far longer than the host's bound on it.  All threads of the CTA; 1 where there are
// none (paged_seq leaves out the first itself).
__device__ __forceinline__ int ascending_seqs(int first, int B, int* smem, int* status) {
    if (B > 1 && __syncthreads_or(first < B)) {
        if (threadIdx.x == 0) {
            *smem = B;
            set_status(status, GCA_ERR_DEVICE_INDEX);
        }
        __syncthreads();
        atomicMin(smem, first);
        __syncthreads();
        B = max(*smem, 1);
        __syncthreads();
    }
    return B;
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
    PagedArgs p;
};

template <bool PAGED>
__device__ __forceinline__ SeqInfo sink_seq(const SinkSched& a, int b, int* status) {
    if (!PAGED) return SeqInfo{b * a.L, a.L, 0};
    return paged_seq(a.p, b, status);
}

// The key tiles that query tile mt of a sequence sees: nsk tiles of sinks from tile 0
// on, then tiles k0 .. of the window.  nt = 0: no such query tile.  A query tile
// that sees no key at all (negative positions) has one, fully masked.
struct KeyTiles {
    int p0, p1;          // positions of its first and last token
    int k0, nsk, nt;
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
    int wid;             // the worker's number, in the order of the stream
    int qb = -1;         // paged: the sequence that q describes (kept from part to part)
    SeqInfo q = {0, 0, 0};
};

// The shares of this CTA (SHARES workers, neighbours in the stream; where there are
// fewer steps than CTAs, each CTA has one worker with a share at most) in a stream of
// equally long steps: sequence b has entries i < n, entry i takes count(seq(b), i)
// steps for each of `heads` heads, in the order (b, head, i, step): a worker follows one
// head along the sequence and finds most of an entry's tiles in the L2 cache, where its
// last entries brought them.  Every worker gets total / workers steps, rounded up.  All
// THREADS threads of the CTA take part; ends with __syncthreads.  The host bounds the
// total below 2^31.  whole: cuts move to the next entry's first step, which may be one that
// the sequence does not have (the walk passes over it).
template <int THREADS, int SHARES, class Seq, class Count>
__device__ __forceinline__ void find_shares(int B, int n, int heads, bool whole, int* wsum, int (*found)[3],
                                            StreamPos* pos, Seq seq, Count count) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int E = B * n;                            // entries, a run of them for each thread
    const int per = (E + THREADS - 1) / THREADS;
    const int e0 = min(E, tid * per), e1 = min(E, e0 + per);
    const int b0 = e0 / n, i0 = e0 - b0 * n;
    const auto q0 = seq(min(b0, B - 1));
    auto each = [&](auto f) {                       // f(sequence, entry, steps) for this thread's entries
        int b = b0, i = i0;
        auto q = q0;
#pragma unroll 1
        for (int e = e0; e < e1; ++e) {
            if (e > e0 && i == 0) q = seq(b);
            f(b, i, count(q, i));
            if (++i == n) { i = 0; ++b; }
        }
    };
    int mine = 0;
    each([&](int, int, int c) { mine += c; });
    int inc = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) wsum[warp] = inc;
    if (tid < SHARES) pos[tid] = StreamPos{0, 0, 0, 0, 0, 0, -1, {0, 0, 0}};
    __syncthreads();
    int base = inc - mine, row = 0;                 // steps of one head: before this thread's entries, in all
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += wsum[w];
        row += wsum[w];
    }
    const int total = row * heads, workers = SHARES * gridDim.x;
    const int quota = (total + workers - 1) / workers;
    auto wid = [&](int w) {
        return total <= static_cast<int>(gridDim.x) ? static_cast<int>(blockIdx.x + w * gridDim.x)
                                                    : static_cast<int>(blockIdx.x) * SHARES + w;
    };
    // worker w's share: its first step (k = 2 w) and its end, one past its last step (2 w + 1)
    auto cut = [&](int k) {
        const int from = wid(k >> 1) * quota;
        return from >= total ? total : (k & 1) ? min(total, from + quota) : from;
    };
    if (tid < SHARES) {                             // a share that ends with the stream
        const int from = cut(2 * tid);
        pos[tid].wid = wid(tid);
        if (from < total && from + quota >= total) atomicAdd(&pos[tid].left, total - from);
    }
    if (n > 1) {
        // the sequence of each cut: where its steps begin and end
        if (tid < 2 * SHARES) {
            found[tid][0] = 0;
            found[tid][1] = row;
        }
        __syncthreads();
        int at = base;
        each([&](int, int i, int c) {
            if (i == 0)
#pragma unroll 1
                for (int k = 0; k < 2 * SHARES; ++k) {
                    if (at * heads <= cut(k)) atomicMax(&found[k][0], at);
                    else atomicMin(&found[k][1], at);
                }
            at += c;
        });
        __syncthreads();
    }
    // which entry holds a cut
    int at = base;
    each([&](int b, int i, int c) {
#pragma unroll 1
        for (int k = 0; k < 2 * SHARES; ++k) {
            const int x = cut(k), first = n > 1 ? found[k][0] : at, len = n > 1 ? found[k][1] - first : c;
            const int r = x - first * heads;
            if (x == total || c == 0 || r < 0 || r >= len * heads) continue;
            const int h = r / len, j = first + r - h * len - at;
            if (j < 0 || j >= c || h >= heads) continue;
            const int w = k >> 1, skip = whole && j > 0 ? c - j : 0;
            if (k & 1) {
                atomicAdd(&pos[w].left, x - wid(w) * quota + skip);
            } else {
                atomicAdd(&pos[w].left, -skip);
                pos[w].b = b; pos[w].h = h; pos[w].mt = i + (skip > 0); pos[w].j = skip ? 0 : j;
            }
        }
        at += c;
    });
    __syncthreads();
}

// The same for dense sequences, which all have the same entries: those of one (sequence, head)
// are summed up, and the cuts divide by their total.
template <int THREADS, int SHARES, class Count>
__device__ __forceinline__ void find_shares_dense(int B, int n, int heads, bool whole, int* wsum, StreamPos* pos,
                                                  Count count) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int per = (n + THREADS - 1) / THREADS;
    const int e0 = min(n, tid * per), e1 = min(n, e0 + per);
    int mine = 0;
#pragma unroll 1
    for (int e = e0; e < e1; ++e) mine += count(e);
    int inc = mine;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
    }
    if (lane == 31) wsum[warp] = inc;
    if (tid < SHARES) pos[tid] = StreamPos{0, 0, 0, 0, 0, 0, -1, {0, 0, 0}};
    __syncthreads();
    int base = inc - mine, row = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) base += wsum[w];
        row += wsum[w];
    }
    const int total = row * heads * B, workers = SHARES * gridDim.x;
    const int quota = (total + workers - 1) / workers;
#pragma unroll 1
    for (int k = 0; k < 2 * SHARES; ++k) {
        // worker w's share: its first step (k even) and its end, one past its last step
        const int w = k >> 1;
        const int wid = total <= static_cast<int>(gridDim.x) ? blockIdx.x + w * gridDim.x : blockIdx.x * SHARES + w;
        if (tid == 0 && (k & 1)) pos[w].wid = wid;
        const int from = wid * quota;
        if (from >= total) continue;
        const int x = (k & 1) ? min(total, from + quota) : from;
        int bh = x / row;
        const int r = x - bh * row;
        int at = base;
#pragma unroll 1
        for (int e = e0; e < e1; ++e) {
            const int c = count(e);
            if (r >= at && r < at + c) {
                const int skip = whole && r > at ? at + c - r : 0;
                if (k & 1) {
                    atomicAdd(&pos[w].left, x - from + skip);
                } else {
                    atomicAdd(&pos[w].left, -skip);
                    int i = e;
                    if (skip && ++i == n) { i = 0; ++bh; }
                    pos[w].b = bh / heads;
                    pos[w].h = bh % heads;
                    pos[w].mt = i;
                    pos[w].j = skip ? 0 : r - at;
                }
            }
            at += c;
        }
    }
    __syncthreads();
}

__device__ __forceinline__ uint32_t full_par(int k) { return static_cast<uint32_t>(k) & 1u; }
__device__ __forceinline__ uint32_t empty_par(int k) { return (static_cast<uint32_t>(k) & 1u) ^ 1u; }

// The lowest n bits (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Bounded wait in as little code as it takes (the kernels' hot code has to stay in the
// instruction cache): each try may suspend the thread for up to 20 us, and after about
// 2 s of tries the wait gives up; its role then ends early and notes it for the CTA's
// report, and the CTA's other roles run out of their waits.
__device__ __forceinline__ bool wait_ctrl(uint64_t* bar, uint32_t parity) {
    const uint32_t addr = tc::smem_u32(bar);
#pragma unroll 1
    for (int n = 0; n < 100000; ++n) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(addr), "r"(parity), "r"(20000u)
            : "memory");
        if (ok) return true;
    }
    return false;
}
// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
// Bounded wait for work in flight at the end.
__device__ __forceinline__ void wait_copy(uint64_t* bar, uint32_t parity) { wait_ctrl(bar, parity); }

// 32 fp32 columns of the warp's 32 rows of an accumulator (a row a lane), times this lane's
// `scale`, as bf16 pairs in the order that store_rows32 takes: four lanes have 64
// consecutive bytes of a row, eight rows at a time.  The exchange between lanes goes
// through the accumulator's own columns, written by rows and read back four lanes a row.
// (With a row per lane the 32 lanes of a store touch 32 lines, and a tile's stores cost
// as much as half a key tile; with shuffles in place of tensor memory the forward took
// 0.333 instead of 0.325 ms at B = 8 x 16K, W = 512.)
__device__ __forceinline__ void load_rows32(uint32_t taddr, float scale, uint32_t (&q)[16]) {
    uint32_t r[32], pk[16];
    tc::tmem_ld_32x32b_x32(taddr, r);
    tc::tmem_wait_ld();
    const uint64_t s2 = tcx::f2_pack(scale, scale);
#pragma unroll
    for (int u = 0; u < 16; ++u)                        // pair u: column 4 (u % 4) + u / 4
        pk[4 * (u & 3) + (u >> 2)] = tcx::pack_bf16x2(
            tcx::fmul2(tcx::f2_pack(__uint_as_float(r[2 * u]), __uint_as_float(r[2 * u + 1])), s2));
    tc::tmem_st_32x32b_x16(taddr, pk);
    tc::tmem_wait_st();
#pragma unroll
    for (int h = 0; h < 2; ++h) {                       // rows 16 h ..
        uint32_t x[8];
        tc::tmem_ld_16x128b_x4(taddr + (h << 20), x);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) q[8 * h + 4 * (i & 1) + (i >> 1)] = x[i];
    }
}

// Those to global memory: this lane's row is row `row` (rows of ld elements; row < 0: none)
// from out on.
__device__ __forceinline__ void store_rows32(const uint32_t* q, __nv_bfloat16* out, int ld, int row) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int rk = __shfl_sync(0xffffffffu, row, 8 * k + (lane >> 2));
        if (rk >= 0)
            *reinterpret_cast<uint4*>(out + (size_t)rk * ld + 8 * (lane & 3)) =
                make_uint4(q[4 * k], q[4 * k + 1], q[4 * k + 2], q[4 * k + 3]);
    }
}

// Programmatic dependent launch within a call: a kernel lets its successor's CTAs start
// as its own leave, and the successor waits for its completion before it reads or
// writes anything.
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P, class... A>
inline cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<A&&>(args)...);
}

// What a launch needs of the current device and context, looked up once for each: the
// kernels' attributes are set in a context, so a new one (after cudaDeviceReset, for
// instance) sets them again.
struct LaunchSetup {
    std::mutex mu;
    unsigned long long ctx = 0;
    int dev = -1, sms = 0;
    // Runs `set` (cudaError_t()) unless it has run for the current device and context.
    template <class F>
    cudaError_t once(F set, int* sms_out) {
        int d = 0;
        cudaError_t e = cudaGetDevice(&d);
        if (e != cudaSuccess) return e;
        std::lock_guard<std::mutex> lock(mu);
        const unsigned long long c = current_context_id();
        if (c == 0 || c != ctx || d != dev) {
            if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d)) != cudaSuccess) return e;
            if ((e = set()) != cudaSuccess) return e;
            ctx = current_context_id();
            dev = d;
        }
        *sms_out = sms;
        return cudaSuccess;
    }
};

// Parts of an item that begins in worker w's share and goes on in the next ones: w's own
// and those of the workers behind it up to the first whose head is not a middle part.
__device__ __forceinline__ int parts_of(const int* head, int w, int workers) {
    const int lane = threadIdx.x & 31;
    int n = 1;
    for (int at = w + 1; at < workers; at += 32) {
        const int h = at + lane < workers ? head[at + lane] : 0;
        const unsigned ends = __ballot_sync(0xffffffffu, h != 2);
        if (ends) return n + __ffs(ends);
        n += 32;
    }
    return n;
}

}  // namespace gca
