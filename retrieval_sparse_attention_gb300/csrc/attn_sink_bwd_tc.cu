// attn_sink_bwd_tc.cu -- gradients of the windowed attention with sinks on the
// Blackwell tensor cores (bf16, d = 64 or 128).
//
// With p_ts = exp(attn_scale q_t . k_s - lse_t) over V(t) = { s <= t : s > t - W or
// s < ns }, delta_t = dO_t . o_t and ds_ts = attn_scale p_ts (dO_t . v_s - delta_t):
//   dQ_t = sum_s ds_ts k_s,   dK_s = sum_t ds_ts q_t,   dV_s = sum_t p_ts dO_t,
// dK and dV summed over the query heads of the key head.  Four launches:
//   vectors  -lse log2(e) and -attn_scale delta of every (token, query head), in the
//            row order of both passes.
//   pass A   query-major: the forward's 128-row query tiles (tokens x heads of a
//            group); step = 64 keys: S = Q K^T, dP = dO V^T (M = 128, N = 64), ds over
//            the columns of S that have been read, dQ += ds K (A from tensor memory).
//   pass B   key-major: 128 keys of a key head; step = 64 queries of one query head:
//            S^T = K Q^T, dP^T = V dO^T, dK += ds^T Q, dV += P^T dO (A from tensor
//            memory).  The steps of an item are the queries whose window reaches its
//            keys, for each head of the group, and for the items that hold sinks
//            all later queries as well: those items are many times longer than the others.
//   join     adds up the parts of the items that were cut, if any.
// Both passes cut the stream of all their steps into equal shares, one a CTA
// (attn_sink.cuh), so a sink's long item is spread over as many CTAs as it takes
// and short problems fill the machine; parts are fp32 sums in the workspace, added in
// the order of the stream.  No atomics: bitwise reproducible.
// Within a CTA: warp 0 walks the share, writes its parts down as records and loads; one
// thread each issues S, dP, and dQ (pass B: dK and dV); the math warpgroups take
// alternate steps (pass A: one of two each, pass B: two of four, half the queries
// each); a thread owns a query row (pass A) or a key row (pass B), a lane of tensor
// memory, which is the layout of the A operands that it writes.
//
// Roundings: P and ds to bf16, the type of the products' operands (relative 2^-8 at most, as
// the gradients' own rounding, and as many random terms' errors they add up to about as much as
// that: rms 1.7e-3 each); delta takes o as the forward rounded it (rms 5e-4 of a gradient).
// Together 2.4e-3 to 2.7e-3 of a gradient's norm, where its own rounding alone is 1.7e-3.
// Scores, lse, dP, delta and all sums are fp32.  (ds as two bf16 operands would halve the
// excess for a third more products and a quarter more arithmetic in pass A.)
//
// Measured (GB300), B = 8 x 16K, 12 heads of 64, W = 512, 4 sinks: vectors 0.07 ms (6.2
// TB/s), pass A 0.433, pass B 0.615, join 0.01: 1.12 ms in all, 0.99 without sinks and join (the
// plain window's gradients, gca_swa_bwd, 1.22).  2 x 16K, 16/4 heads of 128, W = 1024, 16
// sinks: 0.05, 0.387, 0.515, 0.02: 0.98-1.01 ms.  3 x 1000, 6/2 heads: 38 us.
// What bounds it: pass A and B keep the tensor pipe 31% and 33% busy and the issue
// slots 49% and 51%; the math warps' latency a step and the issuing threads' share of
// the slots pace them (pass B, a clock trace: a step every 1,165 cycles; a math pair's two
// steps take 2 x 1,165 of which its arithmetic 1,310 and its waits and stores the rest; the
// loading thread needs 900 a step, the accumulating products' issuer 780).  A sink's far
// steps cost as much as others (0.10 ms of pass B) although 32 of their 128 key rows at most carry anything; taking them in pass A,
// where sinks have narrow steps, would need its dK and dV sums joined across all CTAs.
#include <math.h>

#include "attn_sink.cuh"
#include "common.cuh"
#include "kernels.h"
#include "tc_common.cuh"
#include "tc_ptx.cuh"
#include "tma_host.h"

namespace gca {
namespace {

using namespace tc;
using tcx::fast_exp2;
using tcx::kLog2e;
using tcx::Ring;

// Pass A: 4 control warps and 2 math warpgroups (with 4, as in pass B, 0.51 instead of 0.47 ms
// at B = 8 x 16K).  Pass B: 4 math warpgroups, two to a step (with 2: 0.78 instead of 0.74 ms).
constexpr int kThreadsA = 384, kThreadsB = 640;
// Pass B's register split: the control roles use 64, and the math warps spill at the launch's 96 (0.635
// instead of 0.62 ms at B = 8 x 16K).
constexpr int kRegsB = 96, kRegsCtrlB = 64, kRegsMathB = 104;
static_assert(128 * kRegsCtrlB + 512 * kRegsMathB <= kThreadsB * kRegsB, "register split exceeds the launch allocation");
constexpr int kMaxCtas = 152;              // one per SM; the workspace is sized for them
constexpr int kParts = 4;                  // part records in flight
constexpr int kSmemMax = 232448;
constexpr uint32_t TMEM_COLS = 512;

struct BwdArgs {
    SinkSched s;             // query tiles (pass A)
    int nKT;                 // 128-key tiles a row (pass B)
    int Lp;                  // L rounded up to 128
    const __nv_bfloat16 *o, *g;
    const float* lse;
    float *nlA, *ndA;        // [B * Hkv * nMT][128]: rows of the query tiles
    float *nlB, *ndB;        // [B * H][Lp]
    __nv_bfloat16 *dq, *dk, *dv;
    float* partA;            // [2 * workers][D / 4][128][4]
    float* partB;            // [2 * workers][2][D / 4][128][4]: dK, dV
    int4 *tailA, *tailB;     // [workers]: the item (b, i, h, 1) whose first part this worker holds, or .w = 0
    int *headA, *headB;      // [workers]: 0, 1 (holds the last part of an earlier worker's item), 2 (a middle part)
    int R;
    int wholeA, wholeB;      // shares end between items: nothing to join
    int* status;
    float scale_log2, scale;
};

// ============================================================================ vectors
// A block: 32 tokens x 8 heads; delta from coalesced 16-byte reads, then both layouts.
// Memory-bound: reads o, dO and lse once (B = 8 x 16K, 12 heads of 64: 0.43 GB in 70 us, 6.2 TB/s).
template <int D>
__global__ void __launch_bounds__(256) sink_bwd_vec_kernel(const BwdArgs a) {
    __shared__ float sd[8][33];
    pdl_release();
    const SinkSched& sc = a.s;
    constexpr int LPR = D / 8;                       // lanes a row
    constexpr int RPW = 32 / LPR;                    // rows (heads) a warp reads at once
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nt = a.Lp / 32;
    const int b = blockIdx.x / nt, t0 = (blockIdx.x % nt) * 32, h0 = blockIdx.y * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int tl = warp * 4 + i, t = t0 + tl;
#pragma unroll
        for (int u = 0; u < 8 / RPW; ++u) {
            const int hl = u * RPW + lane / LPR, h = h0 + hl;
            float acc = 0.f;
            if (t < sc.L && h < sc.H) {
                const size_t off = (((size_t)b * sc.L + t) * sc.H + h) * D + (lane % LPR) * 8;
                const uint4 x = *reinterpret_cast<const uint4*>(a.o + off);
                const uint4 y = *reinterpret_cast<const uint4*>(a.g + off);
                const __nv_bfloat162* hx = reinterpret_cast<const __nv_bfloat162*>(&x);
                const __nv_bfloat162* hy = reinterpret_cast<const __nv_bfloat162*>(&y);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float2 fx = __bfloat1622float2(hx[v]), fy = __bfloat1622float2(hy[v]);
                    acc = fmaf(fx.x, fy.x, fmaf(fx.y, fy.y, acc));
                }
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
            if (lane % LPR == 0) sd[hl][tl] = acc;
        }
    }
    __syncthreads();
    // thread: token t0 + lane, head h0 + warp
    const int t = t0 + lane, h = h0 + warp;
    if (h >= sc.H) return;
    const bool live = t < sc.L;
    const float nl = live ? -a.lse[((size_t)b * sc.L + t) * sc.H + h] * kLog2e : 0.f;
    const float nd = live ? -a.scale * sd[warp][lane] : 0.f;
    const size_t ib = ((size_t)b * sc.H + h) * a.Lp + t;
    a.nlB[ib] = nl;
    a.ndB[ib] = nd;
    if (live) {
        const int hk = h / sc.G, mt = t / sc.TM;
        const size_t ia = (((size_t)b * sc.Hkv + hk) * sc.nMT + mt) * 128 + (t - mt * sc.TM) * sc.G + h - hk * sc.G;
        a.nlA[ia] = nl;
        a.ndA[ia] = nd;
    }
}

// N columns of this lane's row of an fp32 accumulator to a [N / 4][128][4] array of the
// workspace (rows side by side: the lanes of a store write 512 consecutive bytes).
template <int N>
__device__ __forceinline__ void store_rows_f32(uint32_t taddr, float* dst, int row, bool live) {
#pragma unroll 1
    for (int ci = 0; ci < N / 32; ++ci) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(taddr + 32 * ci, r);
        tmem_wait_ld();
        if (live) {
            uint4* d4 = reinterpret_cast<uint4*>(dst) + 8 * ci * 128 + row;
#pragma unroll
            for (int u = 0; u < 8; ++u) d4[u * 128] = make_uint4(r[4 * u], r[4 * u + 1], r[4 * u + 2], r[4 * u + 3]);
        }
    }
}

// ============================================================================ pass A (dQ)
namespace pa {

// 64-key tiles of a query tile: nsk tiles of sinks from tile 0 on, then k0 .. of the window.
struct Tiles {
    int k0, nsk, nt;
};
__device__ __forceinline__ Tiles tiles(const SinkSched& s, int mt) {
    Tiles k;
    const int p0 = mt * s.TM, p1 = min(s.L, p0 + s.TM) - 1;
    k.k0 = max(0, p0 - s.W + 1) >> 6;
    k.nsk = min((s.ns + 63) >> 6, k.k0);
    k.nt = k.nsk + (p1 >> 6) - k.k0 + 1;
    return k;
}

struct __align__(16) Part {
    int b, h, mt, k0, nsk;
    int j0, j1;              // steps of this part (j0 == j1: the share is done)
    int slot;                // -1: the whole item; else the workspace slot of its sums
    int nar;                 // steps of this part (its first, or none) that are narrow: 32 columns hold all sinks
    __device__ __forceinline__ int tile(int j) const { return j < nsk ? j : k0 + j - nsk; }
};

template <int D>
struct Cfg {
    static constexpr int SUB = D / 64;
    static constexpr int STILE = 128 * 128, SKEY = 64 * 128;      // bytes of a sub-tile: 128 rows, 64 rows
    static constexpr int TILE = SUB * STILE, KTILE = SUB * SKEY;
    static constexpr int ITEM = 2 * TILE;                         // Q, dO
    static constexpr int SLOT = 2 * KTILE;                        // K, V
    static constexpr int IBUF = 2;
    static constexpr int NSLOT = D == 64 ? 6 : 3;
    static constexpr int OFF_KV = IBUF * ITEM;
    static constexpr int OFF_VEC = OFF_KV + NSLOT * SLOT;         // two vectors of 128 floats
    static constexpr int SMEM = OFF_VEC + 1024 + 1024;
    static constexpr int NX = 3, NY = 3;                          // 64-column buffers of S (then ds) and of dP
    static constexpr int NACC = D == 64 ? 2 : 1;
    static constexpr uint32_t COL_X = 0, COL_Y = NX * 64, COL_ACC = COL_Y + NY * 64;
    static_assert(COL_ACC + NACC * D <= TMEM_COLS, "tensor memory");
};

template <class C>
struct __align__(16) Bars {
    Part part[kParts];
    uint64_t part_full[kParts], part_empty[kParts];
    uint64_t it_full[C::IBUF], it_empty[C::IBUF];
    uint64_t vec_full, vec_empty;
    uint64_t kv_full[C::NSLOT], kv_empty[C::NSLOT];
    uint64_t x_full[C::NX], x_empty[C::NX], y_empty[C::NY];
    uint64_t p_full[4];
    uint64_t o_full[2], o_empty[2];      // per storing warpgroup (it sees every phase); per accumulator
    uint64_t done[3];
    uint32_t tmem;
    int error;
    StreamPos pos;
    int wsum[12];
};

__device__ __forceinline__ Part next_part(const BwdArgs& a, StreamPos& p, int wid) {
    const SinkSched& s = a.s;
    Part u{};
    if (p.left <= 0) return u;
    const Tiles k = tiles(s, p.mt);
    u.b = p.b; u.h = p.h; u.mt = p.mt;
    u.k0 = k.k0; u.nsk = k.nsk;
    u.j0 = p.j;
    u.j1 = min(k.nt, p.j + p.left);
    u.nar = k.nsk == 1 && s.ns <= 32 && p.j == 0;
    u.slot = u.j0 > 0 ? 2 * wid : (u.j1 < k.nt ? 2 * wid + 1 : -1);
    if (u.j0 > 0) a.headA[wid] = u.j1 < k.nt ? 2 : 1;
    if (u.slot == 2 * wid + 1) a.tailA[wid] = make_int4(p.b, p.mt, p.h, 1);
    p.left -= u.j1 - u.j0;
    p.j = 0;
    if (++p.mt == s.nMT) {
        p.mt = 0;
        if (++p.h == s.Hkv) { p.h = 0; ++p.b; }
    }
    return u;
}

template <int D>
__global__ void __launch_bounds__(kThreadsA, 1)
sink_bwd_q_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
                  const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                  const BwdArgs a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
    __shared__ Bars<C> sb;
    static_assert(C::SMEM + sizeof(Bars<C>) <= kSmemMax, "shared memory (pass A)");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto wait = [&](uint64_t* bar, uint32_t par) { return wait_ctrl(bar, par); };
    const SinkSched& sc = a.s;

    if (threadIdx.x == 0) {
        sb.error = 0;
        for (int i = 0; i < kParts; ++i) {
            mbar_init(&sb.part_full[i], 1);
            mbar_init(&sb.part_empty[i], 3 + 8);          // the issuers and the math warps
        }
        for (int i = 0; i < C::IBUF; ++i) {
            mbar_init(&sb.it_full[i], 1);
            mbar_init(&sb.it_empty[i], 2);                // S and dP issuers
        }
        mbar_init(&sb.vec_full, 1);
        mbar_init(&sb.vec_empty, 256);
        for (int i = 0; i < C::NSLOT; ++i) {
            mbar_init(&sb.kv_full[i], 1);
            mbar_init(&sb.kv_empty[i], 1);
        }
        for (int i = 0; i < C::NX; ++i) {
            mbar_init(&sb.x_full[i], 2);
            mbar_init(&sb.x_empty[i], 1);
        }
        for (int i = 0; i < C::NY; ++i) mbar_init(&sb.y_empty[i], 128);
        for (int i = 0; i < 4; ++i) mbar_init(&sb.p_full[i], 128);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sb.o_full[i], 1);
            mbar_init(&sb.o_empty[i], 128);
        }
        for (int i = 0; i < 3; ++i) mbar_init(&sb.done[i], 1);
        fence_barrier_init();
        prefetch_tmap(&tq);
        prefetch_tmap(&tdo);
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
    }
    if (warp == 1) {
        tmem_alloc(&sb.tmem, TMEM_COLS);
        tmem_relinquish();
    }
    find_shares_dense<kThreadsA, 1>(sc.B, sc.nMT, sc.Hkv, a.wholeA, sb.wsum, &sb.pos,
                                   [&](int mt) { return tiles(sc, mt).nt; });
    tc_fence_before();
    pdl_release();
    pdl_wait();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sb.tmem;

    if (warp == 0) {
        // ------------------------------------------------------------ records and loads
        if (lane == 0) {
            Ring kv{0, 0};
            int np = 0;
            uint32_t used = 0;
            a.headA[blockIdx.x] = 0;
            a.tailA[blockIdx.x] = make_int4(0, 0, 0, 0);
            bool ok = true, done = false;
            while (ok) {
                const int r = np % kParts, ib = np % C::IBUF;
                if (!wait(&sb.part_empty[r], empty_par(np / kParts))) break;
                sb.part[r] = next_part(a, sb.pos, blockIdx.x);
                mbar_arrive(&sb.part_full[r]);
                const Part& u = sb.part[r];
                if (u.j0 == u.j1) { done = true; break; }
                if (!wait(&sb.it_empty[ib], empty_par(np / C::IBUF)) || !wait(&sb.vec_empty, empty_par(np))) break;
                uint8_t* it = sm + ib * C::ITEM;
                mbar_arrive_expect_tx(&sb.vec_full, 1024);
                mbar_arrive_expect_tx(&sb.it_full[ib], 2 * C::SUB * a.R * 128);
#pragma unroll
                for (int c = 0; c < C::SUB; ++c) {
                    tma_load_4d(it + c * C::STILE, &tq, &sb.it_full[ib], c * 64, u.h * sc.G, u.mt * sc.TM, u.b);
                    tma_load_4d(it + C::TILE + c * C::STILE, &tdo, &sb.it_full[ib], c * 64, u.h * sc.G, u.mt * sc.TM, u.b);
                }
                const size_t vrow = (((size_t)u.b * sc.Hkv + u.h) * sc.nMT + u.mt) * 128;
                tcx::bulk_load(sm + C::OFF_VEC, a.nlA + vrow, 512, &sb.vec_full);
                tcx::bulk_load(sm + C::OFF_VEC + 512, a.ndA + vrow, 512, &sb.vec_full);
                ++np;
                const int j1 = u.j1;
#pragma unroll 1
                for (int j = u.j0; j < j1; ++j) {
                    if (!wait(&sb.kv_empty[kv.i], kv.ph ^ 1u)) { ok = false; break; }
                    uint8_t* dst = sm + C::OFF_KV + kv.i * C::SLOT;
                    mbar_arrive_expect_tx(&sb.kv_full[kv.i], C::SLOT);
                    const int y = u.tile(j) * 64;
#pragma unroll
                    for (int c = 0; c < C::SUB; ++c) {
                        tma_load_3d(dst + c * C::SKEY, &tk, &sb.kv_full[kv.i], u.h * D + c * 64, y, u.b);
                        tma_load_3d(dst + C::KTILE + c * C::SKEY, &tv, &sb.kv_full[kv.i], u.h * D + c * 64, y, u.b);
                    }
                    used |= 1u << kv.i;
                    kv.next(C::NSLOT);
                }
            }
            if (!done) sb.error = GCA_ERR_TIMEOUT;
            // no copy may still be writing shared memory when the CTA exits
#pragma unroll 1
            for (int i = 0; i < C::NSLOT; ++i)
                if (used >> i & 1u) wait_copy(&sb.kv_full[i], i < kv.i ? kv.ph : kv.ph ^ 1u);
#pragma unroll 1
            for (int q = 0; q < C::IBUF; ++q) {
                const int n = (np - q + C::IBUF - 1) / C::IBUF;
                if (n > 0) wait_copy(&sb.it_full[q], full_par(n - 1));
            }
            if (np > 0) wait_copy(&sb.vec_full, full_par(np - 1));
        }
    } else if (warp == 1 || warp == 11) {
        // ------------------------------------------------------------ warp 1: S = Q K^T, warp 11: dP = dO V^T
        // (two issuing threads: one alone cannot keep the tensor pipe fed)
        const bool dpi = warp == 11;
        if (lane == 0) {
            Ring kv{0, 0};
            int u = 0;
            bool issued = false, ok = true, done = false;
            const uint32_t id_s = idesc_bf16(128, 64, false, false), id_n = idesc_bf16(128, 32, false, false);
            for (int np = 0; ok; ++np) {
                const int r = np % kParts, ib = np % C::IBUF;
                if (!wait(&sb.part_full[r], full_par(np / kParts))) break;
                const int n = sb.part[r].j1 - sb.part[r].j0, nar = sb.part[r].nar;
                mbar_arrive(&sb.part_empty[r]);
                if (n == 0) { done = true; break; }
                if (!wait(&sb.it_full[ib], full_par(np / C::IBUF))) break;
                const uint32_t aaddr = smem_u32(sm + ib * C::ITEM) + (dpi ? C::TILE : 0);
#pragma unroll 1
                for (int j = 0; j < n; ++j, ++u) {
                    const int xs = u % C::NX, ys = u % C::NY;
                    if (!wait(&sb.kv_full[kv.i], kv.ph) ||
                        !(dpi ? wait(&sb.y_empty[ys], empty_par(u / C::NY)) : wait(&sb.x_empty[xs], empty_par(u / C::NX)))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t baddr = smem_u32(sm + C::OFF_KV + kv.i * C::SLOT) + (dpi ? C::KTILE : 0);
                    tcx::mma_kmajor_dh<D>(dpi ? tmem + C::COL_Y + ys * 64 : tmem + C::COL_X + xs * 64, aaddr, 128, baddr,
                                          64, j < nar ? id_n : id_s, 0);
                    mma_commit(&sb.x_full[xs]);
                    issued = true;
                    kv.next(C::NSLOT);
                }
                if (ok) mma_commit(&sb.it_empty[ib]);
            }
            if (!done) sb.error = GCA_ERR_TIMEOUT;
            if (issued) {
                mma_commit(&sb.done[dpi ? 2 : 0]);
                wait_copy(&sb.done[dpi ? 2 : 0], 0);
            }
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ dQ += ds K (A from tensor memory)
        if (lane == 0) {
            Ring kv{0, 0};
            int u = 0;
            bool issued = false, ok = true, done = false;
            const uint32_t id_acc = idesc_bf16(128, D, false, true);
            for (int np = 0; ok; ++np) {
                const int r = np % kParts, ob = np % C::NACC;
                if (!wait(&sb.part_full[r], full_par(np / kParts))) break;
                const int n = sb.part[r].j1 - sb.part[r].j0, nar = sb.part[r].nar;
                mbar_arrive(&sb.part_empty[r]);
                if (n == 0) { done = true; break; }
                if (!wait(&sb.o_empty[ob], empty_par(np / C::NACC))) break;
                tc_fence_after();
#pragma unroll 1
                for (int j = 0; j < n; ++j, ++u) {
                    const int xs = u % C::NX;
                    // (the K tile has landed: the S product of this step, before p_full, waited for it)
                    if (!wait(&sb.p_full[u & 3], full_par(u >> 2))) { ok = false; break; }
                    tc_fence_after();
                    const uint32_t kaddr = smem_u32(sm + C::OFF_KV + kv.i * C::SLOT);
                    const uint64_t kd = smem_desc(kaddr, C::SKEY, 1024, 2);      // K: keys x D, D along N
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        if (ks == 2 && j < nar) break;
                        tc::mma_bf16_ts(tmem + C::COL_ACC + ob * D, tmem + C::COL_X + xs * 64 + 8 * ks, kd + 128 * ks, id_acc,
                                        (ks > 0 || j > 0) ? 1u : 0u);
                    }
                    mma_commit(&sb.x_empty[xs]);
                    mma_commit(&sb.kv_empty[kv.i]);       // S and dP are complete before ds exists
                    issued = true;
                    kv.next(C::NSLOT);
                }
                if (ok) mma_commit(&sb.o_full[np & 1]);
            }
            if (!done) sb.error = GCA_ERR_TIMEOUT;
            if (issued) {
                mma_commit(&sb.done[1]);
                wait_copy(&sb.done[1], 0);
            }
        }
    } else {
        // ------------------------------------------------------------ math warpgroups
        auto wwait = [&](uint64_t* bar, uint32_t par) { return __all_sync(0xffffffffu, wait(bar, par)); };
        const int wg = (warp - 3) >> 2;
        const int qd = warp & 3;
        const int row = 32 * qd + lane;               // query row of the tile = lane of tensor memory
        const int rt = row / sc.G, rg = row - rt * sc.G;
        const uint32_t lane_base = static_cast<uint32_t>(32 * qd) << 16;
        const uint64_t sl2 = tcx::f2_pack(a.scale_log2, a.scale_log2);
        const uint64_t sc2 = tcx::f2_pack(a.scale, a.scale);
        int u = 0;
        // the dQ rows of a part that this warpgroup stores leave after its first step of
        // the next one, so the wait for the part's last product overlaps work
        int pend = -1, pend_slot = -1;                // part number; workspace slot or -1
        int pend_row = -1;                            // token * H + head, or -1: no such row
        auto epilogue = [&]() {
            const int ob = pend % C::NACC;
            if (!wwait(&sb.o_full[pend & 1], full_par(pend >> 1))) return false;
            tc_fence_after();
            const uint32_t acc = tmem + lane_base + C::COL_ACC + ob * D;
            if (pend_slot < 0) {
                // (into registers first: the accumulator is free before the stores)
                uint32_t pk[D / 32][16];
#pragma unroll
                for (int ci = 0; ci < D / 32; ++ci) load_rows32(acc + 32 * ci, 1.f, pk[ci]);
                tc_fence_before();
                mbar_arrive(&sb.o_empty[ob]);
#pragma unroll
                for (int ci = 0; ci < D / 32; ++ci) store_rows32(pk[ci], a.dq + 32 * ci, D, pend_row);
            } else {
                store_rows_f32<D>(acc, a.partA + (size_t)pend_slot * 128 * D, row, pend_row >= 0);
                tc_fence_before();
                mbar_arrive(&sb.o_empty[ob]);
            }
            pend = -1;
            return true;
        };
        bool ok = true, done = false;
        for (int np = 0; ok; ++np) {
            const int r = np % kParts;
            if (!wwait(&sb.part_full[r], full_par(np / kParts))) break;
            const Part& w = sb.part[r];
            const int j0 = w.j0, j1 = w.j1, nar = w.nar, p0 = w.mt * sc.TM;
            if (j0 == j1) { done = true; break; }
            if (!wwait(&sb.vec_full, full_par(np))) break;
            const float* vec = reinterpret_cast<const float*>(sm + C::OFF_VEC);
            const float nl2 = vec[row], ndsc = vec[128 + row];
            mbar_arrive(&sb.vec_empty);
            const uint64_t nl22 = tcx::f2_pack(nl2, nl2), ndsc2 = tcx::f2_pack(ndsc, ndsc);
            const int p = p0 + rt, plast = min(sc.L, p0 + sc.TM) - 1;
#pragma unroll 1
            for (int j = j0; j < j1; ++j, ++u) {
                if ((u & 1) != wg) continue;
                const int xs = u % C::NX, ys = u % C::NY;
                if (!wwait(&sb.x_full[xs], full_par(u / C::NX))) { ok = false; break; }
                tc_fence_after();
                const int kbase = w.tile(j) * 64;
                // every row sees the whole tile, unless the diagonal or the window's edge crosses it
                const bool narrow = j - j0 < nar;
                const bool edge = kbase + 63 > p0 || (kbase < plast - sc.W + 1 && kbase + 63 >= sc.ns);
                const uint32_t xb = tmem + lane_base + C::COL_X + xs * 64;
                const uint32_t yb = tmem + lane_base + C::COL_Y + ys * 64;
                const int c_lo = p - sc.W + 1 - kbase, c_hi = p - kbase, c_s = min(sc.ns, p + 1) - kbase;
#pragma unroll
                for (int pc = 0; pc < 2; ++pc) {
                    if (pc == 1 && narrow) {                      // (columns that no product wrote)
                        tc_fence_before();
                        mbar_arrive(&sb.y_empty[ys]);
                        break;
                    }
                    // keys kbase + 32 pc .. + 31: S (X columns 32 pc ..) and dP (Y columns 32 pc ..)
                    uint32_t r0[16], r1[16], r2[16], r3[16];
                    tmem_ld_32x32b_x16(xb + 32 * pc, r0);
                    tmem_ld_32x32b_x16(xb + 32 * pc + 16, r1);
                    tmem_ld_32x32b_x16(yb + 32 * pc, r2);
                    tmem_ld_32x32b_x16(yb + 32 * pc + 16, r3);
                    tmem_wait_ld();
                    if (pc == 1) {                                // dP fully read: free its buffer
                        tc_fence_before();
                        mbar_arrive(&sb.y_empty[ys]);
                    }
                    const uint32_t vis = (below(c_hi + 1 - 32 * pc) & ~below(c_lo - 32 * pc)) | below(c_s - 32 * pc);
                    uint32_t pk[16];
                    auto body = [&](bool msk) {
#pragma unroll
                        for (int p2 = 0; p2 < 16; ++p2) {
                            const uint32_t* rs = p2 < 8 ? r0 : r1;
                            const uint32_t* rd = p2 < 8 ? r2 : r3;
                            const int tt = 2 * (p2 & 7);
                            float y0, y1;
                            tcx::f2_unpack(tcx::ffma2(tcx::f2_pack(__uint_as_float(rs[tt]), __uint_as_float(rs[tt + 1])),
                                                      sl2, nl22), y0, y1);
                            float e0 = fast_exp2(y0), e1 = fast_exp2(y1);
                            if (msk) {
                                e0 = (vis >> (2 * p2) & 1u) ? e0 : 0.f;
                                e1 = (vis >> (2 * p2 + 1) & 1u) ? e1 : 0.f;
                            }
                            const uint64_t gd = tcx::ffma2(
                                tcx::f2_pack(__uint_as_float(rd[tt]), __uint_as_float(rd[tt + 1])), sc2, ndsc2);
                            pk[p2] = tcx::pack_bf16x2(tcx::fmul2(tcx::f2_pack(e0, e1), gd));
                        }
                    };
                    if (edge) body(true);
                    else body(false);
                    tmem_st_32x32b_x16(xb + 16 * pc, pk);         // ds over S columns that have been read
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&sb.p_full[u & 3]);
                if (pend >= 0 && !epilogue()) { ok = false; break; }
            }
            if (!ok) break;
            if ((np & 1) == wg) {
                // (a part shorter than two steps may leave this warpgroup's last one pending)
                if (pend >= 0 && !epilogue()) break;
                pend = np;
                pend_slot = w.slot;
                const bool live = row < a.R && p <= plast;
                pend_row = live ? (w.b * sc.L + p) * sc.H + w.h * sc.G + rg : -1;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sb.part_empty[r]);
        }
        if (done && pend >= 0) done = epilogue();
        if (!done) sb.error = GCA_ERR_TIMEOUT;
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sb.error) set_status(a.status, sb.error);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}
}  // namespace pa

// ============================================================================ pass B (dK, dV)
namespace pb {

// Query blocks (64 queries) of key tile kt: g0 .. g0 + nw - 1 whose window reaches its
// keys, and for tiles that hold sinks the nf blocks behind them, up to the row's end.
struct Blocks {
    int g0, nw, nf;
};
__device__ __forceinline__ Blocks blocks(const SinkSched& s, int kt) {
    Blocks k;
    k.g0 = kt * 2;
    const int end = (s.L - 1) >> 6;
    const int last = min(s.L - 1, kt * 128 + 127 + s.W - 1) >> 6;
    k.nw = last - k.g0 + 1;
    k.nf = kt * 128 < s.ns ? end - last : 0;
    return k;
}

struct __align__(16) Part {
    int b, h, kt;
    int nw, nf;
    int j0, j1;              // steps: (query head, window block), then (query head, far block)
    int slot;
};

// A step's query head within the group and its query block, counted along.
struct Step {
    int g, i, n;             // i-th of n blocks, from block `first` on
    int first, far_first, nf;
    __device__ __forceinline__ void init(const Part& u, int G) {
        const int nwin = G * u.nw;
        far_first = 2 * u.kt + u.nw;
        nf = u.nf;
        if (u.j0 < nwin) {
            first = 2 * u.kt;
            n = u.nw;
            g = u.j0 / n;
            i = u.j0 - g * n;
        } else {
            first = far_first;
            n = nf;
            g = (u.j0 - nwin) / n;
            i = u.j0 - nwin - g * n;
        }
    }
    __device__ __forceinline__ int block() const { return first + i; }
    __device__ __forceinline__ void next(int G) {
        if (++i < n) return;
        i = 0;
        if (++g < G) return;
        g = 0;
        first = far_first;
        n = nf;
    }
};

template <int D>
struct Cfg {
    static constexpr int SUB = D / 64;
    static constexpr int STILE = 128 * 128, SQ = 64 * 128;
    static constexpr int TILE = SUB * STILE, QTILE = SUB * SQ;
    static constexpr int ITEM = 2 * TILE;                         // K, V
    static constexpr int SLOT = 2 * QTILE + 1024;                 // Q, dO, two vectors of 64 floats
    static constexpr int IBUF = D == 64 ? 2 : 1;
    static constexpr int NSLOT = D == 64 ? 8 : 4;
    static constexpr int OFF_ST = IBUF * ITEM;
    static constexpr int SMEM = OFF_ST + NSLOT * SLOT + 1024;
    static constexpr int NX = D == 64 ? 3 : 2, NY = NX;
    static constexpr uint32_t COL_X = 0, COL_Y = NX * 64, COL_ACC = COL_Y + NY * 64;   // dK, dV
    static_assert(COL_ACC + 2 * D <= TMEM_COLS, "tensor memory");
};

template <class C>
struct __align__(16) Bars {
    Part part[kParts];
    uint64_t part_full[kParts], part_empty[kParts];
    uint64_t it_full[C::IBUF], it_empty[C::IBUF];
    uint64_t st_full[C::NSLOT], st_empty[C::NSLOT];
    uint64_t x_full[C::NX], x_empty[C::NX], y_empty[C::NY];
    uint64_t p_full[4];
    uint64_t o_full[2], o_empty;         // o_full per storing warpgroup: it sees every phase
    uint64_t done[3];
    uint32_t tmem;
    int error;
    StreamPos pos;
    int wsum[20];
};

__device__ __forceinline__ Part next_part(const BwdArgs& a, StreamPos& p, int wid) {
    const SinkSched& s = a.s;
    Part u{};
    if (p.left <= 0) return u;
    const Blocks k = blocks(s, p.mt);
    const int n = s.G * (k.nw + k.nf);
    u.b = p.b; u.h = p.h; u.kt = p.mt;
    u.nw = k.nw; u.nf = k.nf;
    u.j0 = p.j;
    u.j1 = min(n, p.j + p.left);
    u.slot = u.j0 > 0 ? 2 * wid : (u.j1 < n ? 2 * wid + 1 : -1);
    if (u.j0 > 0) a.headB[wid] = u.j1 < n ? 2 : 1;
    if (u.slot == 2 * wid + 1) a.tailB[wid] = make_int4(p.b, p.mt, p.h, 1);
    p.left -= u.j1 - u.j0;
    p.j = 0;
    if (++p.mt == a.nKT) {
        p.mt = 0;
        if (++p.h == s.Hkv) { p.h = 0; ++p.b; }
    }
    return u;
}

template <int D>
__global__ void __launch_bounds__(kThreadsB, 1)
sink_bwd_kv_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tdo,
                   const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                   const BwdArgs a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
    __shared__ Bars<C> sb;
    static_assert(C::SMEM + sizeof(Bars<C>) <= kSmemMax, "shared memory (pass B)");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto wait = [&](uint64_t* bar, uint32_t par) { return wait_ctrl(bar, par); };
    const SinkSched& sc = a.s;

    if (threadIdx.x == 0) {
        sb.error = 0;
        for (int i = 0; i < kParts; ++i) {
            mbar_init(&sb.part_full[i], 1);
            mbar_init(&sb.part_empty[i], 3 + 16);          // the issuers and the math warps
        }
        for (int i = 0; i < C::IBUF; ++i) {
            mbar_init(&sb.it_full[i], 1);
            mbar_init(&sb.it_empty[i], 2);
        }
        for (int i = 0; i < C::NSLOT; ++i) {
            mbar_init(&sb.st_full[i], 1);
            mbar_init(&sb.st_empty[i], 1);
        }
        for (int i = 0; i < C::NX; ++i) {
            mbar_init(&sb.x_full[i], 2);
            mbar_init(&sb.x_empty[i], 1);
        }
        for (int i = 0; i < C::NY; ++i) mbar_init(&sb.y_empty[i], 256);
        for (int i = 0; i < 4; ++i) mbar_init(&sb.p_full[i], 256);
        mbar_init(&sb.o_full[0], 1);
        mbar_init(&sb.o_full[1], 1);
        mbar_init(&sb.o_empty, 256);
        for (int i = 0; i < 3; ++i) mbar_init(&sb.done[i], 1);
        fence_barrier_init();
        prefetch_tmap(&tq);
        prefetch_tmap(&tdo);
        prefetch_tmap(&tk);
        prefetch_tmap(&tv);
    }
    if (warp == 1) {
        tmem_alloc(&sb.tmem, TMEM_COLS);
        tmem_relinquish();
    }
    find_shares_dense<kThreadsB, 1>(sc.B, a.nKT, sc.Hkv, a.wholeB, sb.wsum, &sb.pos, [&](int kt) {
        const Blocks k = blocks(sc, kt);
        return sc.G * (k.nw + k.nf);
    });
    tc_fence_before();
    pdl_release();
    pdl_wait();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sb.tmem;

    if (warp < 4) {
        setmaxnreg_dec<kRegsCtrlB>();
        if (warp == 0) {
            // ------------------------------------------------------------ records and loads
            if (lane == 0) {
                Ring st{0, 0};
                int np = 0;
                uint32_t used = 0;
                a.headB[blockIdx.x] = 0;
                a.tailB[blockIdx.x] = make_int4(0, 0, 0, 0);
                bool ok = true, done = false;
                while (ok) {
                    const int r = np % kParts, ib = np % C::IBUF;
                    if (!wait(&sb.part_empty[r], empty_par(np / kParts))) break;
                    sb.part[r] = next_part(a, sb.pos, blockIdx.x);
                    mbar_arrive(&sb.part_full[r]);
                    const Part& u = sb.part[r];
                    if (u.j0 == u.j1) { done = true; break; }
                    if (!wait(&sb.it_empty[ib], empty_par(np / C::IBUF))) break;
                    uint8_t* it = sm + ib * C::ITEM;
                    mbar_arrive_expect_tx(&sb.it_full[ib], C::ITEM);
#pragma unroll
                    for (int c = 0; c < C::SUB; ++c) {
                        tma_load_3d(it + c * C::STILE, &tk, &sb.it_full[ib], u.h * D + c * 64, u.kt * 128, u.b);
                        tma_load_3d(it + C::TILE + c * C::STILE, &tv, &sb.it_full[ib], u.h * D + c * 64, u.kt * 128, u.b);
                    }
                    ++np;
                    Step sp;
                    sp.init(u, sc.G);
                    const int n = u.j1 - u.j0;
#pragma unroll 1
                    for (int j = 0; j < n; ++j) {
                        if (!wait(&sb.st_empty[st.i], st.ph ^ 1u)) { ok = false; break; }
                        uint8_t* dst = sm + C::OFF_ST + st.i * C::SLOT;
                        const int qb = sp.block() * 64, h = u.h * sc.G + sp.g;
                        mbar_arrive_expect_tx(&sb.st_full[st.i], 2 * C::QTILE + 512);
#pragma unroll
                        for (int c = 0; c < C::SUB; ++c) {
                            tma_load_4d(dst + c * C::SQ, &tq, &sb.st_full[st.i], c * 64, h, qb, u.b);
                            tma_load_4d(dst + C::QTILE + c * C::SQ, &tdo, &sb.st_full[st.i], c * 64, h, qb, u.b);
                        }
                        const size_t vrow = ((size_t)u.b * sc.H + h) * a.Lp + qb;
                        tcx::bulk_load(dst + 2 * C::QTILE, a.nlB + vrow, 256, &sb.st_full[st.i]);
                        tcx::bulk_load(dst + 2 * C::QTILE + 256, a.ndB + vrow, 256, &sb.st_full[st.i]);
                        used |= 1u << st.i;
                        st.next(C::NSLOT);
                        sp.next(sc.G);
                    }
                }
                if (!done) sb.error = GCA_ERR_TIMEOUT;
                // no copy may still be writing shared memory when the CTA exits
#pragma unroll 1
                for (int i = 0; i < C::NSLOT; ++i)
                    if (used >> i & 1u) wait_copy(&sb.st_full[i], i < st.i ? st.ph : st.ph ^ 1u);
#pragma unroll 1
                for (int q = 0; q < C::IBUF; ++q) {
                    const int n = (np - q + C::IBUF - 1) / C::IBUF;
                    if (n > 0) wait_copy(&sb.it_full[q], full_par(n - 1));
                }
            }
        } else if (warp == 1 || warp == 3) {
            // ------------------------------------------------------------ warp 1: S^T = K Q^T, warp 3: dP^T = V dO^T
            const bool dpi = warp == 3;
            if (lane == 0) {
                Ring st{0, 0};
                int u = 0;
                bool issued = false, ok = true, done = false;
                const uint32_t id_s = idesc_bf16(128, 64, false, false);
                for (int np = 0; ok; ++np) {
                    const int r = np % kParts, ib = np % C::IBUF;
                    if (!wait(&sb.part_full[r], full_par(np / kParts))) break;
                    const int n = sb.part[r].j1 - sb.part[r].j0;
                    mbar_arrive(&sb.part_empty[r]);
                    if (n == 0) { done = true; break; }
                    if (!wait(&sb.it_full[ib], full_par(np / C::IBUF))) break;
                    const uint32_t aaddr = smem_u32(sm + ib * C::ITEM) + (dpi ? C::TILE : 0);
#pragma unroll 1
                    for (int j = 0; j < n; ++j, ++u) {
                        const int xs = u % C::NX;
                        if (!wait(&sb.st_full[st.i], st.ph) ||
                            !wait(dpi ? &sb.y_empty[xs] : &sb.x_empty[xs], empty_par(u / C::NX))) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t baddr = smem_u32(sm + C::OFF_ST + st.i * C::SLOT) + (dpi ? C::QTILE : 0);
                        tcx::mma_kmajor_dh<D>(tmem + (dpi ? C::COL_Y : C::COL_X) + xs * 64, aaddr, 128, baddr, 64, id_s, 0);
                        mma_commit(&sb.x_full[xs]);
                        issued = true;
                        st.next(C::NSLOT);
                    }
                    if (ok) mma_commit(&sb.it_empty[ib]);     // K (V) is read only by these products
                }
                if (!done) sb.error = GCA_ERR_TIMEOUT;
                if (issued) {
                    mma_commit(&sb.done[dpi ? 2 : 0]);
                    wait_copy(&sb.done[dpi ? 2 : 0], 0);
                }
            }
        } else {
            // ------------------------------------------------------------ dK += ds^T Q, dV += P^T dO
            if (lane == 0) {
                Ring st{0, 0};
                int u = 0;
                bool issued = false, ok = true, done = false;
                const uint32_t id_acc = idesc_bf16(128, D, false, true);
                for (int np = 0; ok; ++np) {
                    const int r = np % kParts;
                    if (!wait(&sb.part_full[r], full_par(np / kParts))) break;
                    const int n = sb.part[r].j1 - sb.part[r].j0;
                    mbar_arrive(&sb.part_empty[r]);
                    if (n == 0) { done = true; break; }
                    if (!wait(&sb.o_empty, empty_par(np))) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int j = 0; j < n; ++j, ++u) {
                        const int xs = u % C::NX;
                        if (!wait(&sb.p_full[u & 3], full_par(u >> 2))) { ok = false; break; }
                        tc_fence_after();
                        // A: K = 16 query steps at X columns 0, 16, 32, 48 (ds^T) and 8, 24, 40, 56 (P^T);
                        // B: queries x D with D along N
                        const uint64_t qd = smem_desc(smem_u32(sm + C::OFF_ST + st.i * C::SLOT), C::SQ, 1024, 2);
                        const uint32_t xa = tmem + C::COL_X + xs * 64;
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            const uint32_t col = xa + 16 * ks;
                            const uint32_t acc = (ks > 0 || j > 0) ? 1u : 0u;
                            tc::mma_bf16_ts(tmem + C::COL_ACC, col, qd + 128 * ks, id_acc, acc);
                            tc::mma_bf16_ts(tmem + C::COL_ACC + D, col + 8, qd + (C::QTILE >> 4) + 128 * ks, id_acc, acc);
                        }
                        mma_commit(&sb.x_empty[xs]);
                        mma_commit(&sb.st_empty[st.i]);
                        issued = true;
                        st.next(C::NSLOT);
                    }
                    if (ok) mma_commit(&sb.o_full[np & 1]);
                }
                if (!done) sb.error = GCA_ERR_TIMEOUT;
                if (issued) {
                    mma_commit(&sb.done[1]);
                    wait_copy(&sb.done[1], 0);
                }
            }
        }
    } else {
        setmaxnreg_inc<kRegsMathB>();
        auto wwait = [&](uint64_t* bar, uint32_t par) { return __all_sync(0xffffffffu, wait(bar, par)); };
        // warpgroup pair `wg` takes every other step; `half` of a step's columns each
        const int wg = (warp - 4) >> 3, half = (warp >> 2) & 1;
        const int qd = warp & 3;
        const int row = 32 * qd + lane;               // key row of the tile = lane of tensor memory
        const uint32_t lane_base = static_cast<uint32_t>(32 * qd) << 16;
        const uint64_t sl2 = tcx::f2_pack(a.scale_log2, a.scale_log2);
        const uint64_t sc2 = tcx::f2_pack(a.scale, a.scale);
        Ring st{0, 0};
        int u = 0;
        // The sums of a part that this pair stores (dK rows one warpgroup, dV rows the other) leave
        // after its first step of the next one, so the wait for the part's last products overlaps
        // work (d = 64: 1.29 -> 1.24 ms at B = 8 x 16K; at d = 128, with two score buffers in place of
        // three, at once: 1.08 -> 1.06 ms at 2 x 16K with 16/4 heads).
        int pend = -1, pend_slot = -1, pend_row = -1;
        auto epilogue = [&]() {
            if (!wwait(&sb.o_full[wg], full_par(pend >> 1))) return false;
            tc_fence_after();
            const uint32_t acc = tmem + lane_base + C::COL_ACC + half * D;
            if (pend_slot < 0) {
                __nv_bfloat16* const out = half ? a.dv : a.dk;
                if constexpr (D == 64) {
                    // into registers first: the next part may accumulate before the stores
                    uint32_t pk[2][16];
                    load_rows32(acc, 1.f, pk[0]);
                    load_rows32(acc + 32, 1.f, pk[1]);
                    tc_fence_before();
                    mbar_arrive(&sb.o_empty);
                    store_rows32(pk[0], out, D, pend_row);
                    store_rows32(pk[1], out + 32, D, pend_row);
                } else {
#pragma unroll 1
                    for (int ci = 0; ci < D / 32; ++ci) {         // (too many for the registers)
                        uint32_t pk[16];
                        load_rows32(acc + 32 * ci, 1.f, pk);
                        if (ci + 1 == D / 32) {
                            tc_fence_before();
                            mbar_arrive(&sb.o_empty);
                        }
                        store_rows32(pk, out + 32 * ci, D, pend_row);
                    }
                }
            } else {
                store_rows_f32<D>(acc, a.partB + ((size_t)pend_slot * 256 + half * 128) * D, row, pend_row >= 0);
                tc_fence_before();
                mbar_arrive(&sb.o_empty);
            }
            pend = -1;
            return true;
        };
        bool ok = true, done = false;
        for (int np = 0; ok; ++np) {
            const int r = np % kParts;
            if (!wwait(&sb.part_full[r], full_par(np / kParts))) break;
            const Part& w = sb.part[r];
            const int n = w.j1 - w.j0;
            if (n == 0) { done = true; break; }
            const int s0 = w.kt * 128, s = s0 + row;  // this thread's key
            Step sp;
            sp.init(w, sc.G);
            // the last query that sees key s
            const int last = min(sc.L - 1, s < sc.ns ? sc.L - 1 : s + sc.W - 1);
#pragma unroll 1
            for (int j = 0; j < n; ++j, ++u, st.next(C::NSLOT), sp.next(sc.G)) {
                if ((u & 1) != wg) continue;
                const int xs = u % C::NX, ys = u % C::NY;
                // (x_full: the stage has landed too, so the phase of its barrier is the one meant)
                if (!wwait(&sb.x_full[xs], full_par(u / C::NX)) || !wwait(&sb.st_full[st.i], st.ph)) { ok = false; break; }
                tc_fence_after();
                const int qb = sp.block() * 64;
                const int c_lo = s - qb, c_hi = last - qb;
                const uint8_t* vec = sm + C::OFF_ST + st.i * C::SLOT + 2 * C::QTILE;
                const uint64_t* nl = reinterpret_cast<const uint64_t*>(vec);              // pairs
                const uint64_t* nd = reinterpret_cast<const uint64_t*>(vec + 256);
                const uint32_t xb = tmem + lane_base + C::COL_X + xs * 64;
                const uint32_t yb = tmem + lane_base + C::COL_Y + ys * 64;
                // does any key of this warp see any query of the block, and every key every query?
                const bool some = __any_sync(0xffffffffu, c_hi >= 0 && c_lo <= 63 && c_hi >= c_lo);
                const bool all = __all_sync(0xffffffffu, c_lo <= 0 && c_hi >= 63);
                if (!some) {
                    tc_fence_before();
                    mbar_arrive(&sb.y_empty[ys]);
                    const uint32_t z[16] = {};
#pragma unroll
                    for (int c = 0; c < 2; ++c) tmem_st_32x32b_x16(xb + 32 * half + 16 * c, z);
                } else {
                    // (without the masks where every key sees every query: 0.64 instead of 0.67 ms at
                    // B = 8 x 16K)
                    auto body = [&](bool msk) {
#pragma unroll
                        for (int cc = 0; cc < 2; ++cc) {
                            const int c = 2 * half + cc;
                            uint32_t rs[16], rd[16];
                            tmem_ld_32x32b_x16(xb + 16 * c, rs);
                            tmem_ld_32x32b_x16(yb + 16 * c, rd);
                            tmem_wait_ld();
                            if (cc == 1) {
                                tc_fence_before();
                                mbar_arrive(&sb.y_empty[ys]);
                            }
                            const uint32_t vis = below(c_hi + 1 - 16 * c) & ~below(c_lo - 16 * c);
                            uint32_t pd[8], pp[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                float y0, y1;
                                tcx::f2_unpack(tcx::ffma2(tcx::f2_pack(__uint_as_float(rs[2 * i]), __uint_as_float(rs[2 * i + 1])),
                                                          sl2, nl[8 * c + i]), y0, y1);
                                float e0 = fast_exp2(y0), e1 = fast_exp2(y1);
                                if (msk) {
                                    e0 = (vis >> (2 * i) & 1u) ? e0 : 0.f;
                                    e1 = (vis >> (2 * i + 1) & 1u) ? e1 : 0.f;
                                }
                                const uint64_t ev = tcx::f2_pack(e0, e1);
                                const uint64_t gd = tcx::ffma2(tcx::f2_pack(__uint_as_float(rd[2 * i]), __uint_as_float(rd[2 * i + 1])),
                                                               sc2, nd[8 * c + i]);
                                pd[i] = tcx::pack_bf16x2(tcx::fmul2(ev, gd));
                                pp[i] = tcx::pack_bf16x2(ev);
                            }
                            // ds^T, then P^T, over the 16 S^T columns just read
                            tmem_st_32x32b_x8(xb + 16 * c, pd);
                            tmem_st_32x32b_x8(xb + 16 * c + 8, pp);
                        }
                    };
                    if (all) body(false);
                    else body(true);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(&sb.p_full[u & 3]);
                if (D == 64 && pend >= 0 && !epilogue()) { ok = false; break; }
            }
            if (!ok) break;
            if ((np & 1) == wg) {                     // this pair stores the part's sums
                // (a part shorter than two steps may leave its last one pending)
                if (pend >= 0 && !epilogue()) break;
                pend = np;
                pend_slot = w.slot;
                pend_row = s < sc.L ? (w.b * sc.L + s) * sc.Hkv + w.h : -1;
                if (D == 128 && !epilogue()) break;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sb.part_empty[r]);
        }
        if (done && pend >= 0) done = epilogue();
        if (!done) sb.error = GCA_ERR_TIMEOUT;
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sb.error) set_status(a.status, sb.error);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}
}  // namespace pb

// Adds up the parts of the items that were cut (10 to 18 us, launch and latency), in the order
// of the stream: blocks (w, *, *) the item that begins in worker w's share and goes on in the next ones (pass A for
// blockIdx.z = 0, pass B's dK and dV for 1 and 2).
template <int D>
__global__ void __launch_bounds__(256) sink_bwd_join_kernel(const BwdArgs a, int workers) {
    pdl_wait();
    const SinkSched& sc = a.s;
    const bool pass_a = blockIdx.z == 0;
    const int w = blockIdx.x;
    const int4 it = (pass_a ? a.tailA : a.tailB)[w];
    if (it.w == 0) return;
    const int n = parts_of(pass_a ? a.headA : a.headB, w, workers);
    constexpr int VEC = D / 4;
    constexpr int ROWS = 256 / VEC;
    const int row = blockIdx.y * ROWS + threadIdx.x % ROWS, c = threadIdx.x / ROWS;
    size_t orow;
    if (pass_a) {
        const int rt = row / sc.G, t = it.y * sc.TM + rt;
        if (row >= a.R || t >= sc.L) return;
        orow = (size_t)(it.x * sc.L + t) * sc.H + it.z * sc.G + (row - rt * sc.G);
    } else {
        const int s = it.y * 128 + row;
        if (s >= sc.L) return;
        orow = (size_t)(it.x * sc.L + s) * sc.Hkv + it.z;
    }
    const size_t slot_rows = pass_a ? 128 : 256;
    const float* base = pass_a ? a.partA : a.partB + (blockIdx.z == 2 ? 128 * D : 0);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
        const size_t slot = k == 0 ? 2 * w + 1 : 2 * (w + k);
        const float4 x = reinterpret_cast<const float4*>(base + slot * slot_rows * D)[c * 128 + row];
        acc.x += x.x; acc.y += x.y; acc.z += x.z; acc.w += x.w;
    }
    __nv_bfloat16* dst = pass_a ? a.dq : blockIdx.z == 1 ? a.dk : a.dv;
    reinterpret_cast<uint2*>(dst + orow * D)[c] = make_uint2(tcx::pack_bf16(acc.x, acc.y), tcx::pack_bf16(acc.z, acc.w));
}

struct Layout {
    size_t nlA, ndA, nlB, ndB, partA, partB, tailA, tailB, headA, headB, total;
    int TM, R, nMT, Lp;
};
Layout layout(const SinkShape& s) {
    Layout w;
    const int G = s.H / s.Hkv;
    w.TM = 128 / G < s.L ? 128 / G : s.L;
    w.R = w.TM * G;
    w.nMT = (s.L + w.TM - 1) / w.TM;
    w.Lp = (s.L + 127) / 128 * 128;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t p = at;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    const size_t va = (size_t)s.B * s.Hkv * w.nMT * 128 * 4, vb = (size_t)s.B * s.H * w.Lp * 4;
    w.nlA = take(va);
    w.ndA = take(va);
    w.nlB = take(vb);
    w.ndB = take(vb);
    w.partA = take((size_t)2 * kMaxCtas * 128 * s.d * 4);
    w.partB = take((size_t)2 * kMaxCtas * 256 * s.d * 4);
    w.tailA = take(kMaxCtas * 16);
    w.tailB = take(kMaxCtas * 16);
    w.headA = take(kMaxCtas * 4);
    w.headB = take(kMaxCtas * 4);
    w.total = at;
    return w;
}

template <int D>
cudaError_t launch(const SinkShape& s, const BwdArgs& a, const CUtensorMap (&m)[8], cudaStream_t st,
                   int* launches) {
    static LaunchSetup setup;
    int sms = 0;
    cudaError_t e = setup.once(
        [] {
            const cudaError_t r = cudaFuncSetAttribute(pa::sink_bwd_q_kernel<D>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, pa::Cfg<D>::SMEM);
            if (r != cudaSuccess) return r;
            // (a build that gave the kernel fewer registers would wait forever at the split: refuse it)
            cudaFuncAttributes fa;
            if (const cudaError_t x = cudaFuncGetAttributes(&fa, pb::sink_bwd_kv_kernel<D>)) return x;
            if (fa.numRegs < kRegsB) return cudaErrorInvalidConfiguration;
            return cudaFuncSetAttribute(pb::sink_bwd_kv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        pb::Cfg<D>::SMEM);
        },
        &sms);
    if (e != cudaSuccess) return e;
    const int grid = sms < kMaxCtas ? sms : kMaxCtas;
    const dim3 vgrid((unsigned)(s.B * (a.Lp / 32)), (unsigned)((s.H + 7) / 8));
    GCA_LAUNCH("sink_bwd_vec", st, sink_bwd_vec_kernel<D><<<vgrid, 256, 0, st>>>(a));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    GCA_LAUNCH("sink_bwd_q", st,
               e = launch_pdl(pa::sink_bwd_q_kernel<D>, dim3(grid), kThreadsA, pa::Cfg<D>::SMEM, st, m[0], m[1], m[2], m[3], a));
    if (e != cudaSuccess) return e;
    GCA_LAUNCH("sink_bwd_kv", st,
               e = launch_pdl(pb::sink_bwd_kv_kernel<D>, dim3(grid), kThreadsB, pb::Cfg<D>::SMEM, st, m[4], m[5], m[6], m[7], a));
    if (e != cudaSuccess) return e;
    *launches += 3;
    if (a.wholeA && a.wholeB) return e;
    GCA_LAUNCH("sink_bwd_join", st,
               e = launch_pdl(sink_bwd_join_kernel<D>, dim3(grid, 128 * D / 1024, 3), 256, 0, st, a, grid));
    if (e == cudaSuccess) *launches += 1;
    return e;
}

}  // namespace

bool sink_bwd_supported(const SinkShape& s) {
    // steps are counted in 32 bits.  Key-major ones, a query head: tile kt has the blocks from 2 kt on
    // that its window reaches, with sinks all to the row's end
    const double nkt = (s.L + 127) / 128, nb = (s.L + 63) / 64, nst = (s.ns + 127) / 128;
    const double kv = nst * nb - nst * (nst - 1) + causal_sum(nkt - nst, 2, (s.W + 126.0) / 64 + 1);
    // query-major ones, a key head: where 128 / G rounds down, a tile's rows are few and its steps more
    const int tm = std::min(128 / (s.H / s.Hkv), s.L);
    const double q = causal_sum((s.L + tm - 1) / tm, tm / 64.0, ((double)s.W + tm + s.ns) / 64 + 3);
    return s.B * s.H * kv < kMaxSteps && s.B * s.Hkv * q < kMaxSteps && s.B * nkt * 4 < 2e9;
}

size_t sink_bwd_workspace_bytes(const SinkShape& s) { return layout(s).total; }

cudaError_t launch_sink_bwd(const SinkShape& s, const void* q, const void* k, const void* v,
                            const void* o, const float* lse, const void* dout, void* dq, void* dk,
                            void* dv, void* ws, int* status, cudaStream_t st, int* launches) {
    const Layout w = layout(s);
    uint8_t* base = static_cast<uint8_t*>(ws);
    BwdArgs a{};
    a.s.B = s.B; a.s.L = s.L; a.s.H = s.H; a.s.Hkv = s.Hkv; a.s.G = s.H / s.Hkv;
    a.s.W = s.W; a.s.ns = s.ns;
    a.s.TM = w.TM;
    a.s.nMT = w.nMT;
    a.R = w.R;
    a.nKT = w.Lp / 128;
    a.Lp = w.Lp;
    a.o = static_cast<const __nv_bfloat16*>(o);
    a.g = static_cast<const __nv_bfloat16*>(dout);
    a.lse = lse;
    a.nlA = reinterpret_cast<float*>(base + w.nlA);
    a.ndA = reinterpret_cast<float*>(base + w.ndA);
    a.nlB = reinterpret_cast<float*>(base + w.nlB);
    a.ndB = reinterpret_cast<float*>(base + w.ndB);
    a.dq = static_cast<__nv_bfloat16*>(dq);
    a.dk = static_cast<__nv_bfloat16*>(dk);
    a.dv = static_cast<__nv_bfloat16*>(dv);
    a.partA = reinterpret_cast<float*>(base + w.partA);
    a.partB = reinterpret_cast<float*>(base + w.partB);
    a.tailA = reinterpret_cast<int4*>(base + w.tailA);
    a.tailB = reinterpret_cast<int4*>(base + w.tailB);
    a.headA = reinterpret_cast<int*>(base + w.headA);
    a.headB = reinterpret_cast<int*>(base + w.headB);
    a.status = status;
    a.scale = s.scale;
    a.scale_log2 = s.scale * kLog2e;
    // Items are left whole where the longest share is then longer than the mean by less than a cut's
    // sums and the join take, C steps (2 x 4K, 12 heads of 64, W = 512: 83 instead of 96 us), but not
    // pass A's where pass B's are cut, unless shares are short: the join is launched anyway, and long
    // shares are more even with cuts (B = 8 x 16K with sinks: 437 instead of 441 us).  Items with
    // sinks, many times longer than the others, are always cut.
    auto excess = [](long long items, long long steps) {
        return (items + kMaxCtas - 1) / kMaxCtas * steps - items * steps / kMaxCtas;
    };
    constexpr long long C = 12;
    const long long spanA = s.W + a.s.TM - 1 < s.L ? s.W + a.s.TM - 1 : s.L, spanB = s.W + 127 < s.L ? s.W + 127 : s.L;
    const long long itemsA = (long long)s.B * s.Hkv * a.s.nMT, stepsA = (spanA + 62) / 64 + 1 + (s.ns + 63) / 64;
    const long long itemsB = (long long)s.B * s.Hkv * a.nKT, stepsB = a.s.G * ((spanB + 62) / 64 + 1);
    a.wholeB = s.ns == 0 && excess(itemsB, stepsB) <= C;
    a.wholeA = (a.wholeB || itemsA * stepsA <= 40 * kMaxCtas) && excess(itemsA, stepsA) <= C;
    const uint64_t d = s.d, H = s.H, L = s.L, B = s.B, kvcols = (uint64_t)s.Hkv * s.d;
    const uint64_t qn[4] = {d, H, L, B};
    const uint64_t qs[3] = {d, (uint64_t)s.q_stride, (uint64_t)s.q_stride * L}, gs[3] = {d, H * d, H * d * L};
    const uint32_t boxa[3] = {(uint32_t)a.s.G, (uint32_t)a.s.TM, 1}, boxb[3] = {1, 64, 1};
    CUtensorMap m[8];
    const bool wide = s.d == 128;             // (d = 64: a head's row is 128 bytes, as in the forward; pass A -1%)
    bool ok = encode_bf16_4d(&m[0], q, qn, qs, boxa, wide) && encode_bf16_4d(&m[1], dout, qn, gs, boxa, wide) &&
              encode_bf16_4d(&m[4], q, qn, qs, boxb, wide) && encode_bf16_4d(&m[5], dout, qn, gs, boxb, wide);
    for (int i = 0; i < 2; ++i)
        ok = ok && encode_bf16_3d(&m[2 + 4 * i], k, kvcols, L, B, s.kv_stride, s.kv_stride * L, i ? 128 : 64, 1, wide) &&
             encode_bf16_3d(&m[3 + 4 * i], v, kvcols, L, B, s.kv_stride, s.kv_stride * L, i ? 128 : 64, 1, wide);
    if (!ok) return cudaErrorInvalidValue;
    return s.d == 64 ? launch<64>(s, a, m, st, launches) : launch<128>(s, a, m, st, launches);
}

}  // namespace gca
