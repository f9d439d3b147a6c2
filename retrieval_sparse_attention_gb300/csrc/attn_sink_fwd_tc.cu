// attn_sink_fwd_tc.cu -- forward of the windowed attention with sinks on the
// Blackwell tensor cores (bf16, d = 64 or 128), over dense sequences and over a
// paged K/V cache, from one new token to whole prompts.
//
//   o_t = sum_{s in V(t)} softmax_s(attn_scale q_t . k_s) v_s,
//   V(t) = { s <= t : s > t - W or s < ns }.
//
// Work: units (sequence, 128-row query tile, key head) of a few to many key
// tiles (attn_sink.cuh).  All key tiles of all units form one stream, which is cut
// into equal shares, one per worker, wherever the cuts fall: a chunk of a
// prompt, a batch of single tokens over uneven caches and one token over a long
// cache all fill the machine.  Every CTA finds its cuts itself from a scan over
// the sequences' lengths (on the device: a captured graph follows them).  A
// unit cut by a share's end leaves unnormalised fp32 sums with their maxima in
// the workspace, two slots a worker, and a second small kernel joins them in the
// order of the stream (no atomics: bitwise reproducible).  Where whole units make
// shares that are even enough they are not cut, which saves the second launch.
//
// One CTA per SM (12 warps), two workers per CTA:
//   warp 0     walks the two shares and writes each part of a unit down as a record
//              in shared memory, from which the other roles take their turns; Q
//              tiles and the K ring, by TMA (lanes issue one page each)
//   warp 3     the V ring
//   warp 1     S = Q K^T   (M = 128, N = 128) into the worker's S buffer
//   warp 2     O += P V    (A = P from tensor memory)
//   warps 4-11 one softmax warpgroup per worker; a thread owns a query row.
// Producers and issuers walk the two workers' tiles in turn, so one worker's
// softmax overlaps the other's products.  Tensor memory, d = 64: S 2 x 128
// columns, O 2 x 64, P 2 x 64; d = 128: S 2 x 128, O 2 x 128, and P lies over the
// first half of its own S (the next S product then waits for P V).
// The online softmax keeps a stale maximum: sums are rescaled only when a tile's
// maximum exceeds it by more than 2^8, so P <= 256 and its rounding to bf16
// (relative 2^-8, the operand type of P V) is all that is lost.
// Tiles that every row sees whole take the row's maximum from the load itself; the
// others are masked in registers.  Up to 32 sinks take a tile of 32 columns.
//
// Measured (GB300; fractions of the measured 6.7 TB/s and 2.0 PFLOP/s):
//   B = 8 x 16K, 12 heads of 64, W = 512: 0.307 ms, with 4 sinks 0.340 (2.4 TB/s);
//   W = 2048 0.83 ms; 64K, 16/4 heads of 128, W = 1024, 16 sinks: 0.55-0.58 ms (1.0
//   PFLOP/s, 49%); four chunks of 1.5-2K over 6-16K, 16/4 heads of 128: 0.42 ms
//   (1.37 PFLOP/s, 69%); 32 tokens over caches of 4-33K, 24/8 heads of 128: 0.326 to
//   0.337 ms in a loop, 0.343 to 0.353 with a cold L2 (6.3-6.5 TB/s, 95-97%); a token
//   each of 64 requests, 12 heads of 64, W = 512: 38 us in a graph; one over 777: 12 us.
// What bounds it.  Single tokens over long caches: the cache's bytes.  d = 128 with
// many rows: the chain S -> softmax -> P V of each worker, ~3,200 cycles a pair of
// tiles of which the products fill ~2,450.  d = 64: no unit near its rate (issue slots
// 50%, products 24-30% of the time, exponentials as much of their pipe, L2 23% of its rate);
// what is left is latency: the chain of one tile's softmax, 1,250 to 1,850 cycles for a warp
// that shares its sub-partition with one of the other worker, and the issuing warps' turns.
// The hot code of all roles has to stay in the instruction cache, and is near its end: ~100
// instructions more (a role's loop unrolled over the two workers) cost 25%, 3 KB less gained
// 5 to 8%.
// Tried and not kept: tiles of 64 keys with two or three S buffers a worker (1.3
// to 1.5 times slower: the issuing warps' ~1,000 cycles a turn), two pipelines of own
// control warps a CTA, P V started at half of P, barriers tested ahead of their
// waits, masks skipped for 32 columns that a warp sees whole.
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
using tcx::kLn2;
using tcx::kLog2e;
using tcx::Ring;

constexpr int kThreads = 384;
constexpr int kRegsLaunch = 168;
constexpr int kRegsCtrl = 72;                // (the control roles use 64)
constexpr int kRegsSoftmax = 216;
static_assert(128 * kRegsCtrl + 256 * kRegsSoftmax <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
constexpr int kMaxCtas = 152;              // one per SM; the workspace is sized for them
constexpr int kMaxWorkers = 2 * kMaxCtas;
constexpr float kRescaleLog2 = 8.f;
constexpr uint32_t TMEM_COLS = 512;
constexpr size_t kHalfL2 = 64u << 20;
constexpr int kSmemMax = 232448;

template <int D>
struct Cfg {
    static constexpr int SUB = D / 64;                    // 64-column sub-tiles of a tile
    static constexpr int STILE = 128 * 128;               // bytes of a 128-row sub-tile
    static constexpr int TILE = SUB * STILE;
    static constexpr int QB = D == 64 ? 2 : 1;            // Q buffers a worker
    // (d = 64: a fourth K stage takes 0.203 instead of 0.196 ms at W = 128, and 279 instead of
    // 273 us for one token over 18K)
    static constexpr int KST = D == 64 ? 3 : 2;
    static constexpr int VST = D == 64 ? 6 : 3;
    static constexpr int STAGES = VST;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = 2 * QB * TILE;
    static constexpr int OFF_V = OFF_K + KST * TILE;
    static constexpr int SMEM = OFF_V + VST * TILE + 1024;
    static constexpr uint32_t COL_S = 0;                  // + 128 w
    static constexpr uint32_t COL_O = 256;                // + D w
    static constexpr bool P_OVER_S = D == 128;
    static constexpr uint32_t COL_P = P_OVER_S ? 0 : 384; // + 128 w (over S) or + 64 w
    static constexpr uint32_t P_STEP = P_OVER_S ? 128 : 64;
};

struct FwdArgs {
    SinkSched s;
    __nv_bfloat16* o;
    float* lse;
    float4* part_o;          // [2 * workers][D / 4][R], for R < 1024 / D [2 * workers][R][D / 4]
    float2* part_ml;         // [2 * workers][R]: maximum (log2 units), sum
    int4* tail;              // [workers]: unit (b, mt, h, 1) whose first part this worker holds, or .w = 0
    int* head;               // [workers]: 0, 1 (holds the last part of an earlier worker's unit), 2 (a middle part)
    int R;                   // rows of a query tile: TM * G
    int whole;               // shares end between units: nothing to join
    int* status;
    float scale_log2;
};

// One worker's part of a unit: key tiles j0 .. j1 - 1 (j0 == j1: the share is done).
struct __align__(16) Part {
    int b, h, qrow, ntok;    // sequence, key head, first token's row, tokens of the query tile
    int p0, p1, end;         // positions of the first and the last token, and behind the sequence
    int k0, nsk, nw;         // key tiles: nsk of sinks from 0 on, nw of the window from k0 on
    int j0, j1;
    int f0, f1, fl;          // tiles that every row sees whole: f0 <= j < f1, and j = fl
    int slot;                // -1: the whole unit; else the first of its sums' rows in the workspace
    int nar;                 // key tiles j < nar (one or none) are narrow: 32 columns hold all sinks
    // The sinks come first and the window's first tile, which its edge crosses, last: the
    // crossed tiles then mostly find a running maximum that they need not raise.
    __device__ static __forceinline__ int tile(int j, int nsk, int k0, int nw) {
        const int i = j - nsk + 1;
        return i <= 0 ? j : i == nw ? k0 : k0 + i;
    }
    __device__ __forceinline__ int tile(int j) const { return tile(j, nsk, k0, nw); }
};
constexpr int kParts = 4;    // records a worker
constexpr int kNarrow = 32;  // sinks up to here take a tile of this width (28 us at B = 8 x 16K, a full tile 60)

template <int STAGES>
struct __align__(16) Bars {
    Part part[2][kParts];
    uint64_t part_full[2][kParts], part_empty[2][kParts];
    uint64_t q_full[2][2], q_empty[2][2];
    uint64_t k_full[STAGES], k_empty[STAGES];
    uint64_t v_full[STAGES], v_empty[STAGES];
    uint64_t s_full[2], s_empty[2];
    uint64_t p_full[2], p_empty[2];
    uint64_t o_full[2], o_empty[2];
    uint64_t done, done2;
    uint32_t tmem;
    int error;           // what the CTA has to report, or 0
    StreamPos pos[2];
    int wsum[12], found[4][3];
};

// The next part of a share (one thread); moves `p` behind it.  A part that began in an
// earlier share goes to worker wid's first slot, one that goes on in a later share to
// the second slot of worker wid_tail.
template <bool PAGED>
__device__ __forceinline__ Part next_part(const FwdArgs& a, StreamPos& p, int wid_tail) {
    const SinkSched& s = a.s;
    Part u{};
    if (p.left <= 0) return u;
    SeqInfo q;
    if (!PAGED) {
        q = sink_seq<PAGED>(s, p.b, nullptr);
    } else {
        // to the next query tile that exists: of this head, of the sequence's next one, of a later sequence
#pragma unroll 1
        while (true) {
            if (p.qb != p.b) {
                p.q = sink_seq<PAGED>(s, p.b, nullptr);
                p.qb = p.b;
            }
            q = p.q;
            if (p.mt * s.TM < q.n) break;
            p.mt = 0;
            if (q.n > 0 && ++p.h < s.Hkv) break;
            p.h = 0;
            if (p.b + 1 == s.B) { p.left = 0; return u; }
            ++p.b;
        }
    }
    const KeyTiles k = key_tiles(s, q, p.mt);
    u.b = p.b;
    u.h = p.h;
    u.qrow = q.row0 + p.mt * s.TM;
    u.ntok = min(s.TM, q.n - p.mt * s.TM);
    u.p0 = k.p0;
    u.p1 = k.p1;
    u.end = q.pos0 + q.n;
    u.k0 = k.k0;
    u.nsk = k.nsk;
    u.nw = k.nt - k.nsk;
    u.j0 = p.j;
    u.j1 = min(k.nt, p.j + p.left);
    // whole tiles lie between that of the last row's first key and that of the first row's last
    const int lo = (max(0, k.p1 - s.W + 1) + 127) >> 7, hi = ((k.p0 + 1) >> 7) - 1;
    u.f0 = k.nsk + max(lo - k.k0 - 1, 0);
    u.f1 = min(k.nsk + hi - k.k0, k.nt - 1);
    u.fl = lo <= k.k0 && k.k0 <= hi ? k.nt - 1 : -1;
    u.nar = k.nsk == 1 && s.ns <= kNarrow;
    u.slot = -1;
    if (!a.whole) {                                           // (left whole: there is no workspace to write to)
        if (u.j0 > 0) {
            u.slot = 2 * p.wid * a.R;
            a.head[p.wid] = u.j1 < k.nt ? 2 : 1;              // what the join reads
        } else if (u.j1 < k.nt) {
            u.slot = (2 * wid_tail + 1) * a.R;
            a.tail[wid_tail] = make_int4(p.b, p.mt, p.h, 1);
        }
    }
    p.left -= u.j1 - u.j0;
    p.j = 0;
    if (++p.mt == s.nMT && !PAGED) {
        p.mt = 0;
        if (++p.h == s.Hkv) { p.h = 0; ++p.b; }
    }
    return u;
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(kThreads, 1)
sink_fwd_tc_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                   const __grid_constant__ CUtensorMap tv, const FwdArgs a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
    __shared__ Bars<C::STAGES> sb;
    static_assert(C::SMEM + sizeof(Bars<C::STAGES>) <= kSmemMax, "shared memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const SinkSched& sc = a.s;
    const int down = PAGED ? first_decrease<kThreads>(sc.p, sc.B) : 0;

    if (warp == 0) {                                      // a barrier a lane
        if (lane < 2 * kParts) {
            mbar_init(&sb.part_full[0][lane], 1);
            mbar_init(&sb.part_empty[0][lane], 8);        // both producers, both issuers, 4 softmax warps
        }
        if (lane < 4) {
            mbar_init(&sb.q_full[0][lane], 1);
            mbar_init(&sb.q_empty[0][lane], 1);
        }
        if (lane < 2) {
            mbar_init(&sb.s_full[lane], 1);
            mbar_init(&sb.s_empty[lane], C::P_OVER_S ? 1 : 128);
            mbar_init(&sb.p_full[lane], 128);
            mbar_init(&sb.p_empty[lane], 1);
            mbar_init(&sb.o_full[lane], 1);
            mbar_init(&sb.o_empty[lane], 128);
        }
        if (lane < C::STAGES) {
            mbar_init(&sb.k_full[lane], 1);
            mbar_init(&sb.k_empty[lane], 1);
            mbar_init(&sb.v_full[lane], 1);
            mbar_init(&sb.v_empty[lane], 1);
        }
        if (lane == 0) {
            sb.error = 0;
            mbar_init(&sb.done, 1);
            mbar_init(&sb.done2, 1);
            prefetch_tmap(&tq);
            prefetch_tmap(&tk);
            prefetch_tmap(&tv);
        }
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&sb.tmem, TMEM_COLS);
        tmem_relinquish();
    }
    pdl_release();
    if (PAGED)
        find_shares<kThreads, 2>(ascending_seqs(down, sc.B, sb.wsum, a.status), sc.nMT, sc.Hkv, a.whole, sb.wsum,
                                 sb.found, sb.pos,
                                 [&](int b) { return sink_seq<PAGED>(sc, b, a.status); },
                                 [&](const SeqInfo& q, int mt) { return key_tiles(sc, q, mt).nt; });
    else
        find_shares_dense<kThreads, 2>(sc.B, sc.nMT, sc.Hkv, a.whole, sb.wsum, sb.pos,
                                       [&](int mt) { return key_tiles(sc, SeqInfo{0, sc.L, 0}, mt).nt; });
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sb.tmem;

    // Every role takes the two workers' tiles in turn, in the same order: per turn the next
    // part's record where the last one is used up, then one tile.  A role keeps the
    // state of the worker at hand and of the other one, and swaps them after each turn:
    // its code exists once (the instruction cache holds the whole kernel).
    if (warp < 4) {
    setmaxnreg_dec<kRegsCtrl>();
    auto wait = [&](uint64_t* bar, uint32_t par) { return wait_ctrl(bar, par); };
    auto wwait = [&](uint64_t* bar, uint32_t par) { return __all_sync(0xffffffffu, wait(bar, par)); };
    if (warp == 0 || warp == 3) {
        // ------------------------------------------------------------ producers (whole warps)
        const bool kl = warp == 0;
        struct State {
            int j, j1, np, pg;                                        // next tile, end; parts taken so far; page of this lane's box
            bool open;
        };
        State cur{0, 0, 0, 0, true}, oth = cur;
        Ring rg{0, 0};
        uint64_t* full = kl ? sb.k_full : sb.v_full;
        uint64_t* empty = kl ? sb.k_empty : sb.v_empty;
        const CUtensorMap* map = kl ? &tk : &tv;
        uint8_t* ring = sm + (kl ? C::OFF_K : C::OFF_V);
        const int nst = kl ? C::KST : C::VST;
        const int pages = PAGED ? 128 >> sc.p.page_log2 : 1;       // boxes of a tile, one lane each
        // page id of this lane's box of tile j; n_pages (outside the map: reads as zeros)
        // where no row of the unit sees any of the page
        auto lookup = [&](const Part& u) {
            if (!PAGED || cur.j >= cur.j1 || lane >= pages) return 0;
            const int c0 = u.tile(cur.j) * 128 + (lane << sc.p.page_log2);
            const int c1 = c0 + (1 << sc.p.page_log2) - 1;
            if (c0 > u.p1 || (c1 <= u.p0 - sc.W && c0 >= sc.ns)) return sc.p.n_pages;
            int pg = __ldg(sc.p.table + (size_t)u.b * sc.p.width + (c0 >> sc.p.page_log2));
            if (static_cast<unsigned>(pg) >= static_cast<unsigned>(sc.p.n_pages)) {
                sb.error = GCA_ERR_DEVICE_INDEX;
                pg = sc.p.n_pages;
            }
            return pg;
        };
        bool alternate = false;
        if (kl && lane == 0) {
            for (int i = 0; i < 2 && !a.whole; ++i) {
                a.head[sb.pos[i].wid] = 0;
                a.tail[sb.pos[i].wid] = make_int4(0, 0, 0, 0);
            }
            // Where the tiles that all workers go through for one unit each fill more than
            // half of the L2 cache, the two workers take turns at the units of both shares, neighbours
            // in the sequence, so that one finds the tiles the other has just read (B = 8 x 16K, 12
            // heads of 64, W = 2048: 0.85 instead of 1.22 ms; 64K, 16/4 heads of 128, W = 1024: 0.53
            // instead of 0.65).  Shorter windows stay in the cache anyway, and the workers, whose turns
            // then fall apart, meet fewer slow tiles together (W = 512, ns = 4: 0.37 instead of 0.38).
            // Few units: each worker has its own share, so both end at the same time.
            StreamPos& p = sb.pos[0];
            const int both = p.left + sb.pos[1].left;
            if (sb.pos[1].left > 0) {
                const int nt = key_tiles(sc, sink_seq<PAGED>(sc, p.b, nullptr), p.mt).nt;
                alternate = both >= 16 * nt && (p.j > 0 ? p.left >= nt - p.j : true) &&
                            static_cast<size_t>(nt) * (4 * C::TILE) * gridDim.x > kHalfL2;
                if (alternate) p.left = both;
            }
        }
        uint32_t used = 0;                                            // ring stages ever filled
        int i = 0;
#pragma unroll 1
        for (; cur.open || oth.open; i ^= 1) {
            if (cur.open && cur.j == cur.j1) {
                const int r = cur.np % kParts;
                if (kl) {
                    if (!wwait(&sb.part_empty[i][r], empty_par(cur.np / kParts))) break;
                    if (lane == 0) {
                        sb.part[i][r] = next_part<PAGED>(a, sb.pos[alternate ? 0 : i], sb.pos[alternate ? 1 : i].wid);
                        mbar_arrive(&sb.part_full[i][r]);
                    }
                    __syncwarp();
                } else if (!wwait(&sb.part_full[i][r], full_par(cur.np / kParts))) {
                    break;
                }
                const Part& u = sb.part[i][r];
                cur.j = u.j0;
                cur.j1 = u.j1;
                cur.open = cur.j < cur.j1;
                if (cur.open) {
                    if (kl) {                                         // the unit's Q tile
                        const int qb = cur.np % C::QB;
                        if (!wwait(&sb.q_empty[i][qb], empty_par(cur.np / C::QB))) break;
                        if (lane == 0) {
                            uint8_t* dst = sm + C::OFF_Q + (i * C::QB + qb) * C::TILE;
                            mbar_arrive_expect_tx(&sb.q_full[i][qb], C::SUB * a.R * 128);
#pragma unroll
                            for (int c = 0; c < C::SUB; ++c)
                                tma_load_3d(dst + c * C::STILE, &tq, &sb.q_full[i][qb], c * 64, u.h * sc.G, u.qrow);
                        }
                    }
                    ++cur.np;
                    cur.pg = lookup(u);
                }
            }
            if (cur.open) {
                const Part& u = sb.part[i][(cur.np - 1) % kParts];
                if (!wwait(&empty[rg.i], rg.ph ^ 1u)) break;
                if (lane == 0) mbar_arrive_expect_tx(&full[rg.i], C::TILE);
                __syncwarp();
                if (lane < pages) {
                    uint8_t* dst = ring + rg.i * C::TILE + ((lane << sc.p.page_log2) * (PAGED ? 128 : 0));
                    const int y = PAGED ? 0 : u.tile(cur.j) * 128, z = PAGED ? cur.pg : u.b;
#pragma unroll
                    for (int c = 0; c < C::SUB; ++c)
                        tma_load_3d(dst + c * C::STILE, map, &full[rg.i], u.h * D + c * 64, y, z);
                }
                used |= 1u << rg.i;
                rg.next(nst);
                ++cur.j;
                cur.pg = lookup(u);                                   // a turn ahead of its use
                if (cur.j == cur.j1) {                                // the record is read no more
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sb.part_empty[i][(cur.np - 1) % kParts]);
                }
            }
            const State t = cur;
            cur = oth;
            oth = t;
        }
        if (cur.open || oth.open) sb.error = GCA_ERR_TIMEOUT;
        const int q_loads[2] = {i == 0 ? cur.np : oth.np, i == 0 ? oth.np : cur.np};
        // no copy may still be writing shared memory when the CTA exits: the last load of
        // each buffer has completed its current phase (Q's have, where their products ran;
        // after an abort they are given time)
        if (lane == 0) {
#pragma unroll 1
            for (int i = 0; i < nst; ++i)
                if (used >> i & 1u) wait_copy(&full[i], i < rg.i ? rg.ph : rg.ph ^ 1u);
            if (kl)
#pragma unroll 1
                for (int i = 0; i < 2 * C::QB; ++i) {
                    const int w = i / C::QB, q = i % C::QB;
                    const int n = (q_loads[w] - q + C::QB - 1) / C::QB;      // loads into buffer q
                    if (n > 0) wait_copy(&sb.q_full[w][q], full_par(n - 1));
                }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ S issuer
        if (lane == 0) {
            struct State {
                int j, j1, np, ts, nar;
                bool open;
            };
            State cur{0, 0, 0, 0, 0, true}, oth = cur;
            Ring kv{0, 0};
            bool issued = false;
            const uint32_t id_s = idesc_bf16(128, 128, false, false), id_n = idesc_bf16(128, kNarrow, false, false);
#pragma unroll 1
            for (int i = 0; cur.open || oth.open; i ^= 1) {
                if (cur.open && cur.j == cur.j1) {
                    const int r = cur.np % kParts;
                    if (!wait(&sb.part_full[i][r], full_par(cur.np / kParts))) break;
                    cur.j = sb.part[i][r].j0;
                    cur.j1 = sb.part[i][r].j1;
                    cur.nar = sb.part[i][r].nar;
                    mbar_arrive(&sb.part_empty[i][r]);
                    cur.open = cur.j < cur.j1;
                    if (cur.open) {
                        if (!wait(&sb.q_full[i][cur.np % C::QB], full_par(cur.np / C::QB))) break;
                        ++cur.np;
                    }
                }
                if (cur.open) {
                    const int qb = (cur.np - 1) % C::QB;
                    if (!wait(&sb.k_full[kv.i], kv.ph) || !wait(&sb.s_empty[i], empty_par(cur.ts))) break;
                    tc_fence_after();
                    const uint32_t qaddr = smem_u32(sm + C::OFF_Q + (i * C::QB + qb) * C::TILE);
                    const uint32_t kaddr = smem_u32(sm + C::OFF_K + kv.i * C::TILE);
                    tcx::mma_kmajor_dh<D>(tmem + C::COL_S + i * 128, qaddr, 128, kaddr, 128, cur.j < cur.nar ? id_n : id_s,
                                          0);
                    mma_commit(&sb.s_full[i]);
                    mma_commit(&sb.k_empty[kv.i]);
                    issued = true;
                    ++cur.ts;
                    if (++cur.j == cur.j1) mma_commit(&sb.q_empty[i][qb]);
                    kv.next(C::KST);
                }
                const State t = cur;
                cur = oth;
                oth = t;
            }
            if (cur.open || oth.open) sb.error = GCA_ERR_TIMEOUT;
            if (issued) {
                mma_commit(&sb.done);
                wait_copy(&sb.done, 0);
            }
        }
    } else {
        // ------------------------------------------------------------ P V issuer (whole warp: it also
        // clears the V rows that no token of the unit sees: such rows of the cache may hold anything)
        struct State {
            int j, j1, np, tp, nar, lo, end, nsk, k0, nw;
            bool open;
        };
        State cur{0, 0, 0, 0, 0, 0, 0, 0, 0, 0, true}, oth = cur;
        Ring kv{0, 0};
        bool issued = false;
        const uint32_t id_o = idesc_bf16(128, D, false, true);
#pragma unroll 1
        for (int i = 0; cur.open || oth.open; i ^= 1) {
            bool first = false;
            if (cur.open && cur.j == cur.j1) {
                const int r = cur.np % kParts;
                if (!wwait(&sb.part_full[i][r], full_par(cur.np / kParts))) break;
                const Part& u = sb.part[i][r];
                cur.j = u.j0;
                cur.j1 = u.j1;
                cur.nar = u.nar;
                if (PAGED) {
                    cur.lo = max(u.p0 - sc.W + 1, 0);
                    cur.end = u.end;
                    cur.nsk = u.nsk;
                    cur.k0 = u.k0;
                    cur.nw = u.nw;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sb.part_empty[i][r]);
                cur.open = cur.j < cur.j1;
                if (cur.open) {
                    if (!wwait(&sb.o_empty[i], empty_par(cur.np))) break;
                    ++cur.np;
                    first = true;
                }
            }
            if (cur.open) {
                if (!wwait(&sb.v_full[kv.i], kv.ph)) break;
                uint8_t* vt = sm + C::OFF_V + kv.i * C::TILE;
                if (PAGED) {
                    // Rows that no token of the unit sees are cleared, in pages that hold some that one
                    // does (the other pages were read as zeros): rows a0 .. a1 - 1 between the sinks and
                    // the first token's window, rows a2 .. a3 - 1 behind the last token.
                    const int base = Part::tile(cur.j, cur.nsk, cur.k0, cur.nw) * 128, pg = 1 << sc.p.page_log2;
                    const int edge = cur.lo - base;                   // the tile that the window's edge crosses, or the sinks'
                    auto row = [](int x) { return min(max(x, 0), 128); };
                    const int a0 = row((sc.ns > base ? sc.ns : cur.lo & -pg) - base);
                    const int a1 = row(edge < 128 ? edge : min(((sc.ns + pg - 1) & -pg) - base, cur.j < cur.nar ? kNarrow : 128));
                    const int a2 = row(cur.end - base), a3 = row(((cur.end + pg - 1) & -pg) - base);
                    if (a0 < a1 || a2 < a3) {
                        auto clear = [&](int r0, int r1) {            // rows r0 .. r1 - 1, eight vectors each
#pragma unroll 1
                            for (int r = r0 * 8 + lane; r < r1 * 8; r += 32)
#pragma unroll
                                for (int c = 0; c < C::SUB; ++c)
                                    reinterpret_cast<uint4*>(vt + c * C::STILE)[r] = make_uint4(0, 0, 0, 0);
                        };
                        clear(a0, a1);
                        clear(a2, a3);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                if (!wwait(&sb.p_full[i], full_par(cur.tp))) break;
                const bool narrow = cur.j < cur.nar;
                ++cur.j;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t to = tmem + C::COL_O + i * D, tp = tmem + C::COL_P + i * C::P_STEP;
                    const uint64_t vd = smem_desc(smem_u32(vt), C::STILE, 1024, 2);   // V: keys x D, D along N
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        if (ks == kNarrow / 16 && narrow) break;
                        tc::mma_bf16_ts(to, tp + 8 * ks, vd + 128 * ks, id_o, (first && ks == 0) ? 0u : 1u);
                    }
                    mma_commit(&sb.v_empty[kv.i]);
                    mma_commit(&sb.p_empty[i]);
                    if (C::P_OVER_S) mma_commit(&sb.s_empty[i]);
                    if (cur.j == cur.j1) mma_commit(&sb.o_full[i]);
                }
                issued = true;
                ++cur.tp;
                kv.next(C::VST);
            }
            const State t = cur;
            cur = oth;
            oth = t;
        }
        if (cur.open || oth.open) sb.error = GCA_ERR_TIMEOUT;
        if (issued && elect_one()) {
            mma_commit(&sb.done2);
            wait_copy(&sb.done2, 0);
        }
    }
    } else {
        // ------------------------------------------------------------ softmax + epilogue
        setmaxnreg_inc<kRegsSoftmax>();
        // the accesses after a wait are warp-collective: a wait that gave up in one lane does in all
        auto wwait = [&](uint64_t* bar, uint32_t par) {
            return __all_sync(0xffffffffu, wait_ctrl(bar, par));
        };
        const int wg = (warp - 4) >> 2;
        const int qd = warp & 3;
        const int row = 32 * qd + lane;                 // TMEM lane = query row of the tile
        const int rt = row / sc.G, rg = row - rt * sc.G;
        const uint32_t lane_base = static_cast<uint32_t>(32 * qd) << 16;
        const uint32_t ts_addr = tmem + lane_base + C::COL_S + wg * 128;
        const uint32_t to_addr = tmem + lane_base + C::COL_O + wg * D;
        const uint32_t tp_addr = tmem + lane_base + C::COL_P + wg * C::P_STEP;
        const float sl = a.scale_log2;

        int ts = 0, ko = 0, np = 0, j = 0, j1 = 0, f0 = 0, f1 = 0, fl = 0;
        bool first = true;                              // at the first tile of a part
        bool have = true, live = false, wlive = false;  // a tile to do; this row exists; some row of the warp does
        float m = -INFINITY, l = 0.f;                   // running max (of s * scale * log2(e)) and sum of exp2(. - m)
        // the finished part whose O still sits in tensor memory
        bool pend = false;
        int pend_row = -1;                              // token * H + head, or -1: no such row
        int pend_slot = -1;                             // -1: whole unit; else its sums' first row in the workspace
        float pm = 0.f, pl = 1.f;
        while (true) {
            if (first) {                                // the next part of the share
                const int r = np % kParts;
                if (!wwait(&sb.part_full[wg][r], full_par(np / kParts))) break;
                ++np;
                j = sb.part[wg][r].j0;
                j1 = sb.part[wg][r].j1;
                f0 = sb.part[wg][r].f0;
                f1 = sb.part[wg][r].f1;
                fl = sb.part[wg][r].fl;
                have = j < j1;
                // rows that do not exist are skipped, where a whole warp has no other
                live = have && row < a.R && rt < sb.part[wg][r].ntok;
                wlive = __any_sync(0xffffffffu, live);
            }
            const Part& w = sb.part[wg][(np - 1) % kParts];
            // the previous part's output leaves while the next part's Q and first S are on their way
            if (first && pend) {
                if (!wwait(&sb.o_full[wg], full_par(ko))) break;
                tc_fence_after();
                const bool wr = pend_row >= 0;
                const float inv = pl == 0.f ? 0.f : 1.f / pl;
                if (__any_sync(0xffffffffu, wr)) {
                    if (pend_slot < 0) {
#pragma unroll 1
                        for (int ci = 0; ci < D / 32; ++ci) {
                            uint32_t pk[16];
                            load_rows32(to_addr + 32 * ci, inv, pk);
                            store_rows32(pk, a.o + 32 * ci, D, pend_row);
                        }
                    } else {
#pragma unroll 1
                        for (int ci = 0; ci < D / 16; ++ci) {
                            uint32_t r[16];
                            tmem_ld_32x32b_x16(to_addr + 16 * ci, r);
                            tmem_wait_ld();
                            // (rows side by side: the lanes of a store write 512 consecutive bytes)
                            const int cs = a.R < 1024 / D ? 1 : a.R, rs = a.R < 1024 / D ? D / 4 : 1;
                            uint4* dst = reinterpret_cast<uint4*>(a.part_o) + (size_t)pend_slot * (D / 4) + 4 * ci * cs + row * rs;
                            if (wr)
#pragma unroll
                                for (int u = 0; u < 4; ++u)
                                    dst[u * cs] = make_uint4(r[4 * u], r[4 * u + 1], r[4 * u + 2], r[4 * u + 3]);
                        }
                    }
                    if (wr && pend_slot >= 0) a.part_ml[pend_slot + row] = make_float2(pm, pl);
                    if (wr && pend_slot < 0 && a.lse) a.lse[pend_row] = pl == 0.f ? -INFINITY : (pm + log2f(pl)) * kLn2;
                }
                tc_fence_before();
                mbar_arrive(&sb.o_empty[wg]);
                ++ko;
                pend = false;
            }
            if (!have || !wwait(&sb.s_full[wg], full_par(ts))) break;
            tc_fence_after();
            float alpha = 1.f;
            // the running maximum follows a tile's (in log2 units) only past a margin
            auto follow = [&](float mts) {
                alpha = 1.f;
                if (mts > m + kRescaleLog2) {
                    if (m != -INFINITY) alpha = fast_exp2(m - mts);
                    m = mts;
                }
                l *= alpha;
            };
            // once the previous tile's P V has completed, O is stable and can be rescaled
            auto rescale = [&]() {
                if (__all_sync(0xffffffffu, alpha == 1.f)) return;
                tc_fence_after();
#pragma unroll 1
                for (int ci = 0; ci < D / 16; ++ci) {
                    uint32_t r[16];
                    tmem_ld_32x32b_x16(to_addr + 16 * ci, r);
                    tmem_wait_ld();
#pragma unroll
                    for (int u = 0; u < 16; ++u) r[u] = __float_as_uint(__uint_as_float(r[u]) * alpha);
                    tmem_st_32x32b_x16(to_addr + 16 * ci, r);
                }
                tmem_wait_st();
            };
            if (!wlive) {
                if (!C::P_OVER_S) {
                    mbar_arrive(&sb.s_empty[wg]);
                    if (!wwait(&sb.p_empty[wg], empty_par(ts))) break;
                }
            } else if (j < w.nar) {
                // The narrow tile: all sinks in its first columns, and every row behind them.  (A
                // unit's first tile: no O to rescale.)
                uint32_t r[32], pk[16];
                tmem_ld_32x32b_x32(ts_addr, r);
                tmem_wait_ld();
                tc_fence_before();
                if (!C::P_OVER_S) mbar_arrive(&sb.s_empty[wg]);
                const uint32_t nvis = below(sc.ns);
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    r[i] = (nvis >> i & 1u) ? r[i] : 0xff800000u;
                    m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(r[i]));
                }
                follow(fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * sl);
                float l4[4];
                const uint64_t nsl2 = tcx::f2_pack(sl, sl), nnm2 = tcx::f2_pack(-m, -m);
                uint64_t la[2] = {0ull, 0ull};
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float y0, y1;
                    tcx::f2_unpack(tcx::ffma2(tcx::f2_pack(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])),
                                              nsl2, nnm2), y0, y1);
                    const uint64_t e = tcx::f2_pack(fast_exp2(y0), fast_exp2(y1));
                    la[i & 1] = tcx::fadd2(la[i & 1], e);
                    pk[i] = tcx::pack_bf16x2(e);
                }
                tcx::f2_unpack(la[0], l4[0], l4[1]);
                tcx::f2_unpack(la[1], l4[2], l4[3]);
                l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
                if (!C::P_OVER_S && !wwait(&sb.p_empty[wg], empty_par(ts))) break;
                tmem_st_32x32b_x16(tp_addr, pk);
                tmem_wait_st();
            } else {
                // The row of S into registers at once, the maximum from the load.
                float x[128];
                {
                    uint32_t r[2][64];
                    float mc[2];
#pragma unroll
                    for (int ci = 0; ci < 2; ++ci) mc[ci] = tmem_ld_max_32x32b_x64(ts_addr + 64 * ci, r[ci]);
                    tmem_wait_ld();
#pragma unroll
                    for (int ci = 0; ci < 2; ++ci)
#pragma unroll
                        for (int u = 0; u < 64; ++u) x[64 * ci + u] = __uint_as_float(r[ci][u]);
                    tc_fence_before();
                    if (!C::P_OVER_S) mbar_arrive(&sb.s_empty[wg]);
                    float mt = fmaxf(mc[0], mc[1]);
                    if (!((j >= f0 && j < f1) || j == fl)) {
                        // The diagonal or the window's edge crosses the tile.  Visible: columns c_lo ..
                        // c_hi (the window) and those below c_s (sinks), as bits.
                        const int p = w.p0 + rt, kbase = w.tile(j) * 128;
                        const int c_lo = p - sc.W + 1 - kbase, c_hi = p - kbase, c_s = min(sc.ns, p + 1) - kbase;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t vis = (below(c_hi + 1 - 32 * c) & ~below(c_lo - 32 * c)) | below(c_s - 32 * c);
#pragma unroll
                            for (int u = 0; u < 32; ++u) x[32 * c + u] = (vis >> u & 1u) ? x[32 * c + u] : -INFINITY;
                        }
                        // the maximum over all columns bounds that over the visible ones: only where it
                        // would move the running one (or is no number) is the latter needed
                        if (__any_sync(0xffffffffu, !(mt * sl <= m + kRescaleLog2))) {
                            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                            for (int i = 0; i < 128; ++i) m4[i & 3] = fmaxf(m4[i & 3], x[i]);
                            mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                        }
                    }
                    follow(mt * sl);
                }
                const float mu = m == -INFINITY ? 0.f : m;
                const uint64_t sl2 = tcx::f2_pack(sl, sl), nmu2 = tcx::f2_pack(-mu, -mu);
                uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
                uint32_t pka[32];                       // the first 64 keys' P, formed before the wait for the P buffer
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    float y0, y1;
                    tcx::f2_unpack(tcx::ffma2(tcx::f2_pack(x[2 * c], x[2 * c + 1]), sl2, nmu2), y0, y1);
                    const float e0 = fast_exp2(y0);
                    const float e1 = fast_exp2(y1);
                    acc2[c & 3] = tcx::fadd2(acc2[c & 3], tcx::f2_pack(e0, e1));
                    pka[c] = tcx::pack_bf16(e0, e1);
                }
                // the previous tile's P V has completed: O is stable, the P buffer free
                // (P over S: already so, since this tile's S product waited for it)
                if (!C::P_OVER_S && !wwait(&sb.p_empty[wg], empty_par(ts))) break;
                rescale();
                {
                    uint32_t h0[16], h1[16];
#pragma unroll
                    for (int u = 0; u < 16; ++u) { h0[u] = pka[u]; h1[u] = pka[16 + u]; }
                    tmem_st_32x32b_x16(tp_addr, h0);
                    tmem_st_32x32b_x16(tp_addr + 16, h1);
                }
                uint32_t pk2[16];
#pragma unroll
                for (int c = 4; c < 8; ++c) {
                    uint32_t pk[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        float y0, y1;
                        const uint64_t s2 = tcx::f2_pack(x[16 * c + 2 * u], x[16 * c + 2 * u + 1]);
                        tcx::f2_unpack(tcx::ffma2(s2, sl2, nmu2), y0, y1);
                        const float e0 = fast_exp2(y0);
                        const float e1 = fast_exp2(y1);
                        acc2[u & 3] = tcx::fadd2(acc2[u & 3], tcx::f2_pack(e0, e1));
                        pk[u] = tcx::pack_bf16(e0, e1);
                    }
                    if (c & 1) {
#pragma unroll
                        for (int u = 0; u < 8; ++u) pk2[8 + u] = pk[u];
                        tmem_st_32x32b_x16(tp_addr + 16 * (c >> 1), pk2);
                    } else {
#pragma unroll
                        for (int u = 0; u < 8; ++u) pk2[u] = pk[u];
                    }
                }
                tmem_wait_st();
                float l4[8];
#pragma unroll
                for (int u = 0; u < 4; ++u) tcx::f2_unpack(acc2[u], l4[2 * u], l4[2 * u + 1]);
                l += ((l4[0] + l4[1]) + (l4[2] + l4[3])) + ((l4[4] + l4[5]) + (l4[6] + l4[7]));
            }
            tc_fence_before();
            mbar_arrive(&sb.p_full[wg]);
            ++ts;
            first = ++j == j1;
            if (first) {                                // this part of the unit is done: it leaves later
                pend = true;
                pend_row = live ? (w.qrow + rt) * sc.H + w.h * sc.G + rg : -1;
                pend_slot = w.slot;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sb.part_empty[wg][(np - 1) % kParts]);
                pm = m;
                // (a row that sees keys has a sum above 0, or scores that are no numbers or all -inf: NaN then)
                pl = l == 0.f && w.slot < 0 && w.p0 + rt >= 0 ? NAN : l;
                m = -INFINITY;
                l = 0.f;
            }
        }
        if (have) sb.error = GCA_ERR_TIMEOUT;
    }

    tc_fence_before();
    __syncthreads();
    // (one report a CTA: with one at each wait the code grew by 3 KB and the kernel took 5% longer)
    if (threadIdx.x == 0 && sb.error) set_status(a.status, sb.error);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Joins the parts of the units that were cut (3 us after the forward, most of it launch: at most 303
// units of 128 rows are cut): blocks (w, *) the unit that begins in worker
// w's share and continues in the next ones.  With m = max_i m_i,
//   o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i, in the order of the stream.
// A thread has four columns of a row; a block 16 rows (d = 64) or 8.
template <int D, bool PAGED>
__global__ void __launch_bounds__(256) sink_join_kernel(const FwdArgs a, int workers) {
    pdl_wait();
    const int w = blockIdx.x;
    const int4 u = a.tail[w];
    if (u.w == 0) return;
    const int n = parts_of(a.head, w, workers);
    const SinkSched& sc = a.s;
    const SeqInfo s = sink_seq<PAGED>(sc, u.x, nullptr);
    constexpr int VEC = D / 4;
    constexpr int ROWS = 256 / VEC;
    const bool few = a.R < ROWS;                        // (one block: its lanes along the columns)
    const int row = blockIdx.y * ROWS + (few ? threadIdx.x / VEC : threadIdx.x % ROWS);
    const int c = few ? threadIdx.x % VEC : threadIdx.x / ROWS;
    const int rt = row / sc.G, t = u.y * sc.TM + rt;
    if (row >= a.R || t >= s.n) return;
    const auto slot = [&](int k) { return (size_t)(k == 0 ? 2 * w + 1 : 2 * (w + k)) * a.R; };   // first row of its sums
    float m = -INFINITY;
#pragma unroll 4
    for (int k = 0; k < n; ++k) m = fmaxf(m, a.part_ml[slot(k) + row].x);
    const float mu = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < n; ++k) {
        const float2 ml = a.part_ml[slot(k) + row];
        const float4 o = a.part_o[slot(k) * VEC + (few ? row * VEC + c : c * a.R + row)];
        const float f = fast_exp2(ml.x - mu);
        acc.x = fmaf(o.x, f, acc.x);
        acc.y = fmaf(o.y, f, acc.y);
        acc.z = fmaf(o.z, f, acc.z);
        acc.w = fmaf(o.w, f, acc.w);
        l = fmaf(ml.y, f, l);
    }
    if (l == 0.f && s.pos0 + t >= 0) l = NAN;           // as in the forward
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const long long orow = (long long)(s.row0 + t) * sc.H + u.z * sc.G + (row - rt * sc.G);
    reinterpret_cast<uint2*>(a.o + orow * D)[c] =
        make_uint2(tcx::pack_bf16(acc.x * inv, acc.y * inv), tcx::pack_bf16(acc.z * inv, acc.w * inv));
    if (c == 0 && a.lse) a.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

int rows_of_tile(const SinkShape& s, int* tm) {
    const int G = s.H / s.Hkv;
    int t = 128 / G;
    if (t > s.max_q) t = s.max_q;
    *tm = t;
    return t * G;
}

struct Layout {
    size_t o_off, ml_off, tail_off, head_off, total;
};
Layout layout(const SinkShape& s) {
    int tm;
    const size_t R = rows_of_tile(s, &tm);
    Layout w;
    w.o_off = 0;
    w.ml_off = w.o_off + (size_t)2 * kMaxWorkers * R * s.d * 4;
    w.tail_off = (w.ml_off + (size_t)2 * kMaxWorkers * R * 8 + 255) / 256 * 256;
    w.head_off = w.tail_off + kMaxWorkers * 16;
    w.total = (w.head_off + kMaxWorkers * 4 + 255) / 256 * 256;
    return w;
}

// Are the units left whole?
bool whole_units(const SinkShape& s) {
    int tm;
    const int R = rows_of_tile(s, &tm);
    // Cutting units costs a join and sums in the workspace, the time of some C tiles by the measurements;
    // leaving them whole costs the difference between the longest share and the mean.  (312 units of 15
    // tiles, 12 heads of 64: 28.4 us whole, 33.1 cut; 308 of 17, 16/4 heads of 128: 34.6 and 43.4; B =
    // 8 x 16K, W = 512, 4 sinks: 0.339 and 0.348 ms; a token of 4 x 128 columns over 7 tiles: 16.7 and
    // 11.3 us.)  C is fitted to these and to a few shapes around them, not derived.  Few tiles a unit only:
    // ragged lengths make shares of whole units less even than this counts.
    const long long span = (long long)s.W + tm - 1;
    const long long keys = s.paged ? (long long)s.width * s.page : s.L;
    const long long nt = span < keys ? (span + 126) / 128 + 1 + (s.ns + 127) / 128 : (keys + 127) / 128;
    const long long pairs = (long long)s.B * ((s.max_q + tm - 1) / tm), packed = (long long)s.T / tm + s.B;
    const long long units = s.Hkv * (s.paged && packed < pairs ? packed : pairs);
    const long long C = (s.d == 64 ? 6 : 3) + R * s.d / 896;
    return nt <= 2 * C + 2 && (units + kMaxWorkers - 1) / kMaxWorkers * nt * kMaxWorkers <= units * nt + C * kMaxWorkers;
}

template <int D, bool PAGED>
cudaError_t launch(const FwdArgs& a, const CUtensorMap& tq, const CUtensorMap& tk,
                   const CUtensorMap& tv, cudaStream_t st, int* launches) {
    using C = Cfg<D>;
    static LaunchSetup setup;
    int sms = 0;
    cudaError_t e = setup.once(
        [] {
            // the setmaxnreg split needs the whole launch allocation: refuse to launch a build that
            // gave the kernel fewer registers a thread (its warps would wait forever)
            cudaFuncAttributes fa;
            const cudaError_t r = cudaFuncGetAttributes(&fa, sink_fwd_tc_kernel<D, PAGED>);
            if (r != cudaSuccess) return r;
            if (fa.numRegs * kThreads < 128 * kRegsCtrl + 256 * kRegsSoftmax) return cudaErrorInvalidConfiguration;
            return cudaFuncSetAttribute(sink_fwd_tc_kernel<D, PAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        },
        &sms);
    if (e != cudaSuccess) return e;
    const int grid = sms < kMaxCtas ? sms : kMaxCtas;
    GCA_LAUNCH("sink_fwd_tc", st, sink_fwd_tc_kernel<D, PAGED><<<grid, kThreads, C::SMEM, st>>>(tq, tk, tv, a));
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    *launches += 1;
    if (a.whole) return e;
    const int rows = 1024 / D;
    GCA_LAUNCH("sink_join", st,
               e = launch_pdl(sink_join_kernel<D, PAGED>, dim3(2 * grid, (a.R + rows - 1) / rows), 256, 0, st, a, 2 * grid));
    if (e == cudaSuccess) *launches += 1;
    return e;
}

}  // namespace

size_t sink_fwd_workspace_bytes(const SinkShape& s) { return whole_units(s) ? 256 : layout(s).total; }

bool sink_fwd_supported(const SinkShape& s) {
    // the kernel counts key tiles and (sequence, query tile) pairs in 32 bits; quota * workers
    // may pass the total by one share
    int tm;
    rows_of_tile(s, &tm);
    const double nmt = (s.max_q + tm - 1) / tm;
    const double vis = (double)s.W + tm + s.ns;
    if (s.B * nmt >= 1e9) return false;
    if (!s.paged) return s.B * s.Hkv * causal_sum(nmt, tm / 128.0, vis / 128 + 3) < kMaxSteps;
    const double keys = (double)s.width * s.page, units = (double)s.T / tm + s.B;
    return units * s.Hkv * (std::min(vis, keys) / 128 + 3) < kMaxSteps;
}

cudaError_t launch_sink_fwd(const SinkShape& s, const void* q, const void* k, const void* v,
                            const int32_t* cu_q, const int32_t* kv_len, const int32_t* table, void* o,
                            float* lse, void* ws, int* status, cudaStream_t st, int* launches) {
    FwdArgs a{};
    a.s.B = s.B; a.s.L = s.L; a.s.H = s.H; a.s.Hkv = s.Hkv; a.s.G = s.H / s.Hkv;
    a.s.W = s.W; a.s.ns = s.ns;
    a.R = rows_of_tile(s, &a.s.TM);
    a.s.nMT = (s.max_q + a.s.TM - 1) / a.s.TM;
    if (s.paged) a.s.p = PagedArgs{cu_q, kv_len, table, s.T, s.max_q, __builtin_ctz(s.page), s.n_pages, s.width};
    if (!sink_fwd_supported(s)) return cudaErrorInvalidConfiguration;
    const Layout w = layout(s);
    uint8_t* base = static_cast<uint8_t*>(ws);
    a.part_o = reinterpret_cast<float4*>(base + w.o_off);
    a.part_ml = reinterpret_cast<float2*>(base + w.ml_off);
    a.tail = reinterpret_cast<int4*>(base + w.tail_off);
    a.head = reinterpret_cast<int*>(base + w.head_off);
    a.o = static_cast<__nv_bfloat16*>(o);
    a.lse = lse;
    a.status = status;
    a.scale_log2 = s.scale * kLog2e;
    a.whole = whole_units(s);
    CUtensorMap tq, tk, tv;
    const uint64_t kvcols = (uint64_t)s.Hkv * s.d;
    bool ok = encode_bf16_3d(&tq, q, s.d, s.H, s.T, s.d, s.q_stride, a.s.G, a.s.TM);
    // (d = 64: a head's row is 128 bytes, and 256-byte L2 fetches would bring a neighbour head's row
    // that another CTA reads at another time: one token over 18K, 12 heads: 0.39 -> 0.28 ms)
    for (int i = 0; i < 2; ++i) {
        CUtensorMap* m = i ? &tv : &tk;
        const void* p = i ? v : k;
        ok = ok && (s.paged ? encode_bf16_3d(m, p, kvcols, s.page, s.n_pages, kvcols, kvcols * s.page, s.page, 1, s.d == 128)
                            : encode_bf16_3d(m, p, kvcols, s.L, s.B, s.kv_stride, (uint64_t)s.kv_stride * s.L, 128, 1, s.d == 128));
    }
    if (!ok) return cudaErrorInvalidValue;
    if (s.paged)
        return s.d == 64 ? launch<64, true>(a, tq, tk, tv, st, launches)
                         : launch<128, true>(a, tq, tk, tv, st, launches);
    return s.d == 64 ? launch<64, false>(a, tq, tk, tv, st, launches)
                     : launch<128, false>(a, tq, tk, tv, st, launches);
}

}  // namespace gca
