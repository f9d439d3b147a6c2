// rope.cu -- rotary positions of queries and keys (gca_rope), and the same on the
// way into the paged K/V cache (gca_paged_rope_append).
//
// Pair i of a head, (x, y), is turned by the angle p f_i of its token's position p:
//   x' = m (x cos - y sin),  y' = m (x sin + y cos),
// the pairs being (i, i + rot/2) of the first `rot` columns, or (2 i, 2 i + 1).  The gradient
// is the turn by the negative angle.
//
// The angle.  p f_i in fp32 is off by 2^-24 p f_i: a hundredth of a radian at p = 2^18.  The
// table holds f_i / (2 pi) as a fraction of a turn in units of 2^-64, so the product
// with an integer position, modulo 2^64, is the angle modulo a turn, exactly; its upper 32
// bits go on.  bf16 takes the hardware's sine and cosine (off by 2^-21 within half a turn, the
// results' own rounding is 2^-9); fp32 reduces to an eighth of a turn first.
//
// Work.  A slot is 16 columns of a head whose pairs belong together (8 and 8 columns rot/2
// apart, or 16 neighbours), two 16-byte vectors of bf16, owned by one thread, so a tensor may be
// turned in place.  A lane has the same slot of every head it meets (32 / (d/16) heads a step): it
// forms its eight sines and cosines once a token.  A warp has up to kSteps steps of a token, all
// loaded before the angles are formed.
//
// Measured (GB300): 8 x 16K tokens, 12/12 heads of 64, bf16: 115 us, at the copy rate (0.40 GB read and as
// much written, of which 0.34 reach memory within the kernel); 517 tokens 2.3 us.  Into the cache: eight
// chunks of 0.9-2K, 12/12 heads of 64: 19.5 us (6.0 TB/s, 89% of the copy rate); a token each of 64 requests,
// 24/8 heads of 128: 3.0 us.  Bound by memory; the write to the cache also by the chain of a row's
// sequence, its page and the store, which more warps a row lengthen (two steps a warp: 24 us).
#include "attn_sink.cuh"
#include "kernels.h"

namespace gca {
namespace {

constexpr int kThreads = 128;
// Steps of 32 slots that a warp takes at most (by its registers).  A kernel has as many as it takes: with
// room for five, three steps are 5% slower (8 x 16K, 12/12 heads of 64: 127 instead of 121 us).
template <class T>
constexpr int kSteps = sizeof(T) == 2 ? 5 : 3;

// Sine and cosine of `a` units of 2^-32 turns.
template <class T>
__device__ __forceinline__ void sin_cos(int a, float& s, float& c) {
    if constexpr (sizeof(T) == 2) {
        const float r = static_cast<float>(a) * 1.4629180792671596e-9f;      // 2 pi 2^-32
        s = __sinf(r);
        c = __cosf(r);
    } else {
        const unsigned q = (static_cast<unsigned>(a) + 0x20000000u) >> 30;   // the nearest quarter turn
        float u, v;
        sincospif(static_cast<float>(static_cast<int>(static_cast<unsigned>(a) - (q << 30))) * 0x1p-31f, &u, &v);
        s = q & 1 ? v : u;
        c = q & 1 ? u : v;
        if (q & 2) s = -s;
        if ((q + 1) & 2) c = -c;
    }
}

struct Turn {
    float s[8], c[8];
};

// Slot j's eight pairs at position p.
template <class T>
__device__ __forceinline__ void angles(const uint64_t* freqs, int j, int p, float m, bool inverse, Turn& t) {
    const ulonglong2* f = reinterpret_cast<const ulonglong2*>(freqs + 8 * j);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const ulonglong2 x = __ldg(f + i);
        const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(p));
        sin_cos<T>(static_cast<int>((x.x * pos) >> 32), t.s[2 * i], t.c[2 * i]);
        sin_cos<T>(static_cast<int>((x.y * pos) >> 32), t.s[2 * i + 1], t.c[2 * i + 1]);
    }
    const float ms = inverse ? -m : m;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        t.s[i] *= ms;
        t.c[i] *= m;
    }
}

// Eight columns.
template <class T>
struct Vec {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void store(T* p) const {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        if constexpr (sizeof(T) == 2) {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[4 * i] = __uint_as_float(v[i].x);
                x[4 * i + 1] = __uint_as_float(v[i].y);
                x[4 * i + 2] = __uint_as_float(v[i].z);
                x[4 * i + 3] = __uint_as_float(v[i].w);
            }
        }
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
        if constexpr (sizeof(T) == 2) {
            v[0] = make_uint4(tcx::pack_bf16(x[0], x[1]), tcx::pack_bf16(x[2], x[3]), tcx::pack_bf16(x[4], x[5]),
                              tcx::pack_bf16(x[6], x[7]));
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                v[i] = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                                  __float_as_uint(x[4 * i + 3]));
        }
    }
};

// Turns a slot's two vectors: pairs (a_i, b_i), or neighbours within a and within b.
template <class T, bool INTER>
__device__ __forceinline__ void turn(Vec<T>& a, Vec<T>& b, const Turn& t) {
    float x[8], y[8], u[8], w[8];
    a.get(x);
    b.get(y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (INTER) {
            float* z = i < 4 ? x : y;
            float* r = i < 4 ? u : w;
            const int k = 2 * (i & 3);
            r[k] = z[k] * t.c[i] - z[k + 1] * t.s[i];
            r[k + 1] = z[k] * t.s[i] + z[k + 1] * t.c[i];
        } else {
            u[i] = x[i] * t.c[i] - y[i] * t.s[i];
            w[i] = x[i] * t.s[i] + y[i] * t.c[i];
        }
    }
    a.set(u);
    b.set(w);
}

// Columns of slot j's two vectors.
template <bool INTER>
__device__ __forceinline__ void columns(int j, int rot, int& a, int& b) {
    const bool halves = !INTER && 16 * j < rot;
    a = halves ? 8 * j : 16 * j;
    b = halves ? rot / 2 + 8 * j : 16 * j + 8;
}

struct RopeArgs {
    const void *q, *k;
    void *qo, *ko;
    const uint64_t* freqs;
    const int32_t* pos;      // [T], or null: start + t % L
    int T, L, start, H, Hkv, d, rot;
    int qs, ks, qos, kos;    // elements between tokens
    int slots;               // of a token: (H + Hkv) d / 16
    int log2_n;              // of d / 16
    int units;               // warps a token
    float m;
    int inverse;
};

template <class T, bool INTER, int STEPS>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a) {
    const int lane = threadIdx.x & 31;
    const long long unit = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const long long t = unit / a.units;
    if (t >= a.T) return;
    const int first = static_cast<int>(unit - t * a.units) * (32 * STEPS) + lane;
    const int j = first & ((1 << a.log2_n) - 1);                 // the same in every step
    int ca, cb;
    columns<INTER>(j, a.rot, ca, cb);
    auto at = [&](int i, const void* q, const void* k, int qs, int ks) -> T* {
        const int h = (first + 32 * i) >> a.log2_n;
        const T* p = h < a.H ? static_cast<const T*>(q) + (size_t)t * qs + (size_t)h * a.d
                             : static_cast<const T*>(k) + (size_t)t * ks + (size_t)(h - a.H) * a.d;
        return const_cast<T*>(p);
    };
    Vec<T> x[STEPS], y[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        if (first + 32 * i < a.slots) {
            const T* p = at(i, a.q, a.k, a.qs, a.ks);
            x[i].load(p + ca);
            y[i].load(p + cb);
        }
    if (16 * j < a.rot) {
        Turn tn;
        angles<T>(a.freqs, j, a.pos ? __ldg(a.pos + t) : a.start + static_cast<int>(t % a.L), a.m, a.inverse, tn);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) turn<T, INTER>(x[i], y[i], tn);
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        if (first + 32 * i < a.slots) {
            T* p = at(i, a.qo, a.ko, a.qos, a.kos);
            x[i].store(p + ca);
            y[i].store(p + cb);
        }
}

struct AppendArgs {
    PagedArgs p;
    const __nv_bfloat16 *q, *k, *v;
    __nv_bfloat16 *qo, *kc, *vc;
    const uint64_t* freqs;
    int B, H, Hkv, d, rot, qs, kvs, slots, log2_n, units;
    float m;
    int* status;
};

// Slots of a row: its queries', its keys', its values'.
template <bool INTER, int STEPS>
__global__ void __launch_bounds__(kThreads) paged_rope_append_kernel(const AppendArgs a) {
    using T = __nv_bfloat16;
    const int lane = threadIdx.x & 31;
    const long long tid = (long long)blockIdx.x * kThreads + threadIdx.x;
    // contradicting entries are reported whether a row belongs to them or not
    for (long long b = tid; b < a.B; b += (long long)gridDim.x * kThreads) paged_seq(a.p, (int)b, a.status);
    const long long unit = tid >> 5, row = unit / a.units;
    if (row >= a.p.T) return;
    const int first = static_cast<int>(unit - row * a.units) * (32 * STEPS) + lane;
    const int j = first & ((1 << a.log2_n) - 1);
    int ca, cb;
    columns<INTER>(j, a.rot, ca, cb);
    Vec<T> x[STEPS], y[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        if (first + 32 * i < a.slots) {
            const int h = (first + 32 * i) >> a.log2_n;
            const T* p = h < a.H ? a.q + row * a.qs + (size_t)h * a.d
                         : h < a.H + a.Hkv ? a.k + row * a.kvs + (size_t)(h - a.H) * a.d
                                           : a.v + row * a.kvs + (size_t)(h - a.H - a.Hkv) * a.d;
            const bool val = h >= a.H + a.Hkv;                    // (values are copied as they are)
            x[i].load(p + (val ? 16 * j : ca));
            y[i].load(p + (val ? 16 * j + 8 : cb));
        }
    int pos;
    const int seq = seq_of_row(a.p, a.B, static_cast<int>(row), &pos);
    if (seq < 0) return;
    // the row's place in the cache, or -1: no such place
    long long dst = -1;
    if (pos >= 0) {
        const int pg = __ldg(a.p.table + (size_t)seq * a.p.width + (pos >> a.p.page_log2));
        if (static_cast<unsigned>(pg) < static_cast<unsigned>(a.p.n_pages))
            dst = ((long long)pg << a.p.page_log2) + (pos & ((1 << a.p.page_log2) - 1));
        else if (lane == 0)
            set_status(a.status, GCA_ERR_DEVICE_INDEX);
    }
    Turn tn;
    if (16 * j < a.rot) angles<T>(a.freqs, j, pos, a.m, false, tn);
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
        if (first + 32 * i < a.slots) {
            const int h = (first + 32 * i) >> a.log2_n;
            const bool val = h >= a.H + a.Hkv;
            if (!val && 16 * j < a.rot) turn<T, INTER>(x[i], y[i], tn);
            if (h >= a.H && dst < 0) continue;
            T* p = h < a.H ? a.qo + ((size_t)row * a.H + h) * a.d
                   : val   ? a.vc + ((size_t)dst * a.Hkv + (h - a.H - a.Hkv)) * a.d
                           : a.kc + ((size_t)dst * a.Hkv + (h - a.H)) * a.d;
            x[i].store(p + (val ? 16 * j : ca));
            y[i].store(p + (val ? 16 * j + 8 : cb));
        }
}

// Steps a warp: as few warps a token as max_steps allows, with equally many steps (12/12 heads of 64 into
// the cache: 144 slots, one warp of five steps), and more warps where all of them would be less than four
// an SM (a token each of 64 requests, 24/8 heads of 128: 3.1 instead of 3.5 us).
int steps_of(int T, int slots, int max_steps) {
    const int n = (slots + 31) / 32;
    const int per = static_cast<int>(std::min<long long>(max_steps, std::max<long long>(1, (long long)T * n / (4 * 152))));
    const int units = (n + per - 1) / per;
    return (n + units - 1) / units;
}

template <class T, int STEPS>
void launch_steps(const RopeArgs& a, bool inter, unsigned blocks, cudaStream_t st) {
    if (inter) rope_kernel<T, true, STEPS><<<blocks, kThreads, 0, st>>>(a);
    else rope_kernel<T, false, STEPS><<<blocks, kThreads, 0, st>>>(a);
}
template <int STEPS>
void launch_steps(const AppendArgs& a, bool inter, unsigned blocks, cudaStream_t st) {
    if (inter) paged_rope_append_kernel<true, STEPS><<<blocks, kThreads, 0, st>>>(a);
    else paged_rope_append_kernel<false, STEPS><<<blocks, kThreads, 0, st>>>(a);
}

unsigned blocks_of(int T, int units) {
    return static_cast<unsigned>(((long long)T * units + kThreads / 32 - 1) / (kThreads / 32));
}

}  // namespace

cudaError_t launch_rope(const RopeShape& s, const void* q, const void* k, const int64_t* freqs,
                        const int32_t* positions, void* q_out, void* k_out, cudaStream_t st,
                        int* launches) {
    RopeArgs a{};
    a.q = q; a.k = k; a.qo = q_out; a.ko = k_out;
    a.freqs = reinterpret_cast<const uint64_t*>(freqs);
    a.pos = positions;
    a.T = s.T; a.L = s.L; a.start = s.start; a.H = s.H; a.Hkv = s.Hkv; a.d = s.d; a.rot = s.rot;
    a.qs = s.q_stride; a.ks = s.k_stride; a.qos = s.qo_stride; a.kos = s.ko_stride;
    a.log2_n = __builtin_ctz(s.d / 16);
    a.slots = (s.H + s.Hkv) << a.log2_n;
    a.m = s.mscale;
    a.inverse = s.inverse;
    const bool half = s.dtype == GCA_BF16;
    const int steps = steps_of(s.T, a.slots, half ? kSteps<__nv_bfloat16> : kSteps<float>);
    a.units = (a.slots + 32 * steps - 1) / (32 * steps);
    const unsigned n = blocks_of(s.T, a.units);
    GCA_LAUNCH("rope", st, {
        if (!half) {
            if (steps == 1) launch_steps<float, 1>(a, s.interleaved, n, st);
            else if (steps == 2) launch_steps<float, 2>(a, s.interleaved, n, st);
            else launch_steps<float, 3>(a, s.interleaved, n, st);
        } else {
            using T = __nv_bfloat16;
            if (steps == 1) launch_steps<T, 1>(a, s.interleaved, n, st);
            else if (steps == 2) launch_steps<T, 2>(a, s.interleaved, n, st);
            else if (steps == 3) launch_steps<T, 3>(a, s.interleaved, n, st);
            else if (steps == 4) launch_steps<T, 4>(a, s.interleaved, n, st);
            else launch_steps<T, 5>(a, s.interleaved, n, st);
        }
    });
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *launches += 1;
    return e;
}

cudaError_t launch_paged_rope_append(const SinkShape& s, const RopeShape& r, const void* q, const void* k_new,
                                     const void* v_new, const int64_t* freqs, const int32_t* cu_q,
                                     const int32_t* kv_len, const int32_t* table, void* q_out, void* k_cache,
                                     void* v_cache, int* status, cudaStream_t st, int* launches) {
    AppendArgs a{};
    a.p = PagedArgs{cu_q, kv_len, table, s.T, s.max_q, __builtin_ctz(s.page), s.n_pages, s.width};
    using T = __nv_bfloat16;
    a.q = static_cast<const T*>(q); a.k = static_cast<const T*>(k_new); a.v = static_cast<const T*>(v_new);
    a.qo = static_cast<T*>(q_out); a.kc = static_cast<T*>(k_cache); a.vc = static_cast<T*>(v_cache);
    a.freqs = reinterpret_cast<const uint64_t*>(freqs);
    a.B = s.B; a.H = s.H; a.Hkv = s.Hkv; a.d = s.d; a.rot = r.rot;
    a.qs = s.q_stride; a.kvs = s.kv_stride;
    a.log2_n = __builtin_ctz(s.d / 16);
    a.slots = (s.H + 2 * s.Hkv) << a.log2_n;
    a.m = r.mscale;
    a.status = status;
    const int steps = steps_of(s.T, a.slots, kSteps<T>);
    a.units = (a.slots + 32 * steps - 1) / (32 * steps);
    const unsigned n = blocks_of(s.T, a.units);
    GCA_LAUNCH("paged_rope_append", st, {
        if (steps == 1) launch_steps<1>(a, r.interleaved, n, st);
        else if (steps == 2) launch_steps<2>(a, r.interleaved, n, st);
        else if (steps == 3) launch_steps<3>(a, r.interleaved, n, st);
        else if (steps == 4) launch_steps<4>(a, r.interleaved, n, st);
        else launch_steps<5>(a, r.interleaved, n, st);
    });
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *launches += 1;
    return e;
}

}  // namespace gca
