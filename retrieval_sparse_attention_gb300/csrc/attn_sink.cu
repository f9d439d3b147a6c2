// attn_sink.cu -- gradients of the windowed self-attention with sinks in fp32
// arithmetic on the CUDA cores.
//
// One warp per (token, query head) for dQ
// and one per (token, key head) for dK and dV, over the tokens that see the key.
#include <math.h>

#include "attn_sink.cuh"
#include "kernels.h"
#include "tc_common.cuh"

namespace gca {
namespace {

using bf16 = __nv_bfloat16;

struct Args {
    const bf16 *q, *k, *v;
    int B, L, H, Hkv, W, ns, q_stride, kv_stride;
    float scale;
    int paged;
    PagedArgs p;
    bf16* o;
    float* lse;
    int* status;
};

template <int D>
__device__ __forceinline__ float dot(const float* a, const bf16* b) {
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        const uint4 x = reinterpret_cast<const uint4*>(b)[c];
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&x);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float2 f = __bfloat1622float2(h[u]);
            s = fmaf(a[8 * c + 2 * u], f.x, fmaf(a[8 * c + 2 * u + 1], f.y, s));
        }
    }
    return s;
}

// Visible keys of position p in order: sinks in front of the window, then the window.
struct Keys {
    int n_sink, lo, n;
    __device__ Keys(int p, int W, int ns) {
        lo = p - W + 1 > 0 ? p - W + 1 : 0;
        n_sink = ns < lo ? ns : lo;
        n = p < 0 ? 0 : n_sink + p - lo + 1;
    }
    __device__ int at(int i) const { return i < n_sink ? i : lo + i - n_sink; }
};

struct BwdArgs {
    Args f;
    const bf16 *o, *g;
    const float* lse;
    bf16 *dq, *dk, *dv;
};

template <int D>
__global__ void __launch_bounds__(128) sink_bwd_q_kernel(BwdArgs a) {
    __shared__ float sq[4][D], sg[4][D];
    const int wp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 4 + wp;
    const int h = static_cast<int>(w % a.f.H);
    const long long tok = w / a.f.H;
    if (tok >= (long long)a.f.B * a.f.L) return;
    const int b = static_cast<int>(tok / a.f.L), t = static_cast<int>(tok % a.f.L);
    const size_t orow = (tok * a.f.H + h) * D;
    float dl = 0.f;
    for (int c = lane; c < D; c += 32) {
        sq[wp][c] = __bfloat162float(a.f.q[tok * a.f.q_stride + h * D + c]);
        sg[wp][c] = __bfloat162float(a.g[orow + c]);
        dl += sg[wp][c] * __bfloat162float(a.o[orow + c]);
    }
    dl = warp_sum(dl);
    __syncwarp();
    const float lse = a.lse[tok * a.f.H + h];
    const Keys ks(t, a.f.W, a.f.ns);
    const int hk = h / (a.f.H / a.f.Hkv);
    float acc[D / 32] = {};
    for (int j0 = 0; j0 < ks.n; j0 += 32) {
        const int j = min(j0 + lane, ks.n - 1);
        const long long r = ((long long)b * a.f.L + ks.at(j)) * a.f.kv_stride + hk * D;
        const float p = __expf(dot<D>(sq[wp], a.f.k + r) * a.f.scale - lse);
        const float ds = p * (dot<D>(sg[wp], a.f.v + r) - dl) * a.f.scale;
        const int cnt = min(32, ks.n - j0);
        for (int u = 0; u < cnt; ++u) {
            const float du = __shfl_sync(~0u, ds, u);
            const long long ru = __shfl_sync(~0u, r, u);
            for (int c = 0; c < D / 32; ++c)
                acc[c] = fmaf(du, __bfloat162float(a.f.k[ru + c * 32 + lane]), acc[c]);
        }
    }
    for (int c = 0; c < D / 32; ++c) a.dq[orow + c * 32 + lane] = __float2bfloat16_rn(acc[c]);
}

template <int D>
__global__ void __launch_bounds__(128) sink_bwd_kv_kernel(BwdArgs a) {
    __shared__ float sk[4][D], sv[4][D];
    const int wp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 4 + wp;
    const int hk = static_cast<int>(w % a.f.Hkv);
    const long long tok = w / a.f.Hkv;
    if (tok >= (long long)a.f.B * a.f.L) return;
    const int b = static_cast<int>(tok / a.f.L), s = static_cast<int>(tok % a.f.L);
    const size_t r = tok * a.f.kv_stride + hk * D;
    for (int c = lane; c < D; c += 32) {
        sk[wp][c] = __bfloat162float(a.f.k[r + c]);
        sv[wp][c] = __bfloat162float(a.f.v[r + c]);
    }
    __syncwarp();
    const int last = s < a.f.ns ? a.f.L - 1 : min(a.f.L - 1, s + a.f.W - 1);
    const int G = a.f.H / a.f.Hkv;
    float ak[D / 32] = {}, av[D / 32] = {};
    for (int h = hk * G; h < hk * G + G; ++h)
        for (int t0 = s; t0 <= last; t0 += 32) {
            const int t = min(t0 + lane, last);
            const size_t tt = (size_t)b * a.f.L + t;
            const size_t qr = tt * a.f.q_stride + h * D, gr = (tt * a.f.H + h) * D;
            const float p = __expf(dot<D>(sk[wp], a.f.q + qr) * a.f.scale - a.lse[tt * a.f.H + h]);
            float dl = 0.f;
            for (int c = 0; c < D; ++c) dl += __bfloat162float(a.g[gr + c]) * __bfloat162float(a.o[gr + c]);
            const float ds = p * (dot<D>(sv[wp], a.g + gr) - dl) * a.f.scale;
            const int cnt = min(32, last - t0 + 1);
            for (int u = 0; u < cnt; ++u) {
                const float du = __shfl_sync(~0u, ds, u), pu = __shfl_sync(~0u, p, u);
                const size_t tu = (size_t)b * a.f.L + t0 + u;
                for (int c = 0; c < D / 32; ++c) {
                    ak[c] = fmaf(du, __bfloat162float(a.f.q[tu * a.f.q_stride + h * D + c * 32 + lane]), ak[c]);
                    av[c] = fmaf(pu, __bfloat162float(a.g[(tu * a.f.H + h) * D + c * 32 + lane]), av[c]);
                }
            }
        }
    const size_t orow = (tok * a.f.Hkv + hk) * D;
    for (int c = 0; c < D / 32; ++c) {
        a.dk[orow + c * 32 + lane] = __float2bfloat16_rn(ak[c]);
        a.dv[orow + c * 32 + lane] = __float2bfloat16_rn(av[c]);
    }
}

Args make_args(const SinkShape& s, const void* q, const void* k, const void* v, int* status) {
    Args a{};
    a.q = static_cast<const bf16*>(q);
    a.k = static_cast<const bf16*>(k);
    a.v = static_cast<const bf16*>(v);
    a.B = s.B; a.L = s.L; a.H = s.H; a.Hkv = s.Hkv; a.W = s.W; a.ns = s.ns;
    a.q_stride = s.q_stride; a.kv_stride = s.kv_stride;
    a.scale = s.scale;
    a.paged = s.paged;
    a.status = status;
    return a;
}

}  // namespace

size_t sink_bwd_workspace_bytes(const SinkShape&) { return 256; }

cudaError_t launch_sink_bwd(const SinkShape& s, const void* q, const void* k, const void* v,
                            const void* o, const float* lse, const void* dout, void* dq, void* dk,
                            void* dv, void*, int* status, cudaStream_t st, int* launches) {
    BwdArgs a{};
    a.f = make_args(s, q, k, v, status);
    a.o = static_cast<const bf16*>(o);
    a.g = static_cast<const bf16*>(dout);
    a.lse = lse;
    a.dq = static_cast<bf16*>(dq);
    a.dk = static_cast<bf16*>(dk);
    a.dv = static_cast<bf16*>(dv);
    const unsigned bq = (unsigned)(((long long)s.T * s.H + 3) / 4), bk = (unsigned)(((long long)s.T * s.Hkv + 3) / 4);
    GCA_LAUNCH("sink_bwd_q", st, (s.d == 64 ? sink_bwd_q_kernel<64><<<bq, 128, 0, st>>>(a)
                                            : sink_bwd_q_kernel<128><<<bq, 128, 0, st>>>(a)));
    GCA_LAUNCH("sink_bwd_kv", st, (s.d == 64 ? sink_bwd_kv_kernel<64><<<bk, 128, 0, st>>>(a)
                                             : sink_bwd_kv_kernel<128><<<bk, 128, 0, st>>>(a)));
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *launches += 2;
    return e;
}

}  // namespace gca
