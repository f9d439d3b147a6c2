// paged_append.cu -- the write of new tokens' keys and values into the paged K/V
// cache of the window self-attention (gca_paged_append).
#include "attn_sink.cuh"
#include "kernels.h"

namespace gca {
namespace {

// One warp per new token: 16-byte vectors of its K and V rows.
__global__ void __launch_bounds__(256)
paged_append_kernel(PagedArgs p, const uint4* k_new, const uint4* v_new, int src_vec, int row_vec,
                    uint4* k_cache, uint4* v_cache, int B, int* status) {
    const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * warps + (threadIdx.x >> 5);
    const int b = static_cast<int>(w / p.max_q), i = static_cast<int>(w % p.max_q);
    if (b >= B) return;
    const SeqInfo s = paged_seq(p, b, status);
    if (i >= s.n) return;
    const int pos = s.pos0 + i;
    if (pos < 0) return;
    const int pg = p.table[(size_t)b * p.width + (pos >> p.page_log2)];
    if (pg < 0 || pg >= p.n_pages) {
        if (lane == 0) set_status(status, GCA_ERR_DEVICE_INDEX);
        return;
    }
    const size_t dst = (((size_t)pg << p.page_log2) + (pos & ((1 << p.page_log2) - 1))) * row_vec;
    const size_t src = (size_t)(s.row0 + i) * src_vec;
    for (int c = lane; c < row_vec; c += 32) {
        k_cache[dst + c] = k_new[src + c];
        v_cache[dst + c] = v_new[src + c];
    }
}

}  // namespace

cudaError_t launch_paged_append(const SinkShape& s, const void* k_new, const void* v_new,
                                const int32_t* cu_q, const int32_t* kv_len, const int32_t* table,
                                void* k_cache, void* v_cache, int* status, cudaStream_t st,
                                int* launches) {
    PagedArgs p{cu_q, kv_len, table, s.T, s.max_q, __builtin_ctz(s.page), s.n_pages, s.width};
    const long long warps = (long long)s.B * s.max_q;
    const long long blocks = (warps + 7) / 8;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    GCA_LAUNCH("paged_append", st,
               paged_append_kernel<<<(unsigned)blocks, 256, 0, st>>>(
                   p, static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), s.kv_stride / 8,
                   s.Hkv * s.d / 8, static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), s.B, status));
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *launches += 1;
    return e;
}

}  // namespace gca
