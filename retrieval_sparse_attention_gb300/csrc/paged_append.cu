// paged_append.cu -- the write of new tokens' keys and values into the paged K/V
// cache of the window self-attention (gca_paged_append).
#include "attn_sink.cuh"
#include "kernels.h"

namespace gca {
namespace {

// One warp per row of the token tensors: the lanes look for the sequence that the row belongs
// to, 32 at a time, first where it is if all have equally many tokens, then from the first
// on (a token each of 2000 sequences: 3.6 us, without the guess 17.3); then they copy the row's 16-byte
// vectors, four of K and of V in flight each.  Bound by memory: reads and writes every new
// row once (four prompts of 16K, 8 heads of 128: 77 us, 6.8 TB/s; eight chunks of 0.9-2K, 12 heads
// of 64: 16 us with cold caches, 8.6 with warm ones).  A warp for each of the first max_q
// tokens of every sequence, without the search, took 20 us for the chunks; two or four rows a
// warp 10 and 12 instead of 8.6.
__global__ void __launch_bounds__(256)
paged_append_kernel(PagedArgs p, const uint4* k_new, const uint4* v_new, int src_vec, int row_vec,
                    uint4* k_cache, uint4* v_cache, int B, int* status) {
    const int lane = threadIdx.x & 31;
    const long long tid = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    // contradicting entries are reported whether a row belongs to them or not
    for (long long b = tid; b < B; b += (long long)gridDim.x * blockDim.x) paged_seq(p, (int)b, status);
    if (tid >> 5 >= p.T) return;
    const int row = (int)(tid >> 5);
    int seq = -1, pos = 0;
    const int guess = max(min(static_cast<int>(static_cast<long long>(row) * B / p.T) - 16, B - 32), 0);
    for (int k = -32; k < B && seq < 0; k += 32) {
        const int b0 = k < 0 ? guess : k;
        SeqInfo s{0, 0, 0};
        if (b0 + lane < B) s = paged_seq(p, b0 + lane, nullptr);
        const unsigned hit = __ballot_sync(0xffffffffu, row >= s.row0 && row < s.row0 + s.n);
        if (hit) {
            const int l = __ffs(hit) - 1;
            seq = b0 + l;
            pos = __shfl_sync(0xffffffffu, s.pos0 + row - s.row0, l);
        }
    }
    if (seq < 0 || pos < 0) return;
    const int pg = p.table[(size_t)seq * p.width + (pos >> p.page_log2)];
    if (pg < 0 || pg >= p.n_pages) {
        if (lane == 0) set_status(status, GCA_ERR_DEVICE_INDEX);
        return;
    }
    const size_t dst = (((size_t)pg << p.page_log2) + (pos & ((1 << p.page_log2) - 1))) * row_vec;
    const size_t src = (size_t)row * src_vec;
    for (int c0 = 0; c0 < row_vec; c0 += 128) {
        uint4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + 32 * i + lane;
            if (c < row_vec) {
                x[i] = k_new[src + c];
                y[i] = v_new[src + c];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = c0 + 32 * i + lane;
            if (c < row_vec) {
                k_cache[dst + c] = x[i];
                v_cache[dst + c] = y[i];
            }
        }
    }
}

}  // namespace

cudaError_t launch_paged_append(const SinkShape& s, const void* k_new, const void* v_new,
                                const int32_t* cu_q, const int32_t* kv_len, const int32_t* table,
                                void* k_cache, void* v_cache, int* status, cudaStream_t st,
                                int* launches) {
    PagedArgs p{cu_q, kv_len, table, s.T, s.max_q, __builtin_ctz(s.page), s.n_pages, s.width};
    const long long blocks = ((long long)s.T + 7) / 8;
    GCA_LAUNCH("paged_append", st,
               paged_append_kernel<<<(unsigned)blocks, 256, 0, st>>>(
                   p, static_cast<const uint4*>(k_new), static_cast<const uint4*>(v_new), s.kv_stride / 8,
                   s.Hkv * s.d / 8, static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache), s.B, status));
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) *launches += 1;
    return e;
}

}  // namespace gca
