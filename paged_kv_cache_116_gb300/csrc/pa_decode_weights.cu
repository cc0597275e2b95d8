// pa_decode_weights.cu -- the instances of the tensor-core decode that keep
// the scores and add up the attention weights (pa_decode_weights and its code
// cache form; kernels in pa_decode_tc.cuh).
//
// Bound: HBM, as the plain decode: per (token, KV head) the K and V rows and
// 8 bytes of weight (read and written), plus 8 bytes per query head for the
// scores' way out and back, which mostly stays in L2.
#include "pa_decode_tc.cuh"

namespace pa {
namespace {

template <typename T, int HD, int NT>
cudaError_t launch_scores(const AttnArgs& a, int32_t num_blocks, int grid, void* ws, std::string* err,
                          cudaStream_t st, const DecodeWeights& w) {
    if (!tma_block_size(a.block_size))
        return launch_typed<T, HD, NT, false, false, true, true>(a, num_blocks, grid, ws, err, st, &w);
    return launch_typed<T, HD, NT, false, false, false, true>(a, num_blocks, grid, ws, err, st, &w);
}

// f(kernel pointer, head_dim tag, code cache tag) for this problem's instance.
template <typename T, int NT, typename F>
auto with_instance(int head_dim, int block_size, bool kv_fp8, F f) {
    const bool gather = !tma_block_size(block_size);
    if (kv_fp8)
        return head_dim == 128 ? f(kernel_ptr<T, 128, NT, true, false, false, true>(), 128)
                               : f(kernel_ptr<T, 256, NT, true, false, false, true>(), 256);
    switch (head_dim) {
        case 64: return f(gather ? kernel_ptr<T, 64, NT, false, false, true, true>()
                                 : kernel_ptr<T, 64, NT, false, false, false, true>(), 64);
        case 128: return f(gather ? kernel_ptr<T, 128, NT, false, false, true, true>()
                                  : kernel_ptr<T, 128, NT, false, false, false, true>(), 128);
        default: return f(gather ? kernel_ptr<T, 256, NT, false, false, true, true>()
                                 : kernel_ptr<T, 256, NT, false, false, false, true>(), 256);
    }
}

template <typename T, int NT>
cudaError_t launch_nt(const AttnArgs& a, int32_t num_blocks, int grid, void* ws, std::string* err, cudaStream_t st,
                      const DecodeWeights& w) {
    if (a.kv_fp8)
        return a.head_dim == 128
                   ? launch_typed<T, 128, NT, true, false, false, true>(a, num_blocks, grid, ws, err, st, &w)
                   : launch_typed<T, 256, NT, true, false, false, true>(a, num_blocks, grid, ws, err, st, &w);
    switch (a.head_dim) {
        case 64: return launch_scores<T, 64, NT>(a, num_blocks, grid, ws, err, st, w);
        case 128: return launch_scores<T, 128, NT>(a, num_blocks, grid, ws, err, st, w);
        default: return launch_scores<T, 256, NT>(a, num_blocks, grid, ws, err, st, w);
    }
}

template <typename T, int NT>
int grid_nt(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t max_context,
            int64_t ctas_override, bool kv_fp8) {
    return with_instance<T, NT>(head_dim, block_size, kv_fp8, [&](const void* fn, int hd) {
        if (kv_fp8)
            return hd == 128 ? grid_for<128, true>(fn, num_seqs, num_kv_heads, max_context, ctas_override)
                             : grid_for<256, true>(fn, num_seqs, num_kv_heads, max_context, ctas_override);
        return hd == 64    ? grid_for<64, false>(fn, num_seqs, num_kv_heads, max_context, ctas_override)
               : hd == 128 ? grid_for<128, false>(fn, num_seqs, num_kv_heads, max_context, ctas_override)
                           : grid_for<256, false>(fn, num_seqs, num_kv_heads, max_context, ctas_override);
    });
}

}  // namespace

int decode_weights_grid(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                        int32_t max_context, int dtype, int32_t group, int64_t ctas_override, bool kv_fp8) {
    const int s = std::min(num_seqs, kDecodeMaxSeqsPerLaunch);
    if (dtype == 1)
        return group > 8 ? grid_nt<__nv_bfloat16, 2>(s, num_kv_heads, head_dim, block_size, max_context, ctas_override, kv_fp8)
                         : grid_nt<__nv_bfloat16, 1>(s, num_kv_heads, head_dim, block_size, max_context, ctas_override, kv_fp8);
    return group > 8 ? grid_nt<__half, 2>(s, num_kv_heads, head_dim, block_size, max_context, ctas_override, kv_fp8)
                     : grid_nt<__half, 1>(s, num_kv_heads, head_dim, block_size, max_context, ctas_override, kv_fp8);
}

size_t decode_weights_scores(int32_t num_heads, int32_t max_context) {
    return (size_t)num_heads * (((size_t)max_context + BS - 1) / BS * BS) * sizeof(float);
}

cudaError_t launch_decode_weights(const AttnArgs& a, int32_t num_blocks, int grid_ctas, void* workspace,
                                  const DecodeWeights& w, std::string* err, cudaStream_t stream) {
    if (a.num_seqs == 0) return cudaSuccess;
    const bool two = a.num_heads / a.num_kv_heads > 8;
    if (a.dtype == 1)
        return two ? launch_nt<__nv_bfloat16, 2>(a, num_blocks, grid_ctas, workspace, err, stream, w)
                   : launch_nt<__nv_bfloat16, 1>(a, num_blocks, grid_ctas, workspace, err, stream, w);
    return two ? launch_nt<__half, 2>(a, num_blocks, grid_ctas, workspace, err, stream, w)
               : launch_nt<__half, 1>(a, num_blocks, grid_ctas, workspace, err, stream, w);
}

uint32_t decode_weights_status(bool clear) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_decode_status, sizeof(v));
    if (clear) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_decode_status, &z, sizeof(z));
    }
    return v;
}

}  // namespace pa
