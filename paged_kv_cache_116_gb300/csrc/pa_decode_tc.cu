// pa_decode_tc.cu -- the plain instances of the tensor-core decode
// (pa_decode_tc.cuh).
#include "pa_decode_tc.cuh"

namespace pa {
namespace {

template <typename T>
cudaError_t launch_dtype(const AttnArgs& a, int32_t num_blocks, int grid, void* ws, std::string* err,
                         cudaStream_t st) {
    const int G = a.num_heads / a.num_kv_heads;
    const bool two = G > 8;
    if (a.kv_fp8) {
        if (a.head_dim == 128)
            return two ? launch_typed<T, 128, 2, true>(a, num_blocks, grid, ws, err, st)
                       : a.pair_steps ? launch_typed<T, 128, 1, true, true>(a, num_blocks, grid, ws, err, st)
                                      : launch_typed<T, 128, 1, true>(a, num_blocks, grid, ws, err, st);
        return two ? launch_typed<T, 256, 2, true>(a, num_blocks, grid, ws, err, st)
                   : launch_typed<T, 256, 1, true>(a, num_blocks, grid, ws, err, st);
    }
    if (!tma_block_size(a.block_size)) {
        switch (a.head_dim) {
            case 64: return two ? launch_typed<T, 64, 2, false, false, true>(a, num_blocks, grid, ws, err, st)
                                : launch_typed<T, 64, 1, false, false, true>(a, num_blocks, grid, ws, err, st);
            case 128: return two ? launch_typed<T, 128, 2, false, false, true>(a, num_blocks, grid, ws, err, st)
                                 : launch_typed<T, 128, 1, false, false, true>(a, num_blocks, grid, ws, err, st);
            default: return two ? launch_typed<T, 256, 2, false, false, true>(a, num_blocks, grid, ws, err, st)
                                : launch_typed<T, 256, 1, false, false, true>(a, num_blocks, grid, ws, err, st);
        }
    }
    switch (a.head_dim) {
        case 64: return two ? launch_typed<T, 64, 2, false>(a, num_blocks, grid, ws, err, st)
                            : launch_typed<T, 64, 1, false>(a, num_blocks, grid, ws, err, st);
        case 128: return two ? launch_typed<T, 128, 2, false>(a, num_blocks, grid, ws, err, st)
                             : launch_typed<T, 128, 1, false>(a, num_blocks, grid, ws, err, st);
        default: return two ? launch_typed<T, 256, 2, false>(a, num_blocks, grid, ws, err, st)
                            : launch_typed<T, 256, 1, false>(a, num_blocks, grid, ws, err, st);
    }
}

}  // namespace

bool decode_tc_supported(int dtype, int head_dim, int block_size, int group, bool kv_fp8) {
    const bool hd_ok = kv_fp8 ? (head_dim == 128 || head_dim == 256)
                              : (head_dim == 64 || head_dim == 128 || head_dim == 256);
    // 16-bit caches of any block size (boxes or a row gather); code caches by boxes only
    const bool bs_ok = kv_fp8 ? tma_block_size(block_size) : block_size >= 1;
    return (dtype == 1 || dtype == 2) && hd_ok && bs_ok && group >= 1 && group <= 16;
}

int decode_tc_grid(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                   int32_t max_context, int dtype, int32_t group, int64_t ctas_override, bool kv_fp8) {
    const int s = num_seqs < kDecodeMaxSeqsPerLaunch ? num_seqs : kDecodeMaxSeqsPerLaunch;
    const bool two = group > 8;
    const bool bf = dtype == 1;
    if (!kv_fp8 && !tma_block_size(block_size)) {  // the row-gather instances
#define PA_GFN(HD)                                                                                           \
    (bf ? (two ? kernel_ptr<__nv_bfloat16, HD, 2, false, false, true>()                                      \
               : kernel_ptr<__nv_bfloat16, HD, 1, false, false, true>())                                     \
        : (two ? kernel_ptr<__half, HD, 2, false, false, true>() : kernel_ptr<__half, HD, 1, false, false, true>()))
        switch (head_dim) {
            case 64: return grid_for<64, false>(PA_GFN(64), s, num_kv_heads, max_context, ctas_override);
            case 128: return grid_for<128, false>(PA_GFN(128), s, num_kv_heads, max_context, ctas_override);
            default: return grid_for<256, false>(PA_GFN(256), s, num_kv_heads, max_context, ctas_override);
        }
#undef PA_GFN
    }
#define PA_KFN(HD, F8)                                                                                      \
    (bf ? (two ? kernel_ptr<__nv_bfloat16, HD, 2, F8>() : kernel_ptr<__nv_bfloat16, HD, 1, F8>())          \
        : (two ? kernel_ptr<__half, HD, 2, F8>() : kernel_ptr<__half, HD, 1, F8>()))
    if (kv_fp8) {
        if (head_dim == 128) return grid_for<128, true>(PA_KFN(128, true), s, num_kv_heads, max_context, ctas_override);
        return grid_for<256, true>(PA_KFN(256, true), s, num_kv_heads, max_context, ctas_override);
    }
    switch (head_dim) {
        case 64: return grid_for<64, false>(PA_KFN(64, false), s, num_kv_heads, max_context, ctas_override);
        case 128: return grid_for<128, false>(PA_KFN(128, false), s, num_kv_heads, max_context, ctas_override);
        default: return grid_for<256, false>(PA_KFN(256, false), s, num_kv_heads, max_context, ctas_override);
    }
#undef PA_KFN
}

int decode_tc_warps_per_cta(int32_t head_dim, bool kv_fp8) {
    if (kv_fp8) return head_dim == 256 ? Pipe<256, true>::NW : Pipe<128, true>::NW;
    return head_dim == 256 ? Pipe<256, false>::NW : (head_dim == 128 ? Pipe<128, false>::NW : Pipe<64, false>::NW);
}

size_t decode_tc_workspace(int32_t num_seqs, int32_t num_kv_heads, int32_t group, int32_t head_dim, int grid_ctas,
                           bool kv_fp8) {
    const int nw = decode_tc_warps_per_cta(head_dim, kv_fp8);
    return (size_t)grid_ctas * nw * 2 * group * (head_dim + 4) * sizeof(float);
}

cudaError_t launch_decode_tc(const AttnArgs& a, int32_t num_blocks, int grid_ctas, void* workspace,
                             std::string* err, cudaStream_t stream) {
    if (a.num_seqs == 0) return cudaSuccess;
    return a.dtype == 1 ? launch_dtype<__nv_bfloat16>(a, num_blocks, grid_ctas, workspace, err, stream)
                        : launch_dtype<__half>(a, num_blocks, grid_ctas, workspace, err, stream);
}

uint32_t decode_tc_status(bool clear) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_decode_status, sizeof(v));
    if (clear) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_decode_status, &z, sizeof(z));
    }
    return v;
}

}  // namespace pa
