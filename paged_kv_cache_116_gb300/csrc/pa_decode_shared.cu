// pa_decode_shared.cu -- decode of sequences that share leading blocks: the
// prefixes once for all members (pa_prefix_umma.cu), the rest of each context
// by the tensor-core decode (pa_decode_tc.cuh, an instance that keeps its
// states), and the kernel that joins both.
//
// The softmax over a context is the join of its parts' (m, l, o): with
// M = max m_i, out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i, in a fixed
// order (the prefix's pieces, then the rest's), all in fp32.
//
// Bound: the bytes of the prefixes, once a group, and of the rest of each
// context; 64 requests of 20-1,500 tokens behind 8,192 shared ones read 233 MB
// instead of 2,336 (67 us instead of 228).  The decode runs first and the
// prefixes start as it leaves each SM: both need most of an SM's shared memory.
#include "pa_decode_tc.cuh"
#include "pa_shared.cuh"

namespace pa {
namespace {

// Per sequence: the length of the rest of its context and the blocks of it (the
// table row from the shared blocks on).  A CTA per sequence.
__global__ void __launch_bounds__(128) shared_plan_kernel(const SharedGroups g, const int32_t* context_lens,
                                                          const int32_t* block_tables, int max_blocks,
                                                          int32_t* rest_lens, int32_t* rest_tables, int rest_blocks,
                                                          int32_t* group_of) {
    pdl_wait_primary();
    pdl_launch_dependents();
    const int s = blockIdx.x, L = max(context_lens[s], 0);
    // the last group that starts at or before s
    int lo = -1, hi = g.groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (g.starts[mid] <= s) lo = mid;
        else hi = mid - 1;
    }
    int skip = lo >= 0 && s < g.starts[lo + 1] ? shared_tokens(g, lo) : 0;
    if (skip > L) skip = 0;  // (a context shorter than its prefix is the caller's mistake)
    const int rest = L - skip, first = skip / g.block_size;
    const int n = min((rest + g.block_size - 1) / g.block_size, rest_blocks);
    for (int i = threadIdx.x; i < n; i += blockDim.x)
        rest_tables[(int64_t)s * rest_blocks + i] = block_tables[(int64_t)s * max_blocks + first + i];
    if (threadIdx.x == 0) {
        rest_lens[s] = rest;
        group_of[s] = skip ? lo : -1;
    }
}

// Half a warp per (sequence, query head): its records in order, B at a time.
template <typename T, int HD, int B = HD <= 128 ? 8 : 4>
__global__ void __launch_bounds__(256) shared_merge_kernel(const TcParams p, const int64_t TW, const SharedGroups g,
                                                           const int32_t* group_of, const int ctas) {
    extern __shared__ int32_t sm[];
    int32_t* rest = sm;                        // [num_seqs + 1] 16-token tiles of the rests
    int32_t* gcost = sm + p.num_seqs + 1;      // [groups + 1]
    constexpr int E = HD / 16, REC = HD + 4;
    const int S = p.num_seqs, Hkv = p.num_kv_heads, G = p.group;
    // (the plan is older than the two grids before this one)
    tile_prefix(p.context_lens, S, rest, nullptr);
    shared_prefix(g, gcost);
    const int row = blockIdx.x * 16 + (threadIdx.x >> 4), hl = threadIdx.x & 15;
    const bool mine = row < S * p.num_heads;
    const int s = mine ? row / p.num_heads : 0, hq = mine ? row - s * p.num_heads : 0;
    const int kv = hq / G, j = hq - kv * G;
    // the prefix's pieces: the row's own record, then those of the CTAs behind
    int np = 0, c0 = 0, tile_row = 0;
    const int grp = group_of[s];
    if (grp >= 0) {
        const int64_t WP = gcost[g.groups], C = shared_ctas(WP, ctas);
        const int nk = (shared_tokens(g, grp) + kPrefixKeys - 1) / kPrefixKeys, at = s - g.starts[grp];
        const int t = at / g.tokens, unit = kv * shared_row_tiles(g, grp) + t;
        const int64_t u0 = gcost[grp] + (int64_t)unit * (nk + kPrefixUnit) + kPrefixUnit;  // its first key tile
        c0 = (int)(((u0 + 1) * C + WP - 1) / WP) - 1;
        np = (int)(((u0 + nk) * C + WP - 1) / WP) - c0;
        tile_row = (at - t * g.tokens) * G + j;
    }
    // the rest's pieces: warps wf .. of the decode, or (fewer tiles than warps:
    // a warp has one or none) the owners of its tiles one by one
    const int nb = rest[s + 1] - rest[s];
    const int64_t W = (int64_t)rest[S] * Hkv, u0 = (int64_t)rest[s] * Hkv + (int64_t)kv * nb;
    const bool sparse = W < TW;
    auto owner = [&](int64_t f) -> int {
        const int64_t x = (f + 1) * TW + W - 1;
        return (x >> 32 ? (int)(x / W) : (int)((uint32_t)x / (uint32_t)W)) - 1;
    };
    int wf = 0, nw = 0, slot0 = 0;
    if (nb > 0) {
        wf = owner(u0);
        nw = sparse ? nb : owner(u0 + nb - 1) - wf + 1;
        slot0 = u0 == wf * W / TW ? 0 : 1;
    }
    auto record = [&](int i) -> const float* {
        if (i < np) return i == 0 ? g.rows + (int64_t)row * REC : g.cont + ((int64_t)(c0 + i) * 128 + tile_row) * REC;
        i -= np;
        if (nw == 1) return p.rows + (int64_t)row * REC;
        const int w = sparse ? owner(u0 + i) : wf + i;
        return p.ws_part + (((int64_t)w * 2 + (i == 0 ? slot0 : 0)) * G + j) * REC;
    };
    pdl_wait_primary();
    if (!mine) return;
    const int n = np + nw;
    float M = -INFINITY, L = 0.f, o[E];
#pragma unroll
    for (int t = 0; t < E; ++t) o[t] = 0.f;
    for (int i0 = 0; i0 < n; i0 += B) {
        float m[B], l[B];
        float4 a[B][E / 4];
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const float* r = i0 + b < n ? record(i0 + b) : nullptr;
            m[b] = r ? __ldcg(r + HD) : -INFINITY;
            l[b] = r ? __ldcg(r + HD + 1) : 0.f;
#pragma unroll
            for (int t = 0; t < E / 4; ++t)
                a[b][t] = r ? __ldcg(reinterpret_cast<const float4*>(r + hl * E) + t) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        float mn = M;
#pragma unroll
        for (int b = 0; b < B; ++b) mn = fmaxf(mn, m[b]);
        const float ms = mn == -INFINITY ? 0.f : mn, c = exp2f(M - ms);
        L *= c;
#pragma unroll
        for (int t = 0; t < E; ++t) o[t] *= c;
#pragma unroll
        for (int b = 0; b < B; ++b) {
            const float e = exp2f(m[b] - ms);
            L = fmaf(e, l[b], L);
#pragma unroll
            for (int t = 0; t < E / 4; ++t) {
                o[4 * t + 0] = fmaf(e, a[b][t].x, o[4 * t + 0]);
                o[4 * t + 1] = fmaf(e, a[b][t].y, o[4 * t + 1]);
                o[4 * t + 2] = fmaf(e, a[b][t].z, o[4 * t + 2]);
                o[4 * t + 3] = fmaf(e, a[b][t].w, o[4 * t + 3]);
            }
        }
        M = mn;
    }
    const float inv = n > 0 ? 1.f / L : 0.f;  // (no context: a zero row)
    T* out = static_cast<T*>(p.out) + (int64_t)row * HD + hl * E;
#pragma unroll
    for (int t = 0; t < E; t += 4)
        *reinterpret_cast<uint2*>(out + t) =
            make_uint2(pack2<T>(o[t] * inv, o[t + 1] * inv), pack2<T>(o[t + 2] * inv, o[t + 3] * inv));
}

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

// The parts of the workspace behind the decode's records.
struct Space {
    size_t rows, prefix_rows, cont, lens, groups, tables, total;
    int rest_blocks;
};
Space space(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
            int32_t max_context, int grid_ctas) {
    const int G = num_heads / num_kv_heads;
    Space s;
    s.rest_blocks = (int)(((int64_t)max_context + block_size - 1) / block_size);
    size_t at = round256(decode_tc_workspace(num_seqs, num_kv_heads, G, head_dim, grid_ctas));
    auto take = [&](size_t b) {
        const size_t o = at;
        at += round256(b);
        return o;
    };
    const size_t rec = (size_t)(head_dim + 4) * sizeof(float);
    s.rows = take((size_t)num_seqs * num_heads * rec);
    s.prefix_rows = take((size_t)num_seqs * num_heads * rec);
    s.cont = take((size_t)kSms * 128 * rec);
    s.lens = take((size_t)num_seqs * 4);
    s.groups = take((size_t)num_seqs * 4);
    s.tables = take((size_t)num_seqs * s.rest_blocks * 4);
    s.total = at;
    return s;
}

template <typename T, int HD, int NT>
cudaError_t launch_part(const AttnArgs& a, const SharedGroups& g, int32_t num_blocks, int grid, uint8_t* ws,
                        const Space& sp, std::string* err, cudaStream_t stream) {
    CUtensorMap tmK, tmV;
    if (!make_kv_map(&tmK, a.k_cache, a.dtype, false, num_blocks, a.block_size, a.num_kv_heads, HD, err) ||
        !make_kv_map(&tmV, a.v_cache, a.dtype, false, num_blocks, a.block_size, a.num_kv_heads, HD, err))
        return cudaErrorInvalidValue;
    int32_t* lens = reinterpret_cast<int32_t*>(ws + sp.lens);
    int32_t* group_of = reinterpret_cast<int32_t*>(ws + sp.groups);
    int32_t* tables = reinterpret_cast<int32_t*>(ws + sp.tables);
    cudaError_t e = launch_pdl(shared_plan_kernel, dim3((unsigned)a.num_seqs), dim3(128), stream, g, a.seq_lens,
                               a.block_tables, a.max_blocks, lens, tables, sp.rest_blocks, group_of);
    if (e != cudaSuccess) return e;
    TcParams p{};
    p.out = a.out;
    p.q = a.q;
    p.block_tables = tables;
    p.max_blocks = sp.rest_blocks;
    p.context_lens = lens;
    p.num_seqs = a.num_seqs;
    p.num_heads = a.num_heads;
    p.num_kv_heads = a.num_kv_heads;
    p.group = a.num_heads / a.num_kv_heads;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.ws_part = reinterpret_cast<float*>(ws);
    p.k_pool = const_cast<void*>(a.k_cache);
    p.v_pool = const_cast<void*>(a.v_cache);
    p.block_size = a.block_size;
    p.rows = reinterpret_cast<float*>(ws + sp.rows);
    const auto kernel = decode_tc_kernel<T, HD, NT, false, false, false, false, true>;
    e = allow_smem(reinterpret_cast<const void*>(kernel), smem_bytes<HD, false>(kDecodeMaxSeqsPerLaunch));
    if (e != cudaSuccess) return e;
    using Pp = Pipe<HD, false>;
    e = launch_pdl_smem(kernel, dim3((unsigned)grid), dim3(Pp::NW * 32), smem_bytes<HD, false>(a.num_seqs), stream,
                        tmK, tmV, p);
    if (e != cudaSuccess) return e;
    const int ctas = std::min(kSms, sm_count());
    e = launch_prefix_umma(a, g, num_blocks, ctas, err, stream);
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)a.num_seqs * a.num_heads;
    return launch_pdl_smem(shared_merge_kernel<T, HD>, dim3((unsigned)((rows + 15) / 16)), dim3(256),
                           (size_t)(a.num_seqs + g.groups + 2) * sizeof(int32_t), stream, p,
                           (int64_t)grid * Pp::NW, g, (const int32_t*)group_of, ctas);
}

template <typename T, int HD>
cudaError_t launch_hd(const AttnArgs& a, const SharedGroups& g, int32_t num_blocks, int grid, uint8_t* ws,
                      const Space& sp, std::string* err, cudaStream_t stream) {
    return a.num_heads / a.num_kv_heads > 8 ? launch_part<T, HD, 2>(a, g, num_blocks, grid, ws, sp, err, stream)
                                            : launch_part<T, HD, 1>(a, g, num_blocks, grid, ws, sp, err, stream);
}

template <typename T, int HD>
int grid_hd(int32_t num_seqs, int32_t num_kv_heads, int32_t max_context, int32_t group, int64_t override_ctas) {
    const void* fn = group > 8 ? reinterpret_cast<const void*>(&decode_tc_kernel<T, HD, 2, false, false, false, false, true>)
                               : reinterpret_cast<const void*>(&decode_tc_kernel<T, HD, 1, false, false, false, false, true>);
    return grid_for<HD, false>(fn, num_seqs, num_kv_heads, max_context, override_ctas);
}

}  // namespace

bool decode_shared_supported(int dtype, int head_dim, int block_size, int group, int32_t num_seqs, int32_t num_groups,
                             int32_t max_context) {
    return num_groups > 0 && num_groups <= kDecodeMaxSeqsPerLaunch && num_seqs <= kDecodeMaxSeqsPerLaunch &&
           tma_block_size(block_size) && decode_tc_supported(dtype, head_dim, block_size, group) && max_context >= 16;
}

int decode_shared_grid(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t max_context, int dtype,
                       int32_t group, int64_t ctas_override) {
    if (dtype == 1)
        return head_dim == 64    ? grid_hd<__nv_bfloat16, 64>(num_seqs, num_kv_heads, max_context, group, ctas_override)
               : head_dim == 128 ? grid_hd<__nv_bfloat16, 128>(num_seqs, num_kv_heads, max_context, group, ctas_override)
                                 : grid_hd<__nv_bfloat16, 256>(num_seqs, num_kv_heads, max_context, group, ctas_override);
    return head_dim == 64    ? grid_hd<__half, 64>(num_seqs, num_kv_heads, max_context, group, ctas_override)
           : head_dim == 128 ? grid_hd<__half, 128>(num_seqs, num_kv_heads, max_context, group, ctas_override)
                             : grid_hd<__half, 256>(num_seqs, num_kv_heads, max_context, group, ctas_override);
}

size_t decode_shared_workspace(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                               int32_t block_size, int32_t max_context, int grid_ctas) {
    return space(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, grid_ctas).total;
}

cudaError_t launch_decode_shared(const AttnArgs& a, const int32_t* group_starts, const int32_t* prefix_lens,
                                 int32_t num_groups, int32_t num_blocks, int grid_ctas, void* workspace,
                                 std::string* err, cudaStream_t stream) {
    const Space sp = space(a.num_seqs, a.num_heads, a.num_kv_heads, a.head_dim, a.block_size, a.max_context, grid_ctas);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    SharedGroups g;
    g.starts = group_starts;
    g.prefix_lens = prefix_lens;
    g.groups = num_groups;
    g.num_kv_heads = a.num_kv_heads;
    g.tokens = 128 / (a.num_heads / a.num_kv_heads);
    g.block_size = a.block_size;
    g.rows = reinterpret_cast<float*>(ws + sp.prefix_rows);
    g.cont = reinterpret_cast<float*>(ws + sp.cont);
    if (a.dtype == 1)
        return a.head_dim == 64    ? launch_hd<__nv_bfloat16, 64>(a, g, num_blocks, grid_ctas, ws, sp, err, stream)
               : a.head_dim == 128 ? launch_hd<__nv_bfloat16, 128>(a, g, num_blocks, grid_ctas, ws, sp, err, stream)
                                   : launch_hd<__nv_bfloat16, 256>(a, g, num_blocks, grid_ctas, ws, sp, err, stream);
    return a.head_dim == 64    ? launch_hd<__half, 64>(a, g, num_blocks, grid_ctas, ws, sp, err, stream)
           : a.head_dim == 128 ? launch_hd<__half, 128>(a, g, num_blocks, grid_ctas, ws, sp, err, stream)
                               : launch_hd<__half, 256>(a, g, num_blocks, grid_ctas, ws, sp, err, stream);
}

uint32_t decode_shared_status(bool clear) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_decode_status, sizeof(v));
    if (clear) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_decode_status, &z, sizeof(z));
    }
    return v;
}

}  // namespace pa
