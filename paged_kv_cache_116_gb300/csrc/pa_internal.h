// pa_internal.h -- host-side declarations shared by the library's translation
// units (launchers called by the C ABI in pa_api.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <string>

namespace pa {

// Element size of a pa_dtype (PA_F32 = 0, PA_BF16 = 1, PA_F16 = 2, PA_FP8_E4M3 = 3).
inline int elt_size(int dtype) { return dtype == 0 ? 4 : (dtype == 3 ? 1 : 2); }

// Upper limit of sequences one tensor-core decode launch handles (its
// per-sequence block-count prefix lives in shared memory); the C ABI splits
// larger batches into launches of at most this many sequences.
constexpr int kDecodeMaxSeqsPerLaunch = 4096;

// What a launch of the weight operators may keep per token of max_context in
// the workspace (the scores of a decode, a dense copy of the keys of a
// prompt): these grow with sequences times max_context whatever the lengths
// are, so batches beyond it are worked in several launches, of one sequence at
// least.  1.5 % of the GPU's memory; 32 heads' scores over 131,072 tokens are
// 17 MB a sequence, the keys of 8 heads of 128 are 268 MB.
constexpr int64_t kScratchBytes = (int64_t)4 << 30;
inline int32_t seqs_per_launch(int32_t num_seqs, double bytes_per_seq, int32_t most) {
    const int32_t n = num_seqs < most ? num_seqs : most;
    if (n * bytes_per_seq <= kScratchBytes) return n;
    const double fit = kScratchBytes / bytes_per_seq;  // (below n)
    if (fit < 2) return 1;
    // parts of one size: the last is not a single long sequence
    const int64_t parts = ((int64_t)num_seqs + (int64_t)fit - 1) / (int64_t)fit;
    return (int32_t)((num_seqs + parts - 1) / parts);
}

// Most layers one pa_copy_blocks call takes (their pointers travel in the
// kernel's parameter block).  Equal to PA_MAX_LAYERS of pa.h.
#define PA_MAX_LAYERS_INTERNAL 128

// SMs of a GB300: what the rules that cut work into CTAs count on.  Not asked of
// the device, since some of them size workspaces and those answers are also
// given where there is none (sm_count() bounds the grids of persistent kernels).
constexpr int kSms = 152;

// Number of polls a bounded mbarrier wait makes before giving up.
constexpr uint32_t kMaxPolls = 1u << 24;

// Reason reported by pa_last_error() for the calling thread (pa_api.cu).
void record_error(const std::string& msg);

// Check mode (PA_OPT_CHECK_MODE) for entry points outside pa_api.cu: whether
// it is on, and the decode's index validation (lengths in [0, max_context],
// tables long enough, block ids in [0, num_blocks)) on host copies of the
// index arrays.  Returns a pa_status value (PA_OK, PA_ERR_INDEX or
// PA_ERR_CUDA) and records the reason for pa_last_error().
bool check_mode_on();
int check_decode_indices(const int32_t* block_tables, int32_t max_blocks, const int32_t* context_lens,
                         int32_t num_seqs, int32_t num_blocks, int32_t block_size, int32_t max_context,
                         cudaStream_t stream);

// ---- copy kernels (pa_copy.cu)
cudaError_t launch_slot_mapping(const int32_t* block_tables, int32_t max_blocks, const int32_t* seq_idx,
                                const int64_t* positions, int64_t n, int32_t block_size, int64_t* slot_out,
                                cudaStream_t stream);
cudaError_t launch_write_kv(const void* k, const void* v, const int64_t* slot_mapping, int64_t n, void* k_cache,
                            void* v_cache, int64_t row_bytes, cudaStream_t stream);
// Writes k_new[s] / v_new[s] ([S, Hkv, hd]) to each sequence's slot of
// position context_lens[s] - 1 (sequences with length 0 are skipped).
cudaError_t launch_append_kv(const void* k_new, const void* v_new, const int32_t* block_tables, int32_t max_blocks,
                             const int32_t* context_lens, int32_t num_seqs, int32_t block_size, void* k_cache,
                             void* v_cache, int64_t row_bytes, cudaStream_t stream);
cudaError_t launch_swap_blocks(void* const* src_k, void* const* src_v, void* const* dst_k, void* const* dst_v,
                               int32_t num_layers, const int64_t* block_pairs, int32_t num_pairs, int64_t block_bytes,
                               cudaStream_t stream);
// Quantizing write: each (token, KV head) row of k / v ([n, Hkv, hd] of
// dtype) becomes E4M3 codes at its slot of k_codes / v_codes and one fp32
// scale in k_scales / v_scales [num_blocks, Hkv, block_size].
cudaError_t launch_write_kv_fp8(const void* k, const void* v, int dtype, const int64_t* slot_mapping, int64_t n,
                                int32_t num_kv_heads, int32_t head_dim, int32_t block_size, uint8_t* k_codes,
                                uint8_t* v_codes, float* k_scales, float* v_scales, cudaStream_t stream);
// The same for the generation step: sequence s's new rows go to the slot of
// position context_lens[s] - 1.
cudaError_t launch_append_kv_fp8(const void* k_new, const void* v_new, int dtype, const int32_t* block_tables,
                                 int32_t max_blocks, const int32_t* context_lens, int32_t num_seqs,
                                 int32_t num_kv_heads, int32_t head_dim, int32_t block_size, uint8_t* k_codes,
                                 uint8_t* v_codes, float* k_scales, float* v_scales, cudaStream_t stream);
cudaError_t launch_copy_blocks(void* const* k_caches, void* const* v_caches, int32_t num_layers,
                               const int64_t* block_pairs, int32_t num_pairs, int64_t block_bytes,
                               cudaStream_t stream);

// ---- CUDA-core attention (pa_attn_simt.cu): any dtype, head_dim <= 256.
// cu_seqlens_q == nullptr means one query per sequence (row i = sequence i).
struct AttnArgs {
    void* out;
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* block_tables;
    int32_t max_blocks;
    const int32_t* seq_lens;
    const int32_t* cu_seqlens_q;
    int32_t num_seqs;
    int32_t total_q;
    int32_t num_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t block_size;
    float scale;
    int causal;
    int dtype;
    // upper bound of seq_lens (varlen: sizes the work plan's buckets)
    int32_t max_context = 0;
    // decode only: the new token of each sequence (position L-1), written to
    // the pool and attended from these rows (nullptr: plain decode)
    const void* k_new = nullptr;
    const void* v_new = nullptr;
    // quantized cache: k_cache / v_cache hold E4M3 codes and these fp32
    // scales [num_blocks, num_kv_heads, block_size]; dtype is then the type
    // of q and out only
    int kv_fp8 = 0;
    const float* k_scales = nullptr;
    const float* v_scales = nullptr;
    // code cache, head_dim 128: the two tiles of a stage that belong to one
    // unit worked as one 32-token step
    int pair_steps = 0;
};
bool attn_simt_supported(int dtype, int head_dim);  // either cache kind
cudaError_t launch_attn_simt(const AttnArgs& a, cudaStream_t stream);

// ---- tensor-core decode (pa_decode_tc.cu)
// kv_fp8: the cache holds E4M3 codes with scales (AttnArgs::kv_fp8).
bool decode_tc_supported(int dtype, int head_dim, int block_size, int group, bool kv_fp8 = false);
// Grid size (CTAs) the launch will use for this problem on the current device.
int decode_tc_grid(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                   int32_t max_context, int dtype, int32_t group, int64_t ctas_override, bool kv_fp8 = false);
int decode_tc_warps_per_cta(int32_t head_dim, bool kv_fp8 = false);
size_t decode_tc_workspace(int32_t num_seqs, int32_t num_kv_heads, int32_t group, int32_t head_dim, int grid_ctas,
                           bool kv_fp8 = false);
cudaError_t launch_decode_tc(const AttnArgs& a, int32_t num_blocks, int grid_ctas, void* workspace,
                             std::string* err, cudaStream_t stream);
uint32_t decode_tc_status(bool clear);

// ---- the same with the attention weights (pa_decode_weights.cu)
struct DecodeWeights {
    float* weights;  // [num_seqs, num_kv_heads, stride]
    int64_t stride;
    float* scores;      // decode_weights_scores(...) bytes per sequence of the launch
    float2* row_stats;  // [num_seqs, num_heads]
};
int decode_weights_grid(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                        int32_t max_context, int dtype, int32_t group, int64_t ctas_override, bool kv_fp8);
// Bytes of one sequence's scores.
size_t decode_weights_scores(int32_t num_heads, int32_t max_context);
cudaError_t launch_decode_weights(const AttnArgs& a, int32_t num_blocks, int grid_ctas, void* workspace,
                                  const DecodeWeights& w, std::string* err, cudaStream_t stream);
uint32_t decode_weights_status(bool clear);
// ---- self-test of the failure path (pa_selftest.cu): one CTA waits on a
// barrier nothing completes for `polls` polls and sets its status word's
// timeout bit (pa_selftest_wait_timeout).
cudaError_t launch_selftest_wait(uint32_t polls, cudaStream_t stream);
uint32_t selftest_status(bool clear);

// ---- tcgen05 varlen (pa_varlen_umma.cu)
bool varlen_umma_supported(int dtype, int head_dim, int block_size, int group, bool kv_fp8 = false);
// Bytes of the optional workspace that lets the kernel run its work longest first.
size_t varlen_umma_workspace(int32_t num_seqs, int64_t total_q, int32_t group);
// workspace: nullptr (request order), or varlen_umma_workspace(...) bytes.
cudaError_t launch_varlen_umma(const AttnArgs& a, int32_t num_blocks, void* workspace, std::string* err,
                               cudaStream_t stream);
uint32_t varlen_umma_status(bool clear);

// ---- rotary positions with the K/V write (pa_rope.cu)
struct RopeArgs {
    void* q_out;
    const void* q;
    const void* k;
    const void* v;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    const int64_t* positions;              // [num_axes, n]
    int32_t num_axes;
    const double* inv_freq;    // [rot_dim / 2]
    const int32_t* pair_axis;  // [rot_dim / 2], or nullptr: axis 0
    int32_t rot_dim;
    int interleaved;
    const int64_t* slots;
    int64_t n;
    void* k_cache;
    void* v_cache;
    float* k_scales;
    float* v_scales;
    int32_t num_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t block_size;
    int32_t tpb = 1;  // tokens per CTA (set by the launcher)
};
cudaError_t launch_rope_write(const RopeArgs& a, int dtype, bool fp8, cudaStream_t stream);

// ---- attention weights of cached tokens (pa_weights_simt.cu)
struct WeightArgs {
    float* weights;  // [num_seqs, num_kv_heads, weights_stride]
    int64_t weights_stride;
    const void* q;
    const void* k_cache;
    const float* k_scales;
    const int32_t* block_tables;
    int32_t max_blocks;
    const int32_t* seq_lens;
    const int32_t* cu;  // nullptr: one query per request (row s = request s)
    int32_t num_seqs;
    int32_t total_q;
    int32_t num_heads;
    int32_t num_kv_heads;
    int32_t head_dim;
    int32_t block_size;
    int32_t max_context;
    int32_t window;  // 0: every new token
    int causal;
    float scale_log2;
    int dtype;
    int kv_fp8;
    float2* stats;  // [stat_rows, num_heads]: each counted row's maximum (log2 domain) and 1 / sum
    int stat_rows = 0;
    int stat_pitch = 0;  // WeightStatRows::pitch
    uint32_t* next_item = nullptr;  // two counters (workspace)
    void* dense_keys = nullptr;     // [num_seqs, dense_stride, num_kv_heads, head_dim] of the query's type
    float* key_scales = nullptr;    // [num_seqs, num_kv_heads, dense_stride], times scale_log2
    int dense_stride = 0;
    float* tile_stats = nullptr;
    int stat_tiles = 0;
    float* partial = nullptr;
    int key_splits = 1;
    int row_splits = 1;
    int few_rows = 0;
};
// Requests one launch handles (their tile counts' prefix lives in shared memory).
constexpr int kWeightMaxSeqsPerLaunch = 4096;
// Rows of statistics a launch holds.  A window much shorter than the new
// tokens counts few of them: request s of the launch then has `pitch` rows
// from s * pitch on; otherwise (pitch 0) they lie as q's rows do.
struct WeightStatRows {
    int32_t rows, pitch;
};
inline WeightStatRows weight_stat_rows(int32_t seqs, int32_t total_q, int32_t window) {
    if (window > 0 && (int64_t)seqs * window < total_q) return {seqs * window, window};
    return {total_q, 0};
}
cudaError_t launch_weights_simt(const WeightArgs& a, cudaStream_t stream);
// The same on the tensor cores (pa_weights_umma.cu), which cut the work as
// their plan says.  stats then holds key_splits pieces of [stat_rows, num_heads]
// (maximum, sum), partial row_splits pieces of [num_seqs, num_kv_heads,
// max_context].
struct WeightPlan {
    int seqs = 0;           // requests per launch
    int key_splits = 1;
    int row_splits = 1;
    bool few_rows = false;  // row_splits then cuts the keys, without partial weights
    int stat_tiles = 0;     // tile_stats: [num_kv_heads, stat_tiles, 2, 128]
    int dense_stride = 0;   // tokens per request of a dense copy of the keys; 0: read in place
    size_t stats_bytes = 0, tile_stats_bytes = 0, partial_bytes = 0, dense_bytes = 0, scale_bytes = 0;
};
bool weights_umma_supported(int dtype, int head_dim, int group);
WeightPlan weights_umma_plan(int32_t num_seqs, int32_t total_q, int32_t max_q, int32_t num_heads,
                             int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t max_context,
                             int32_t window, bool kv_fp8);
cudaError_t launch_weights_umma(const WeightArgs& a, int32_t num_blocks, std::string* err, cudaStream_t stream);
uint32_t weights_umma_status(bool clear);

// ---- eviction by accumulated weight (pa_evict.cu)
struct EvictArgs {
    float* weights_out;
    int32_t* positions_out;  // may be nullptr
    int32_t* new_lens;
    const float* weights;
    const int32_t* positions;      // read below recorded_lens only
    const int32_t* recorded_lens;  // nullptr: none recorded
    const int32_t* seen_lens;      // nullptr: context_lens
    int64_t stride;
    void* k_cache;
    void* v_cache;
    float* k_scales;  // code pools only
    float* v_scales;
    const int32_t* block_tables;
    int32_t max_blocks;
    const int32_t* new_block_tables;
    int32_t new_max_blocks;
    const int32_t* context_lens;
    int32_t num_seqs;
    int32_t num_kv_heads;
    int32_t block_size;
    int32_t max_context;
    int32_t keep;
    int32_t num_sink;
    int32_t num_recent;
    int64_t row_bytes;  // of one head's K (or V) row
    // workspace (set by the launcher): rows to copy per (sequence, KV head),
    // -1 for all by index; their (source, destination) slots; movers by rank
    int32_t* counts = nullptr;
    int2* list = nullptr;
    int32_t* movers = nullptr;
    int64_t list_stride = 0;
};
// Longest context (the select kernel's bit mask lives in shared memory).
constexpr int32_t kEvictMaxContext = 1 << 19;
size_t evict_workspace(int32_t num_seqs, int32_t num_kv_heads, int32_t max_context, int32_t keep);
cudaError_t launch_evict(const EvictArgs& a, void* workspace, cudaStream_t stream);

// ---- latent cache: the write (pa_latent_write.cu) and attention over it
struct LatentWriteArgs {
    void* q_out;
    const void* q;
    const void* kv;
    int64_t q_out_stride, q_out_head_stride, q_stride, q_head_stride, kv_stride;  // in elements
    const void* norm_weight;  // [latent_dim], or nullptr: no norm
    float eps;
    const int64_t* positions;
    const double* inv_freq;  // [rope_dim / 2]
    int32_t rope_dim;
    int interleaved;
    const int64_t* slots;
    int64_t n;
    void* cache;
    int32_t num_heads;  // 0: no queries
    int32_t latent_dim;
    int32_t tpb = 1;  // tokens per CTA (set by the launcher)
};
cudaError_t launch_latent_write(const LatentWriteArgs& a, int dtype, cudaStream_t stream);

struct LatentArgs {
    void* out;      // [total_q, num_heads, latent_dim]
    const void* q;  // [total_q, num_heads, latent_dim + rope_dim]
    const void* cache;
    const int32_t* block_tables;
    int32_t max_blocks;
    const int32_t* seq_lens;
    const int32_t* cu;  // nullptr: one query per sequence (row s = sequence s)
    int32_t num_seqs;
    int32_t total_q;
    int32_t num_heads;
    int32_t latent_dim;
    int32_t rope_dim;
    int32_t block_size;
    int32_t max_context;
    float scale;
    int causal;
    int dtype;
};
bool latent_simt_supported(int dtype, int32_t row_dim);  // pa_latent_simt.cu
// Bytes for pieces of the rows' keys (few rows), and the launch with them.
size_t latent_simt_workspace(int64_t total_q, int32_t num_heads, int32_t latent_dim, int32_t max_context);
cudaError_t launch_latent_simt(const LatentArgs& a, void* workspace, cudaStream_t stream);
// The same on the tensor cores (pa_latent_umma.cu).  total_q * num_heads and
// the key tiles of a launch must fit in int32.
bool latent_umma_supported(int dtype, int32_t latent_dim, int32_t rope_dim, int32_t block_size);
size_t latent_umma_workspace(int64_t rows);  // rows of a request at most (num_heads per token)
cudaError_t launch_latent_umma(const LatentArgs& a, int32_t num_blocks, void* workspace, std::string* err,
                               cudaStream_t stream);
uint32_t latent_umma_status(bool clear);

// ---- decode of shared prefixes (pa_prefix_umma.cu, pa_decode_shared.cu)
struct SharedGroups;  // pa_shared.cuh
cudaError_t launch_prefix_umma(const AttnArgs& a, const SharedGroups& g, int32_t num_blocks, int ctas,
                               std::string* err, cudaStream_t stream);
uint32_t prefix_umma_status(bool clear);
// Whether the prefixes are worked apart (otherwise the call is the plain decode).
bool decode_shared_supported(int dtype, int head_dim, int block_size, int group, int32_t num_seqs, int32_t num_groups,
                             int32_t max_context);
// Bytes beside the plain decode's workspace for `grid_ctas`.
size_t decode_shared_workspace(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                               int32_t block_size, int32_t max_context, int grid_ctas);
int decode_shared_grid(int32_t num_seqs, int32_t num_kv_heads, int32_t head_dim, int32_t max_context, int dtype,
                       int32_t group, int64_t ctas_override);
cudaError_t launch_decode_shared(const AttnArgs& a, const int32_t* group_starts, const int32_t* prefix_lens,
                                 int32_t num_groups, int32_t num_blocks, int grid_ctas, void* workspace,
                                 std::string* err, cudaStream_t stream);
uint32_t decode_shared_status(bool clear);

// SMs of the current device.
int sm_count();

}  // namespace pa
