// pa_api.cu -- the extern "C" entry points declared in include/pa.h:
// argument validation, optional host-side index checking, and dispatch to
// the kernels' launchers.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <exception>
#include <string>
#include <unordered_map>
#include <unordered_set>
#include <vector>

#include "../../include/pa.h"
#include "pa_internal.h"

namespace {

thread_local std::string g_last_error;
int64_t g_options[5] = {0, 0, 0, 0, 0};
constexpr int32_t kPairMinContext = 2048;  // automatic pair steps above this max_context

pa_status fail(pa_status st, const std::string& msg) {
    g_last_error = msg;
    return st;
}

pa_status cuda_fail(cudaError_t e, const char* where) {
    return fail(PA_ERR_CUDA, std::string(where) + ": " + cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool valid_dtype(int d) { return d == PA_F32 || d == PA_BF16 || d == PA_F16; }
cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }

// The answer of a check that ran out of host memory (no exception leaves a C
// entry point).
pa_status no_host_memory() { return fail(PA_ERR_INVALID_ARG, "check mode: no host memory for the index arrays"); }

template <typename T>
bool to_host(std::vector<T>& dst, const T* src, int64_t n, cudaStream_t st, pa_status* err) {
    try {
        dst.resize((size_t)std::max<int64_t>(n, 0));
    } catch (const std::exception&) {
        *err = no_host_memory();
        return false;
    }
    if (n <= 0) return true;
    cudaError_t e = cudaMemcpyAsync(dst.data(), src, sizeof(T) * (size_t)n, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e != cudaSuccess) {
        *err = cuda_fail(e, "check mode: copying indices to the host");
        return false;
    }
    return true;
}

bool check_mode() { return g_options[PA_OPT_CHECK_MODE] != 0; }

// Check-mode validation of block tables against lengths.
pa_status check_tables(const int32_t* block_tables, int32_t num_seqs, int32_t max_blocks, const std::vector<int32_t>& lens,
                       int32_t num_blocks, int32_t block_size, int32_t max_context, cudaStream_t st) {
    pa_status err = PA_OK;
    std::vector<int32_t> bt;
    if (!to_host(bt, block_tables, (int64_t)num_seqs * max_blocks, st, &err)) return err;
    for (int32_t s = 0; s < num_seqs; ++s) {
        const int32_t L = lens[s];
        if (L < 0 || L > max_context)
            return fail(PA_ERR_INDEX, "sequence " + std::to_string(s) + ": length " + std::to_string(L) +
                                          " outside [0, max_context=" + std::to_string(max_context) + "]");
        const int64_t nb = ((int64_t)L + block_size - 1) / block_size;
        if (nb > max_blocks)
            return fail(PA_ERR_INDEX, "sequence " + std::to_string(s) + " needs " + std::to_string(nb) +
                                          " blocks but the table holds " + std::to_string(max_blocks));
        for (int64_t b = 0; b < nb; ++b) {
            const int32_t id = bt[(size_t)s * max_blocks + b];
            if (id < 0 || id >= num_blocks)
                return fail(PA_ERR_INDEX, "sequence " + std::to_string(s) + " logical block " + std::to_string(b) +
                                              " maps to " + std::to_string(id) + ", outside [0, num_blocks)");
        }
    }
    return PA_OK;
}

// bytes_only: the call moves bytes (copy, swap), so PA_FP8_E4M3 pools are
// accepted as well.
pa_status check_geometry(int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks,
                         int32_t block_size, int dtype, bool bytes_only = false) {
    if (!valid_dtype(dtype) && !(bytes_only && dtype == PA_FP8_E4M3))
        return fail(PA_ERR_INVALID_ARG, bytes_only ? "dtype must be PA_F32, PA_BF16, PA_F16 or PA_FP8_E4M3"
                                                   : "dtype must be PA_F32, PA_BF16 or PA_F16");
    if (num_kv_heads <= 0 || num_heads <= 0 || head_dim <= 0 || num_blocks <= 0 || block_size <= 0)
        return fail(PA_ERR_INVALID_ARG, "head counts, head_dim, num_blocks and block_size must be positive");
    if (num_heads % num_kv_heads != 0)
        return fail(PA_ERR_INVALID_ARG, "num_heads must be a multiple of num_kv_heads");
    if ((int64_t)num_blocks * block_size > INT32_MAX)
        return fail(PA_ERR_UNSUPPORTED, "num_blocks * block_size must fit in int32");
    return PA_OK;
}

// Check-mode validation of a slot mapping: in the pool, or negative (skip); distinct.
pa_status check_slots(const int64_t* slot_mapping, int64_t n, int32_t num_blocks, int32_t block_size,
                      cudaStream_t st) {
    pa_status err = PA_OK;
    std::vector<int64_t> sm;
    if (!to_host(sm, slot_mapping, n, st, &err)) return err;
    const int64_t slots = (int64_t)num_blocks * block_size;
    std::unordered_set<int64_t> seen;
    try {
        for (int64_t i = 0; i < n; ++i) {
            if (sm[i] < 0) continue;
            if (sm[i] >= slots)
                return fail(PA_ERR_INDEX, "token " + std::to_string(i) + ": slot " + std::to_string(sm[i]) +
                                              " outside the pool");
            if (!seen.insert(sm[i]).second)
                return fail(PA_ERR_INDEX, "slot " + std::to_string(sm[i]) + " written twice in one call");
        }
    } catch (const std::exception&) {
        return no_host_memory();
    }
    return PA_OK;
}

// Check-mode validation of a varlen batch: cu_seqlens_q, lengths and tables.
pa_status check_varlen(const int32_t* block_tables, int32_t max_blocks, const int32_t* seq_lens,
                       const int32_t* cu_seqlens_q, int32_t num_seqs, int32_t total_q, int32_t max_q,
                       int32_t num_blocks, int32_t block_size, int32_t max_context, cudaStream_t st) {
    pa_status err = PA_OK;
    std::vector<int32_t> lens, cu;
    if (!to_host(lens, seq_lens, num_seqs, st, &err) || !to_host(cu, cu_seqlens_q, num_seqs + 1, st, &err))
        return err;
    if (cu[0] != 0 || cu[num_seqs] != total_q)
        return fail(PA_ERR_INDEX, "cu_seqlens_q must start at 0 and end at total_q");
    for (int32_t i = 0; i < num_seqs; ++i) {
        const int32_t nn = cu[i + 1] - cu[i];
        if (nn < 0) return fail(PA_ERR_INDEX, "cu_seqlens_q must be non-decreasing");
        if (nn > max_q) return fail(PA_ERR_INDEX, "request " + std::to_string(i) + " has more than max_q queries");
        if (nn > lens[i])
            return fail(PA_ERR_INDEX, "request " + std::to_string(i) + " has more new tokens than context");
    }
    return check_tables(block_tables, num_seqs, max_blocks, lens, num_blocks, block_size, max_context, st);
}

// Check-mode validation of an eviction: lengths, both tables, and that a
// block that may be written is read or written for one (sequence, logical
// block) only.
pa_status check_evict(const int32_t* recorded_lens, const int32_t* seen_lens, const int32_t* block_tables, int32_t max_blocks,
                      const int32_t* new_block_tables, int32_t new_max_blocks, const int32_t* context_lens,
                      int32_t num_seqs, int32_t num_blocks, int32_t block_size, int32_t max_context, int32_t keep,
                      cudaStream_t st) {
    pa_status err = PA_OK;
    std::vector<int32_t> lens, kept, rec, seen, from, to;
    if (!to_host(lens, context_lens, num_seqs, st, &err)) return err;
    err = check_tables(block_tables, num_seqs, max_blocks, lens, num_blocks, block_size, max_context, st);
    if (err != PA_OK) return err;
    if (!to_host(kept, context_lens, num_seqs, st, &err)) return err;
    for (int32_t& L : kept) L = std::min(L, keep);
    err = check_tables(new_block_tables, num_seqs, new_max_blocks, kept, num_blocks, block_size, max_context, st);
    if (err != PA_OK) return err;
    if (recorded_lens && !to_host(rec, recorded_lens, num_seqs, st, &err)) return err;
    if (seen_lens && !to_host(seen, seen_lens, num_seqs, st, &err)) return err;
    for (int32_t s = 0; s < num_seqs; ++s) {
        if (recorded_lens && (rec[s] < 0 || rec[s] > lens[s]))
            return fail(PA_ERR_INDEX, "sequence " + std::to_string(s) + ": recorded_lens outside [0, context length]");
        if (seen_lens && seen[s] < lens[s])
            return fail(PA_ERR_INDEX, "sequence " + std::to_string(s) + ": seen_lens below the context length");
    }
    if (!to_host(from, block_tables, (int64_t)num_seqs * max_blocks, st, &err) ||
        !to_host(to, new_block_tables, (int64_t)num_seqs * new_max_blocks, st, &err))
        return err;
    // who reads and who writes a block: its (sequence, logical block), or several
    constexpr int64_t kNobody = -1, kSeveral = -2;
    struct Users {
        int64_t reader = kNobody, writer = kNobody;
    };
    std::unordered_map<int32_t, Users> users;
    try {
        for (int32_t s = 0; s < num_seqs; ++s)
            for (int64_t b = 0; b * block_size < lens[s]; ++b) {
                int64_t& r = users[from[(size_t)s * max_blocks + b]].reader;
                r = r == kNobody ? ((int64_t)s << 32 | b) : kSeveral;
            }
        for (int32_t s = 0; s < num_seqs; ++s)
            for (int64_t b = 0; b * block_size < kept[s]; ++b) {
                const int32_t id = to[(size_t)s * new_max_blocks + b];
                const int64_t me = (int64_t)s << 32 | b;
                if (id == from[(size_t)s * max_blocks + b] && lens[s] <= keep) continue;  // in place, nothing dropped
                Users& u = users[id];
                if (u.writer != kNobody)
                    return fail(PA_ERR_INDEX, "block " + std::to_string(id) + " is the destination of two blocks");
                u.writer = me;
                if (u.reader != kNobody && u.reader != me)
                    return fail(PA_ERR_INDEX, "block " + std::to_string(id) +
                                                  " is written for one sequence and read for another logical block");
            }
    } catch (const std::exception&) {
        return no_host_memory();
    }
    return PA_OK;
}

}  // namespace

namespace pa {
// Sets the reason pa_last_error() reports (used by entry points defined in
// other translation units).
void record_error(const std::string& msg) { g_last_error = msg; }

bool check_mode_on() { return check_mode(); }

int sm_count() {
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

int check_decode_indices(const int32_t* block_tables, int32_t max_blocks, const int32_t* context_lens,
                         int32_t num_seqs, int32_t num_blocks, int32_t block_size, int32_t max_context,
                         cudaStream_t stream) {
    pa_status err = PA_OK;
    std::vector<int32_t> lens;
    if (!to_host(lens, context_lens, num_seqs, stream, &err)) return err;
    return check_tables(block_tables, num_seqs, max_blocks, lens, num_blocks, block_size, max_context, stream);
}
}  // namespace pa

extern "C" {

const char* pa_status_string(int status) {
    switch (status) {
        case PA_OK: return "PA_OK";
        case PA_ERR_INVALID_ARG: return "PA_ERR_INVALID_ARG";
        case PA_ERR_UNSUPPORTED: return "PA_ERR_UNSUPPORTED";
        case PA_ERR_INDEX: return "PA_ERR_INDEX";
        case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE";
        case PA_ERR_CUDA: return "PA_ERR_CUDA";
        case PA_ERR_TIMEOUT: return "PA_ERR_TIMEOUT";
        default: return "unknown pa_status";
    }
}

const char* pa_last_error(void) { return g_last_error.c_str(); }

pa_status pa_set_option(int option, int64_t value) {
    if (option < 0 || option > PA_OPT_FP8_PAIR_STEP) return fail(PA_ERR_INVALID_ARG, "unknown option");
    if ((option == PA_OPT_DECODE_KERNEL && value > 2) || (option == PA_OPT_VARLEN_KERNEL && value > 2) ||
        (option == PA_OPT_FP8_PAIR_STEP && value > 2))
        return fail(PA_ERR_INVALID_ARG, "unknown kernel choice");
    if (value < 0) return fail(PA_ERR_INVALID_ARG, "option values are non-negative");
    g_options[option] = value;
    return PA_OK;
}

int64_t pa_get_option(int option) {
    if (option < 0 || option > PA_OPT_FP8_PAIR_STEP) return -1;
    return g_options[option];
}

pa_status pa_set_check_mode(int on) { return pa_set_option(PA_OPT_CHECK_MODE, on ? 1 : 0); }

pa_status pa_device_status(int clear) {
    cudaError_t e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return cuda_fail(e, "pa_device_status");
    const uint32_t bits =
        pa::decode_tc_status(clear != 0) | pa::decode_weights_status(clear != 0) |
                          pa::varlen_umma_status(clear != 0) | pa::weights_umma_status(clear != 0) |
                          pa::latent_umma_status(clear != 0) | pa::prefix_umma_status(clear != 0) |
                          pa::decode_shared_status(clear != 0) |
                          pa::selftest_status(clear != 0);
    if (bits & 1u) return fail(PA_ERR_TIMEOUT, "a kernel's bounded barrier wait ran out");
    return PA_OK;
}

pa_status pa_selftest_wait_timeout(int32_t polls, void* stream) {
    if (polls < 1 || polls > (1 << 20)) return fail(PA_ERR_INVALID_ARG, "polls must be in [1, 2^20]");
    cudaError_t e = pa::launch_selftest_wait((uint32_t)polls, as_stream(stream));
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "pa_selftest_wait_timeout launch");
}

pa_status pa_slot_mapping(const int32_t* block_tables, int32_t num_seqs, int32_t max_blocks, const int32_t* seq_idx,
                          const int64_t* positions, int64_t n, int32_t block_size, int64_t* slot_out,
                          void* stream) {
    if (n < 0 || num_seqs < 0 || max_blocks < 0 || block_size <= 0)
        return fail(PA_ERR_INVALID_ARG, "sizes must be non-negative and block_size positive");
    if (n == 0) return PA_OK;
    if (!block_tables || !seq_idx || !positions || !slot_out) return fail(PA_ERR_INVALID_ARG, "null pointer");
    cudaStream_t st = as_stream(stream);
    if (check_mode()) {
        pa_status err = PA_OK;
        std::vector<int32_t> si;
        std::vector<int64_t> pos;
        if (!to_host(si, seq_idx, n, st, &err) || !to_host(pos, positions, n, st, &err)) return err;
        for (int64_t i = 0; i < n; ++i) {
            if (pos[i] < 0) continue;
            if (si[i] < 0 || si[i] >= num_seqs)
                return fail(PA_ERR_INDEX, "token " + std::to_string(i) + ": sequence index out of range");
            if (pos[i] / block_size >= max_blocks)
                return fail(PA_ERR_INDEX, "token " + std::to_string(i) + ": position beyond the block table");
        }
    }
    cudaError_t e = pa::launch_slot_mapping(block_tables, max_blocks, seq_idx, positions, n, block_size, slot_out, st);
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "pa_slot_mapping launch");
}

pa_status pa_write_kv(const void* k, const void* v, const int64_t* slot_mapping, int64_t n, void* k_cache,
                      void* v_cache, int32_t num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim,
                      int dtype, void* stream) {
    pa_status g = check_geometry(num_kv_heads, num_kv_heads, head_dim, num_blocks, block_size, dtype);
    if (g != PA_OK) return g;
    if (n < 0) return fail(PA_ERR_INVALID_ARG, "n must be non-negative");
    if (n == 0) return PA_OK;
    if (!k || !v || !slot_mapping || !k_cache || !v_cache) return fail(PA_ERR_INVALID_ARG, "null pointer");
    const int64_t row_bytes = (int64_t)num_kv_heads * head_dim * pa::elt_size(dtype);
    if (row_bytes % 16 != 0)
        return fail(PA_ERR_UNSUPPORTED, "num_kv_heads * head_dim * element size must be a multiple of 16 bytes");
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
        return fail(PA_ERR_INVALID_ARG, "k, v and the caches must be 16-byte aligned");
    cudaStream_t st = as_stream(stream);
    if (check_mode()) {
        pa_status err = check_slots(slot_mapping, n, num_blocks, block_size, st);
        if (err != PA_OK) return err;
    }
    cudaError_t e = pa::launch_write_kv(k, v, slot_mapping, n, k_cache, v_cache, row_bytes, st);
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "pa_write_kv launch");
}

pa_status pa_write_kv_fp8(const void* k, const void* v, const int64_t* slot_mapping, int64_t n, void* k_codes,
                          void* v_codes, float* k_scales, float* v_scales, int32_t num_blocks, int32_t block_size,
                          int32_t num_kv_heads, int32_t head_dim, int dtype, void* stream) {
    pa_status g = check_geometry(num_kv_heads, num_kv_heads, head_dim, num_blocks, block_size, dtype);
    if (g != PA_OK) return g;
    if (head_dim > 256) return fail(PA_ERR_UNSUPPORTED, "head_dim must be at most 256");
    if (n < 0) return fail(PA_ERR_INVALID_ARG, "n must be non-negative");
    if (n == 0) return PA_OK;
    if (!k || !v || !slot_mapping || !k_codes || !v_codes || !k_scales || !v_scales)
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_codes) || !aligned16(v_codes))
        return fail(PA_ERR_INVALID_ARG, "k, v and the code pools must be 16-byte aligned");
    cudaStream_t st = as_stream(stream);
    if (check_mode()) {
        pa_status err = check_slots(slot_mapping, n, num_blocks, block_size, st);
        if (err != PA_OK) return err;
    }
    cudaError_t e = pa::launch_write_kv_fp8(k, v, dtype, slot_mapping, n, num_kv_heads, head_dim, block_size,
                                            static_cast<uint8_t*>(k_codes), static_cast<uint8_t*>(v_codes), k_scales,
                                            v_scales, st);
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "pa_write_kv_fp8 launch");
}

pa_status pa_copy_blocks(void* const* k_caches, void* const* v_caches, int32_t num_layers, const int64_t* block_pairs,
                         int32_t num_pairs, int32_t num_blocks, int32_t block_size, int32_t num_kv_heads,
                         int32_t head_dim, int dtype, void* stream) {
    pa_status g = check_geometry(num_kv_heads, num_kv_heads, head_dim, num_blocks, block_size, dtype, true);
    if (g != PA_OK) return g;
    if (num_pairs < 0) return fail(PA_ERR_INVALID_ARG, "num_pairs must be non-negative");
    if (num_layers < 1 || num_layers > PA_MAX_LAYERS)
        return fail(PA_ERR_INVALID_ARG, "num_layers must be in [1, PA_MAX_LAYERS]");
    if (num_pairs == 0) return PA_OK;
    if (!k_caches || !v_caches || !block_pairs) return fail(PA_ERR_INVALID_ARG, "null pointer");
    for (int l = 0; l < num_layers; ++l) {
        if (!k_caches[l] || !v_caches[l]) return fail(PA_ERR_INVALID_ARG, "null cache pointer");
        if (!aligned16(k_caches[l]) || !aligned16(v_caches[l]))
            return fail(PA_ERR_INVALID_ARG, "caches must be 16-byte aligned");
    }
    const int64_t block_bytes = (int64_t)block_size * num_kv_heads * head_dim * pa::elt_size(dtype);
    if (block_bytes % 16 != 0) return fail(PA_ERR_UNSUPPORTED, "a block must be a multiple of 16 bytes");
    cudaStream_t st = as_stream(stream);
    if (check_mode()) {
        pa_status err = PA_OK;
        std::vector<int64_t> pr;
        if (!to_host(pr, block_pairs, 2 * (int64_t)num_pairs, st, &err)) return err;
        std::unordered_set<int64_t> dsts, srcs;
        for (int32_t p = 0; p < num_pairs; ++p) {
            const int64_t s = pr[2 * p], d = pr[2 * p + 1];
            if (s < 0 || s >= num_blocks || d < 0 || d >= num_blocks)
                return fail(PA_ERR_INDEX, "pair " + std::to_string(p) + ": block id outside [0, num_blocks)");
            if (!dsts.insert(d).second)
                return fail(PA_ERR_INDEX, "block " + std::to_string(d) + " is the destination of two pairs");
            srcs.insert(s);
        }
        for (int32_t p = 0; p < num_pairs; ++p) {
            const int64_t s = pr[2 * p], d = pr[2 * p + 1];
            if (d != s && srcs.count(d))
                return fail(PA_ERR_INDEX, "block " + std::to_string(d) + " is both a destination and a source");
        }
    }
    cudaError_t e = pa::launch_copy_blocks(k_caches, v_caches, num_layers, block_pairs, num_pairs, block_bytes, st);
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "pa_copy_blocks launch");
}

// Device address a kernel can use for p: device memory as is, pinned or
// registered host memory through its device mapping; nullptr otherwise.
static const void* device_view(const void* p) {
    cudaPointerAttributes at;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();
        return nullptr;
    }
    if (at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged) return p;
    if (at.type == cudaMemoryTypeHost && at.devicePointer) {
        const uint8_t* base = static_cast<const uint8_t*>(at.hostPointer);
        return static_cast<const uint8_t*>(at.devicePointer) + (static_cast<const uint8_t*>(p) - base);
    }
    return nullptr;
}

pa_status pa_swap_blocks(void* const* src_k, void* const* src_v, void* const* dst_k, void* const* dst_v,
                         int32_t num_layers, const int64_t* block_pairs, int32_t num_pairs, int32_t src_num_blocks,
                         int32_t dst_num_blocks, int32_t block_size, int32_t num_kv_heads, int32_t head_dim, int dtype,
                         void* stream) {
    if (num_pairs < 0 || src_num_blocks <= 0 || dst_num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARG, "num_pairs must be non-negative and both pools non-empty");
    pa_status g = check_geometry(num_kv_heads, num_kv_heads, head_dim, src_num_blocks, block_size, dtype, true);
    if (g != PA_OK) return g;
    if (num_layers < 1 || num_layers > PA_MAX_LAYERS)
        return fail(PA_ERR_INVALID_ARG, "num_layers must be in [1, PA_MAX_LAYERS]");
    if (num_pairs == 0) return PA_OK;
    if (!src_k || !src_v || !dst_k || !dst_v || !block_pairs) return fail(PA_ERR_INVALID_ARG, "null pointer");
    const int64_t block_bytes = (int64_t)block_size * num_kv_heads * head_dim * pa::elt_size(dtype);
    if (block_bytes % 16 != 0) return fail(PA_ERR_UNSUPPORTED, "a block must be a multiple of 16 bytes");
    std::vector<void*> sk(num_layers), sv(num_layers), dk(num_layers), dv(num_layers);
    for (int l = 0; l < num_layers; ++l) {
        const void* in[4] = {src_k[l], src_v[l], dst_k[l], dst_v[l]};
        void** out[4] = {&sk[l], &sv[l], &dk[l], &dv[l]};
        for (int i = 0; i < 4; ++i) {
            if (!in[i] || !aligned16(in[i])) return fail(PA_ERR_INVALID_ARG, "pools must be non-null and 16-byte aligned");
            const void* d = device_view(in[i]);
            if (!d)
                return fail(PA_ERR_INVALID_ARG, "a pool is neither device memory nor pinned/registered host memory");
            *out[i] = const_cast<void*>(d);
        }
    }
    const void* pairs_dev = device_view(block_pairs);
    if (!pairs_dev) return fail(PA_ERR_INVALID_ARG, "block_pairs must be device or pinned host memory");
    cudaStream_t st = as_stream(stream);
    if (check_mode()) {
        pa_status err = PA_OK;
        std::vector<int64_t> pr;
        if (!to_host(pr, static_cast<const int64_t*>(pairs_dev), 2 * (int64_t)num_pairs, st, &err)) return err;
        std::unordered_set<int64_t> dsts;
        for (int32_t p = 0; p < num_pairs; ++p) {
            const int64_t s = pr[2 * p], d = pr[2 * p + 1];
            if (s < 0 || s >= src_num_blocks || d < 0 || d >= dst_num_blocks)
                return fail(PA_ERR_INDEX, "pair " + std::to_string(p) + ": block id outside its pool");
            if (!dsts.insert(d).second)
                return fail(PA_ERR_INDEX, "block " + std::to_string(d) + " is the destination of two pairs");
        }
    }
    cudaError_t e = pa::launch_swap_blocks(sk.data(), sv.data(), dk.data(), dv.data(), num_layers,
                                           static_cast<const int64_t*>(pairs_dev), num_pairs, block_bytes, st);
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "pa_swap_blocks launch");
}

// ------------------------------------------------------------------ decode

static bool use_decode_tc(int dtype, int head_dim, int block_size, int group, bool kv_fp8, pa_status* st) {
    const int64_t want = g_options[PA_OPT_DECODE_KERNEL];
    const bool ok = pa::decode_tc_supported(dtype, head_dim, block_size, group, kv_fp8);
    *st = PA_OK;
    if (want == 1) return false;
    if (want == 2 && !ok) {
        *st = fail(PA_ERR_UNSUPPORTED, kv_fp8 ? "the tensor-core decode kernel over an FP8 cache takes bf16/f16 "
                                                "queries, head_dim 128/256, block_size 8 or a multiple of 16 up "
                                                "to 256, and at most 16 query heads per KV head"
                                              : "the tensor-core decode kernel takes bf16/f16, head_dim 64/128/256 "
                                                "and at most 16 query heads per KV head");
        return false;
    }
    return ok;
}

static size_t decode_workspace(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                               int32_t block_size, int32_t max_context, int dtype, bool kv_fp8) {
    if (num_seqs <= 0 || num_kv_heads <= 0 || num_heads <= 0 || num_heads % num_kv_heads || max_context < 0)
        return 0;
    pa_status st;
    const int G = num_heads / num_kv_heads;
    if (!use_decode_tc(dtype, head_dim, block_size, G, kv_fp8, &st)) return 0;
    const int grid = pa::decode_tc_grid(num_seqs, num_kv_heads, head_dim, block_size, max_context, dtype, G,
                                        g_options[PA_OPT_DECODE_CTAS], kv_fp8);
    return pa::decode_tc_workspace(num_seqs, num_kv_heads, G, head_dim, grid, kv_fp8);
}

size_t pa_decode_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                int32_t block_size, int32_t max_context, int dtype) {
    return decode_workspace(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype, false);
}

size_t pa_decode_fp8_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                    int32_t block_size, int32_t max_context, int dtype) {
    return decode_workspace(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype, true);
}

}  // extern "C"

// The decode's argument checks and kernel arguments.  k_scales != nullptr: the
// caches hold E4M3 codes with these scales.
static pa_status decode_args(pa::AttnArgs& a, void* out, const void* q, const void* k_new, const void* v_new,
                             const void* k_cache, const void* v_cache, const float* k_scales, const float* v_scales,
                             const int32_t* block_tables, int32_t max_blocks, const int32_t* context_lens,
                             int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                             int32_t num_blocks, int32_t block_size, int32_t max_context, float scale, int dtype,
                             cudaStream_t st) {
    const bool fp8 = k_scales != nullptr;
    pa_status g = check_geometry(num_heads, num_kv_heads, head_dim, num_blocks, block_size, dtype);
    if (g != PA_OK) return g;
    if (num_seqs < 0 || max_blocks < 0 || max_context < 0)
        return fail(PA_ERR_INVALID_ARG, "num_seqs, max_blocks and max_context must be non-negative");
    if (num_seqs == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens)
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    const bool append = k_new != nullptr || v_new != nullptr;
    if (append && (!k_new || !v_new)) return fail(PA_ERR_INVALID_ARG, "k_new and v_new go together");
    if (append && (!aligned16(k_new) || !aligned16(v_new)))
        return fail(PA_ERR_INVALID_ARG, "k_new and v_new must be 16-byte aligned");
    if (append && ((int64_t)num_kv_heads * head_dim * pa::elt_size(dtype)) % 16 != 0)
        return fail(PA_ERR_UNSUPPORTED, "num_kv_heads * head_dim * element size must be a multiple of 16 bytes");
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
        return fail(PA_ERR_INVALID_ARG, "out, q and the caches must be 16-byte aligned");
    if (!pa::attn_simt_supported(dtype, head_dim)) return fail(PA_ERR_UNSUPPORTED, "head_dim must be in [1, 256]");
    if (fp8 && (!v_scales || !aligned16(k_scales) || !aligned16(v_scales)))
        return fail(PA_ERR_INVALID_ARG, "k_scales and v_scales must be non-null and 16-byte aligned");
    if (check_mode()) {
        pa_status err = PA_OK;
        std::vector<int32_t> lens;
        if (!to_host(lens, context_lens, num_seqs, st, &err)) return err;
        err = check_tables(block_tables, num_seqs, max_blocks, lens, num_blocks, block_size, max_context, st);
        if (err != PA_OK) return err;
    }
    a.out = out;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.max_blocks = max_blocks;
    a.seq_lens = context_lens;
    a.cu_seqlens_q = nullptr;
    a.num_seqs = num_seqs;
    a.total_q = num_seqs;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.block_size = block_size;
    a.scale = scale;
    a.causal = 1;
    a.dtype = dtype;
    a.max_context = max_context;
    a.kv_fp8 = fp8 ? 1 : 0;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    return PA_OK;
}

// Sequences s0 .. s0 + count - 1 of a.
static pa::AttnArgs decode_part(const pa::AttnArgs& a, int32_t s0, int32_t count) {
    const int64_t row = (int64_t)a.num_heads * a.head_dim * pa::elt_size(a.dtype);
    pa::AttnArgs c = a;
    c.num_seqs = count;
    c.total_q = count;
    c.out = static_cast<uint8_t*>(a.out) + s0 * row;
    c.q = static_cast<const uint8_t*>(a.q) + s0 * row;
    c.block_tables = a.block_tables + (int64_t)s0 * a.max_blocks;
    c.seq_lens = a.seq_lens + s0;
    return c;
}

static pa_status decode_impl(void* out, const void* q, const void* k_new, const void* v_new, const void* k_cache,
                             const void* v_cache, const float* k_scales, const float* v_scales,
                             const int32_t* block_tables, int32_t max_blocks, const int32_t* context_lens,
                             int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                             int32_t num_blocks, int32_t block_size, int32_t max_context, float scale, int dtype,
                             void* workspace, size_t workspace_bytes, void* stream) {
    const bool fp8 = k_scales != nullptr;
    const bool append = k_new != nullptr || v_new != nullptr;
    cudaStream_t st = as_stream(stream);
    pa::AttnArgs a{};
    pa_status g = decode_args(a, out, q, k_new, v_new, k_cache, v_cache, k_scales, v_scales, block_tables, max_blocks,
                              context_lens, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks, block_size,
                              max_context, scale, dtype, st);
    if (g != PA_OK || num_seqs == 0) return g;
    const int G = num_heads / num_kv_heads;
    const int64_t row_bytes = (int64_t)num_kv_heads * head_dim * pa::elt_size(dtype);
    pa_status sel;
    const bool tc = use_decode_tc(dtype, head_dim, block_size, G, fp8, &sel);
    if (sel != PA_OK) return sel;
    // The tensor-core kernel fuses the append for 16-bit caches, and for code
    // caches of head_dim 128 when the batch has no more (sequence, KV head)
    // units than the grid has warps: quantizing inside the kernel costs the
    // warp that owns a unit's last tile some microseconds (measured: a gain
    // with 512 units on 1,824 warps, a loss with 5,120), while a separate
    // quantizing kernel spreads the rows over the whole GPU.  Otherwise the
    // new rows are written (quantized for a code cache) by a separate kernel
    // first, then attended from the pool; either way the pool and the output
    // are the same bit for bit.
    bool fused_append = append && tc && (!fp8 || head_dim == 128);
    if (fused_append && fp8) {
        const int64_t warps = (int64_t)pa::decode_tc_grid(num_seqs, num_kv_heads, head_dim, block_size, max_context,
                                                          dtype, G, g_options[PA_OPT_DECODE_CTAS], fp8) *
                              pa::decode_tc_warps_per_cta(head_dim, fp8);
        fused_append = (int64_t)num_seqs * num_kv_heads <= warps;
    }
    if (append && !fused_append) {
        cudaError_t e = fp8 ? pa::launch_append_kv_fp8(k_new, v_new, dtype, block_tables, max_blocks, context_lens,
                                                       num_seqs, num_kv_heads, head_dim, block_size,
                                                       static_cast<uint8_t*>(const_cast<void*>(k_cache)),
                                                       static_cast<uint8_t*>(const_cast<void*>(v_cache)),
                                                       const_cast<float*>(k_scales), const_cast<float*>(v_scales), st)
                            : pa::launch_append_kv(k_new, v_new, block_tables, max_blocks, context_lens, num_seqs,
                                                   block_size, const_cast<void*>(k_cache),
                                                   const_cast<void*>(v_cache), row_bytes, st);
        if (e != cudaSuccess) return cuda_fail(e, "pa_decode_append launch");
    }
    if (!tc) {
        cudaError_t e = pa::launch_attn_simt(a, st);
        return e == cudaSuccess ? PA_OK : cuda_fail(e, "pa_decode launch");
    }
    const int grid = pa::decode_tc_grid(num_seqs, num_kv_heads, head_dim, block_size, max_context, dtype, G,
                                        g_options[PA_OPT_DECODE_CTAS], fp8);
    const size_t need = pa::decode_tc_workspace(num_seqs, num_kv_heads, G, head_dim, grid, fp8);
    // Code cache, head_dim 128: the 32-token pair step pays where units are
    // long (measured: 8 x 32k tokens 7 % faster, the 64-sequence batch of up
    // to 3,360 tokens 1 %) and loses where many units are short (128
    // sequences of mean 480 tokens: 8 % slower, the split then leaves some
    // warps with many single tiles).  max_context is the host's only view
    // of the lengths.
    const int64_t pair_opt = g_options[PA_OPT_FP8_PAIR_STEP];
    a.pair_steps = fp8 && head_dim == 128 && (pair_opt == 2 || (pair_opt == 0 && max_context > kPairMinContext));
    if (workspace_bytes < need || (need && !workspace))
        return fail(PA_ERR_WORKSPACE, "workspace holds " + std::to_string(workspace_bytes) + " bytes, " +
                                          std::to_string(need) + " needed");
    if (!aligned16(workspace)) return fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    for (int32_t s0 = 0; s0 < num_seqs; s0 += pa::kDecodeMaxSeqsPerLaunch) {
        pa::AttnArgs c = decode_part(a, s0, std::min(num_seqs - s0, pa::kDecodeMaxSeqsPerLaunch));
        if (fused_append) {
            c.k_new = static_cast<const uint8_t*>(k_new) + (int64_t)s0 * row_bytes;
            c.v_new = static_cast<const uint8_t*>(v_new) + (int64_t)s0 * row_bytes;
        }
        std::string err;
        cudaError_t e = pa::launch_decode_tc(c, num_blocks, grid, workspace, &err, st);
        if (e != cudaSuccess)
            return err.empty() ? cuda_fail(e, "pa_decode launch") : fail(PA_ERR_CUDA, "pa_decode: " + err);
    }
    return PA_OK;
}

extern "C" {

pa_status pa_decode(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                    int32_t max_blocks, const int32_t* context_lens, int32_t num_seqs, int32_t num_heads,
                    int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks, int32_t block_size,
                    int32_t max_context, float scale, int dtype, void* workspace, size_t workspace_bytes,
                    void* stream) {
    return decode_impl(out, q, nullptr, nullptr, k_cache, v_cache, nullptr, nullptr, block_tables, max_blocks,
                       context_lens, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks, block_size, max_context,
                       scale, dtype, workspace, workspace_bytes, stream);
}

pa_status pa_decode_fp8(void* out, const void* q, const void* k_codes, const void* v_codes, const float* k_scales,
                        const float* v_scales, const int32_t* block_tables, int32_t max_blocks,
                        const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                        int32_t head_dim, int32_t num_blocks, int32_t block_size, int32_t max_context, float scale,
                        int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (num_seqs > 0 && (!k_scales || !v_scales)) return fail(PA_ERR_INVALID_ARG, "null pointer");
    return decode_impl(out, q, nullptr, nullptr, k_codes, v_codes, k_scales, v_scales, block_tables, max_blocks,
                       context_lens, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks, block_size, max_context,
                       scale, dtype, workspace, workspace_bytes, stream);
}

pa_status pa_decode_append(void* out, const void* q, const void* k_new, const void* v_new, void* k_cache,
                           void* v_cache, const int32_t* block_tables, int32_t max_blocks,
                           const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                           int32_t head_dim, int32_t num_blocks, int32_t block_size, int32_t max_context,
                           float scale, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (num_seqs > 0 && (!k_new || !v_new)) return fail(PA_ERR_INVALID_ARG, "null pointer");
    return decode_impl(out, q, k_new, v_new, k_cache, v_cache, nullptr, nullptr, block_tables, max_blocks,
                       context_lens, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks, block_size, max_context,
                       scale, dtype, workspace, workspace_bytes, stream);
}

pa_status pa_decode_append_fp8(void* out, const void* q, const void* k_new, const void* v_new, void* k_codes,
                               void* v_codes, float* k_scales, float* v_scales, const int32_t* block_tables,
                               int32_t max_blocks, const int32_t* context_lens, int32_t num_seqs, int32_t num_heads,
                               int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks, int32_t block_size,
                               int32_t max_context, float scale, int dtype, void* workspace, size_t workspace_bytes,
                               void* stream) {
    if (num_seqs > 0 && (!k_new || !v_new || !k_scales || !v_scales)) return fail(PA_ERR_INVALID_ARG, "null pointer");
    return decode_impl(out, q, k_new, v_new, k_codes, v_codes, k_scales, v_scales, block_tables, max_blocks,
                       context_lens, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks, block_size, max_context,
                       scale, dtype, workspace, workspace_bytes, stream);
}

// ------------------------------------------------------------------ varlen

size_t pa_varlen_workspace_size(int32_t num_seqs, int32_t total_q, int32_t max_q, int32_t num_heads,
                                int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t max_context,
                                int dtype) {
    (void)max_q, (void)max_context;
    if (num_seqs <= 0 || total_q <= 0 || num_kv_heads <= 0 || num_heads <= 0 || num_heads % num_kv_heads) return 0;
    const int G = num_heads / num_kv_heads;
    const int64_t want = g_options[PA_OPT_VARLEN_KERNEL];
    if (want == 1 || !pa::varlen_umma_supported(dtype, head_dim, block_size, G)) return 0;
    return pa::varlen_umma_workspace(num_seqs, total_q, G);
}

}  // extern "C"

// k_scales != nullptr: the caches hold E4M3 codes with these scales.
static pa_status varlen_impl(void* out, const void* q, const void* k_cache, const void* v_cache,
                             const float* k_scales, const float* v_scales, const int32_t* block_tables,
                             int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu_seqlens_q,
                             int32_t num_seqs, int32_t total_q, int32_t max_q, int32_t num_heads,
                             int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks, int32_t block_size,
                             int32_t max_context, float scale, int causal, int dtype, void* workspace,
                             size_t workspace_bytes, void* stream) {
    const bool fp8 = k_scales != nullptr;
    pa_status g = check_geometry(num_heads, num_kv_heads, head_dim, num_blocks, block_size, dtype);
    if (g != PA_OK) return g;
    if (num_seqs < 0 || total_q < 0 || max_q < 0 || max_blocks < 0 || max_context < 0)
        return fail(PA_ERR_INVALID_ARG, "sizes must be non-negative");
    if (num_seqs == 0 || total_q == 0) return PA_OK;
    if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !cu_seqlens_q)
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache))
        return fail(PA_ERR_INVALID_ARG, "out, q and the caches must be 16-byte aligned");
    if (fp8 && (!v_scales || !aligned16(k_scales) || !aligned16(v_scales)))
        return fail(PA_ERR_INVALID_ARG, "k_scales and v_scales must be non-null and 16-byte aligned");
    if (!pa::attn_simt_supported(dtype, head_dim)) return fail(PA_ERR_UNSUPPORTED, "head_dim must be in [1, 256]");
    const bool um_ok = pa::varlen_umma_supported(dtype, head_dim, block_size, num_heads / num_kv_heads, fp8);
    const int64_t want = g_options[PA_OPT_VARLEN_KERNEL];
    if (want == 2 && !um_ok)
        return fail(PA_ERR_UNSUPPORTED, fp8 ? "the tcgen05 varlen kernel over a code cache takes bf16/f16 "
                                              "queries, head_dim 128 and block_size 8 or a multiple of 16"
                                            : "the tcgen05 varlen kernel takes bf16/f16, head_dim 64/128/256 and "
                                              "block_size a multiple of 16 (or 8, below head_dim 256)");
    const bool use_um = um_ok && (want == 2 || want == 0);
    cudaStream_t st = as_stream(stream);
    if (check_mode()) {
        pa_status err = check_varlen(block_tables, max_blocks, seq_lens, cu_seqlens_q, num_seqs, total_q, max_q,
                                     num_blocks, block_size, max_context, st);
        if (err != PA_OK) return err;
    }
    pa::AttnArgs a{};
    a.out = out;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.max_blocks = max_blocks;
    a.seq_lens = seq_lens;
    a.cu_seqlens_q = cu_seqlens_q;
    a.num_seqs = num_seqs;
    a.total_q = total_q;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.block_size = block_size;
    a.scale = scale;
    a.causal = causal ? 1 : 0;
    a.dtype = dtype;
    a.max_context = max_context;
    a.kv_fp8 = fp8 ? 1 : 0;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    if (use_um) {
        // optional workspace: the tensor-core kernel then runs its work
        // longest first (a plan kernel sorts it); without one, in request order
        void* ws = nullptr;
        if (workspace && workspace_bytes > 0) {
            const size_t need = pa::varlen_umma_workspace(num_seqs, total_q, num_heads / num_kv_heads);
            if (workspace_bytes < need)
                return fail(PA_ERR_WORKSPACE, "workspace holds " + std::to_string(workspace_bytes) + " bytes, " +
                                                  std::to_string(need) + " needed");
            if (!aligned16(workspace)) return fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
            ws = workspace;
        }
        std::string err;
        cudaError_t e = pa::launch_varlen_umma(a, num_blocks, ws, &err, st);
        if (e != cudaSuccess)
            return err.empty() ? cuda_fail(e, "pa_varlen launch") : fail(PA_ERR_CUDA, "pa_varlen: " + err);
        return PA_OK;
    }
    cudaError_t e = pa::launch_attn_simt(a, st);
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "pa_varlen launch");
}

extern "C" {

pa_status pa_varlen(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                    int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu_seqlens_q, int32_t num_seqs,
                    int32_t total_q, int32_t max_q, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                    int32_t num_blocks, int32_t block_size, int32_t max_context, float scale, int causal, int dtype,
                    void* workspace, size_t workspace_bytes, void* stream) {
    return varlen_impl(out, q, k_cache, v_cache, nullptr, nullptr, block_tables, max_blocks, seq_lens, cu_seqlens_q,
                       num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim, num_blocks, block_size,
                       max_context, scale, causal, dtype, workspace, workspace_bytes, stream);
}

size_t pa_varlen_fp8_workspace_size(int32_t num_seqs, int32_t total_q, int32_t max_q, int32_t num_heads,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                    int32_t max_context, int dtype) {
    (void)max_q, (void)max_context;
    if (num_seqs <= 0 || total_q <= 0 || num_kv_heads <= 0 || num_heads <= 0 || num_heads % num_kv_heads) return 0;
    const int G = num_heads / num_kv_heads;
    if (g_options[PA_OPT_VARLEN_KERNEL] == 1 || !pa::varlen_umma_supported(dtype, head_dim, block_size, G, true))
        return 0;
    return pa::varlen_umma_workspace(num_seqs, total_q, G);
}

pa_status pa_varlen_fp8(void* out, const void* q, const void* k_codes, const void* v_codes, const float* k_scales,
                        const float* v_scales, const int32_t* block_tables, int32_t max_blocks,
                        const int32_t* seq_lens, const int32_t* cu_seqlens_q, int32_t num_seqs, int32_t total_q,
                        int32_t max_q, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks,
                        int32_t block_size, int32_t max_context, float scale, int causal, int dtype, void* workspace,
                        size_t workspace_bytes, void* stream) {
    if (num_seqs > 0 && total_q > 0 && (!k_scales || !v_scales)) return fail(PA_ERR_INVALID_ARG, "null pointer");
    return varlen_impl(out, q, k_codes, v_codes, k_scales, v_scales, block_tables, max_blocks, seq_lens,
                       cu_seqlens_q, num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim, num_blocks,
                       block_size, max_context, scale, causal, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"

// ------------------------------------------------------------------ rotary write

static pa_status rope_impl(void* q_out, const void* q, const void* k, const void* v, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, const int64_t* positions, int32_t num_axes,
                           const double* inv_freq, const int32_t* pair_axis, int32_t rot_dim, int interleaved,
                           const int64_t* slot_mapping, int64_t n, void* k_cache, void* v_cache, float* k_scales,
                           float* v_scales, bool fp8, int32_t num_blocks, int32_t block_size, int32_t num_heads,
                           int32_t num_kv_heads, int32_t head_dim, int dtype, void* stream) {
    if (num_heads < 0) return fail(PA_ERR_INVALID_ARG, "num_heads must be non-negative");
    pa_status g = check_geometry(num_heads ? num_heads : num_kv_heads, num_kv_heads, head_dim, num_blocks, block_size,
                                 dtype);
    if (g != PA_OK) return g;
    if (head_dim > 256) return fail(PA_ERR_UNSUPPORTED, "head_dim must be at most 256");
    if (n < 0) return fail(PA_ERR_INVALID_ARG, "n must be non-negative");
    if (n > INT32_MAX) return fail(PA_ERR_UNSUPPORTED, "n must fit in int32");
    if (num_axes < 1) return fail(PA_ERR_INVALID_ARG, "num_axes must be positive");
    if (rot_dim < 2 || rot_dim % 2 || rot_dim > head_dim)
        return fail(PA_ERR_INVALID_ARG, "rot_dim must be even and in [2, head_dim]");
    if (((int64_t)num_heads + 2 * (int64_t)num_kv_heads) * head_dim > INT32_MAX)
        return fail(PA_ERR_UNSUPPORTED, "a token's q, k and v must be at most 2^31 - 1 elements");
    if (n == 0) return PA_OK;
    if ((num_heads && (!q_out || !q)) || !k || !v || !positions || !inv_freq || !slot_mapping || !k_cache || !v_cache ||
        (fp8 && (!k_scales || !v_scales)))
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    const int64_t krow = (int64_t)num_kv_heads * head_dim;
    if ((num_heads && q_stride < (int64_t)num_heads * head_dim) || k_stride < krow || v_stride < krow)
        return fail(PA_ERR_INVALID_ARG, "strides may not be smaller than a token's row");
    if (num_heads && q_out == q && q_stride != (int64_t)num_heads * head_dim)
        return fail(PA_ERR_INVALID_ARG, "q_out may be q only when q is contiguous");
    if (!aligned16(k_cache) || !aligned16(v_cache))
        return fail(PA_ERR_INVALID_ARG, "the pools must be 16-byte aligned");
    cudaStream_t st = as_stream(stream);
    if (check_mode()) {
        pa_status err = check_slots(slot_mapping, n, num_blocks, block_size, st);
        if (err != PA_OK) return err;
        std::vector<int32_t> ax;
        if (pair_axis) {
            if (!to_host(ax, pair_axis, rot_dim / 2, st, &err)) return err;
            for (int i = 0; i < rot_dim / 2; ++i)
                if (ax[i] < 0 || ax[i] >= num_axes)
                    return fail(PA_ERR_INDEX, "pair " + std::to_string(i) + ": axis outside [0, num_axes)");
        }
    }
    pa::RopeArgs a{};
    a.q_out = num_heads ? q_out : nullptr;
    a.q = num_heads ? q : nullptr;
    a.k = k;
    a.v = v;
    a.q_stride = num_heads ? q_stride : 0;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.positions = positions;
    a.num_axes = num_axes;
    a.inv_freq = inv_freq;
    a.pair_axis = pair_axis;
    a.rot_dim = rot_dim;
    a.interleaved = interleaved ? 1 : 0;
    a.slots = slot_mapping;
    a.n = n;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.block_size = block_size;
    cudaError_t e = pa::launch_rope_write(a, dtype, fp8, st);
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "pa_rope_write_kv launch");
}

// ------------------------------------------------------------------ attention weights

// Sizes and pointers the weight entry points share; `a` gets everything but
// the stats buffer.
static pa_status weights_args(pa::WeightArgs& a, float* weights, int64_t weights_stride, const void* q,
                              const void* k_cache, const float* k_scales, const int32_t* block_tables,
                              int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu, int32_t num_seqs,
                              int32_t total_q, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                              int32_t block_size, int32_t max_context, int32_t window, float scale, int causal,
                              int dtype) {
    if (weights_stride < max_context)
        return fail(PA_ERR_INVALID_ARG, "weights_stride may not be smaller than max_context");
    a.weights = weights;
    a.weights_stride = weights_stride;
    a.q = q;
    a.k_cache = k_cache;
    a.k_scales = k_scales;
    a.block_tables = block_tables;
    a.max_blocks = max_blocks;
    a.seq_lens = seq_lens;
    a.cu = cu;
    a.num_seqs = num_seqs;
    a.total_q = total_q;
    a.num_heads = num_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.block_size = block_size;
    a.max_context = max_context;
    a.window = window;
    a.causal = causal ? 1 : 0;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.dtype = dtype;
    a.kv_fp8 = k_scales != nullptr;
    return PA_OK;
}

// Requests s0 .. s0 + count - 1 of a.
static pa::WeightArgs weights_part(const pa::WeightArgs& a, int32_t s0, int32_t count) {
    pa::WeightArgs c = a;
    c.num_seqs = count;
    c.weights = a.weights + (int64_t)s0 * a.num_kv_heads * a.weights_stride;
    c.block_tables = a.block_tables + (int64_t)s0 * a.max_blocks;
    c.seq_lens = a.seq_lens + s0;
    if (a.cu) {
        c.cu = a.cu + s0;
    } else {  // one query per request
        c.q = static_cast<const uint8_t*>(a.q) + (int64_t)s0 * a.num_heads * a.head_dim * pa::elt_size(a.dtype);
        c.stats = a.stats + (int64_t)s0 * a.num_heads;
        c.total_q = count;
    }
    return c;
}

static size_t align256(size_t b) { return (b + 255) / 256 * 256; }

// Workspace of the weighted decode.  Tensor-core path: the split records,
// the row statistics of units worked whole, the scores; CUDA-core path: the
// row statistics.
struct DecodeWeightsSpace {
    bool tc = false;
    int seqs = 0;  // sequences per launch (tensor-core path)
    int grid = 0;
    size_t records = 0, stats = 0, scores = 0;
    size_t total() const { return records + stats + scores; }
};
static DecodeWeightsSpace decode_weights_space(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                               int32_t head_dim, int32_t block_size, int32_t max_context, int dtype,
                                               bool fp8, pa_status* sel) {
    DecodeWeightsSpace w;
    const int G = num_heads / num_kv_heads;
    w.tc = use_decode_tc(dtype, head_dim, block_size, G, fp8, sel);
    w.stats = align256((size_t)num_seqs * num_heads * sizeof(float2));
    if (w.tc) {
        const size_t scores = pa::decode_weights_scores(num_heads, max_context);
        w.seqs = pa::seqs_per_launch(num_seqs, (double)scores, pa::kDecodeMaxSeqsPerLaunch);
        w.scores = w.seqs * scores;
        w.grid = pa::decode_weights_grid(w.seqs, num_kv_heads, head_dim, block_size, max_context, dtype, G,
                                         g_options[PA_OPT_DECODE_CTAS], fp8);
        w.records = align256(pa::decode_tc_workspace(num_seqs, num_kv_heads, G, head_dim, w.grid, fp8));
    }
    return w;
}

static size_t decode_weights_workspace(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                       int32_t block_size, int32_t max_context, int dtype, bool fp8) {
    if (num_seqs <= 0 || num_kv_heads <= 0 || num_heads <= 0 || num_heads % num_kv_heads || max_context < 0)
        return 0;
    pa_status sel;
    return decode_weights_space(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype, fp8, &sel)
        .total();
}

static pa_status decode_weights_impl(void* out, float* weights, int64_t weights_stride, const void* q,
                                     const void* k_cache, const void* v_cache, const float* k_scales,
                                     const float* v_scales, const int32_t* block_tables, int32_t max_blocks,
                                     const int32_t* context_lens, int32_t num_seqs, int32_t num_heads,
                                     int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks, int32_t block_size,
                                     int32_t max_context, float scale, int dtype, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    const bool fp8 = k_scales != nullptr;
    pa::AttnArgs a{};
    pa_status g = decode_args(a, out, q, nullptr, nullptr, k_cache, v_cache, k_scales, v_scales, block_tables,
                              max_blocks, context_lens, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks,
                              block_size, max_context, scale, dtype, as_stream(stream));
    if (g != PA_OK || num_seqs == 0) return g;
    if (!weights) return fail(PA_ERR_INVALID_ARG, "null pointer");
    pa::WeightArgs wa{};
    g = weights_args(wa, weights, weights_stride, q, k_cache, k_scales, block_tables, max_blocks, context_lens,
                     nullptr, num_seqs, num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, 0, scale,
                     1, dtype);
    if (g != PA_OK) return g;
    const DecodeWeightsSpace sp =
        decode_weights_space(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype, fp8, &g);
    if (g != PA_OK) return g;
    if (!workspace || workspace_bytes < sp.total())
        return fail(PA_ERR_WORKSPACE, "workspace holds " + std::to_string(workspace_bytes) + " bytes, " +
                                          std::to_string(sp.total()) + " needed");
    if (!aligned16(workspace)) return fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    cudaStream_t st = as_stream(stream);
    if (!sp.tc) {
        cudaError_t e = pa::launch_attn_simt(a, st);
        if (e != cudaSuccess) return cuda_fail(e, "pa_decode_weights launch");
        wa.stats = reinterpret_cast<float2*>(ws);
        for (int32_t s0 = 0; s0 < num_seqs; s0 += pa::kWeightMaxSeqsPerLaunch) {
            e = pa::launch_weights_simt(weights_part(wa, s0, std::min(num_seqs - s0, pa::kWeightMaxSeqsPerLaunch)), st);
            if (e != cudaSuccess) return cuda_fail(e, "pa_decode_weights launch");
        }
        return PA_OK;
    }
    for (int32_t s0 = 0; s0 < num_seqs; s0 += sp.seqs) {
        const int32_t cnt = std::min(num_seqs - s0, sp.seqs);
        pa::AttnArgs c = decode_part(a, s0, cnt);
        pa::DecodeWeights w;
        w.weights = weights + (int64_t)s0 * num_kv_heads * weights_stride;
        w.stride = weights_stride;
        w.row_stats = reinterpret_cast<float2*>(ws + sp.records);
        w.scores = reinterpret_cast<float*>(ws + sp.records + sp.stats);
        std::string err;
        cudaError_t e = pa::launch_decode_weights(c, num_blocks, sp.grid, ws, w, &err, st);
        if (e != cudaSuccess)
            return err.empty() ? cuda_fail(e, "pa_decode_weights launch") : fail(PA_ERR_CUDA, "pa_decode_weights: " + err);
    }
    return PA_OK;
}

// The prompt form's path (PA_OPT_VARLEN_KERNEL pins it), how its work is cut,
// and its workspace.
struct PromptWeightsPlan {
    static constexpr size_t kCounters = 256;  // ahead of the rest (tensor-core path)
    bool tc = false;
    pa::WeightPlan cut;
    size_t bytes() const { return (tc ? kCounters : 0) + cut.dense_bytes + cut.scale_bytes + cut.stats_bytes + cut.tile_stats_bytes +
               cut.partial_bytes; }
};
static PromptWeightsPlan prompt_weights_plan(int32_t num_seqs, int32_t total_q, int32_t max_q, int32_t num_heads,
                                             int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                             int32_t max_context, int32_t window, int dtype, bool fp8) {
    PromptWeightsPlan p;
    if (num_seqs <= 0 || total_q <= 0 || max_q <= 0 || max_context <= 0 || block_size <= 0 || window < 0 ||
        num_kv_heads <= 0 || num_heads <= 0 || num_heads % num_kv_heads)
        return p;
    const int G = num_heads / num_kv_heads;
    p.tc = g_options[PA_OPT_VARLEN_KERNEL] != 1 && pa::weights_umma_supported(dtype, head_dim, G);
    if (p.tc) {
        p.cut = pa::weights_umma_plan(num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim, block_size,
                                      max_context, window, fp8);
    } else {
        p.cut.seqs = std::min(num_seqs, pa::kWeightMaxSeqsPerLaunch);
        p.cut.stats_bytes =
            (size_t)pa::weight_stat_rows(p.cut.seqs, total_q, window).rows * num_heads * sizeof(float2);
    }
    return p;
}

static pa_status prompt_weights_impl(float* weights, int64_t weights_stride, const void* q, const void* k_cache,
                                     const float* k_scales, const int32_t* block_tables, int32_t max_blocks,
                                     const int32_t* seq_lens, const int32_t* cu_seqlens_q, int32_t num_seqs,
                                     int32_t total_q, int32_t max_q, int32_t num_heads, int32_t num_kv_heads,
                                     int32_t head_dim, int32_t num_blocks, int32_t block_size, int32_t max_context,
                                     int32_t window, float scale, int causal, int dtype, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    pa_status g = check_geometry(num_heads, num_kv_heads, head_dim, num_blocks, block_size, dtype);
    if (g != PA_OK) return g;
    if (num_seqs < 0 || total_q < 0 || max_q < 0 || max_blocks < 0 || max_context < 0 || window < 0)
        return fail(PA_ERR_INVALID_ARG, "sizes must be non-negative");
    if (num_seqs == 0 || total_q == 0 || max_q == 0 || max_context == 0) return PA_OK;
    if (!weights || !q || !k_cache || !block_tables || !seq_lens || !cu_seqlens_q)
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(q) || !aligned16(k_cache)) return fail(PA_ERR_INVALID_ARG, "q and the cache must be 16-byte aligned");
    if (k_scales && !aligned16(k_scales)) return fail(PA_ERR_INVALID_ARG, "k_scales must be 16-byte aligned");
    if (!pa::attn_simt_supported(dtype, head_dim)) return fail(PA_ERR_UNSUPPORTED, "head_dim must be in [1, 256]");
    pa::WeightArgs a{};
    g = weights_args(a, weights, weights_stride, q, k_cache, k_scales, block_tables, max_blocks, seq_lens,
                     cu_seqlens_q, num_seqs, total_q, num_heads, num_kv_heads, head_dim, block_size, max_context,
                     window, scale, causal, dtype);
    if (g != PA_OK) return g;
    const PromptWeightsPlan plan = prompt_weights_plan(num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim,
                                                       block_size, max_context, window, dtype, k_scales != nullptr);
    if (g_options[PA_OPT_VARLEN_KERNEL] == 2 && !plan.tc)
        return fail(PA_ERR_UNSUPPORTED, "the tcgen05 weight kernels take bf16/f16 queries, head_dim 64/128/256 and at "
                                        "most 128 query heads per KV head");
    if (plan.tc && plan.cut.dense_stride < 0)
        return fail(PA_ERR_UNSUPPORTED, "max_context must be at most 2^29 where the keys are laid out densely");
    if (!workspace || workspace_bytes < plan.bytes())
        return fail(PA_ERR_WORKSPACE, "workspace holds " + std::to_string(workspace_bytes) + " bytes, " +
                                          std::to_string(plan.bytes()) + " needed");
    if (!aligned16(workspace)) return fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    cudaStream_t st = as_stream(stream);
    if (check_mode()) {
        pa_status err = check_varlen(block_tables, max_blocks, seq_lens, cu_seqlens_q, num_seqs, total_q, max_q,
                                     num_blocks, block_size, max_context, st);
        if (err != PA_OK) return err;
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.next_item = reinterpret_cast<uint32_t*>(ws);
    if (plan.tc) ws += PromptWeightsPlan::kCounters;
    a.dense_stride = plan.cut.dense_stride;
    a.dense_keys = ws;
    ws += plan.cut.dense_bytes;
    a.key_scales = reinterpret_cast<float*>(ws);
    ws += plan.cut.scale_bytes;
    const pa::WeightStatRows sr = pa::weight_stat_rows(plan.cut.seqs, total_q, window);
    a.stat_rows = sr.rows;
    a.stat_pitch = sr.pitch;
    a.stats = reinterpret_cast<float2*>(ws);
    a.tile_stats = reinterpret_cast<float*>(ws + plan.cut.stats_bytes);
    a.stat_tiles = plan.cut.stat_tiles;
    a.partial = reinterpret_cast<float*>(ws + plan.cut.stats_bytes + plan.cut.tile_stats_bytes);
    a.key_splits = plan.cut.key_splits;
    a.row_splits = plan.cut.row_splits;
    a.few_rows = plan.cut.few_rows ? 1 : 0;
    for (int32_t s0 = 0; s0 < num_seqs; s0 += plan.cut.seqs) {
        const pa::WeightArgs c = weights_part(a, s0, std::min(num_seqs - s0, plan.cut.seqs));
        std::string err;
        cudaError_t e = plan.tc ? pa::launch_weights_umma(c, num_blocks, &err, st)
                                : pa::launch_weights_simt(c, st);
        if (e != cudaSuccess)
            return err.empty() ? cuda_fail(e, "pa_prompt_weights launch") : fail(PA_ERR_CUDA, "pa_prompt_weights: " + err);
    }
    return PA_OK;
}

extern "C" {

pa_status pa_rope_write_kv(void* q_out, const void* q, const void* k, const void* v, int64_t q_stride,
                           int64_t k_stride, int64_t v_stride, const int64_t* positions, int32_t num_axes,
                           const double* inv_freq, const int32_t* pair_axis, int32_t rot_dim, int interleaved,
                           const int64_t* slot_mapping, int64_t n, void* k_cache, void* v_cache, int32_t num_blocks,
                           int32_t block_size, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int dtype,
                           void* stream) {
    return rope_impl(q_out, q, k, v, q_stride, k_stride, v_stride, positions, num_axes, inv_freq, pair_axis, rot_dim,
                     interleaved, slot_mapping, n, k_cache, v_cache, nullptr, nullptr, false, num_blocks, block_size,
                     num_heads, num_kv_heads, head_dim, dtype, stream);
}

pa_status pa_rope_write_kv_fp8(void* q_out, const void* q, const void* k, const void* v, int64_t q_stride,
                               int64_t k_stride, int64_t v_stride, const int64_t* positions, int32_t num_axes,
                               const double* inv_freq, const int32_t* pair_axis, int32_t rot_dim, int interleaved,
                               const int64_t* slot_mapping, int64_t n, void* k_codes, void* v_codes, float* k_scales,
                               float* v_scales, int32_t num_blocks, int32_t block_size, int32_t num_heads,
                               int32_t num_kv_heads, int32_t head_dim, int dtype, void* stream) {
    return rope_impl(q_out, q, k, v, q_stride, k_stride, v_stride, positions, num_axes, inv_freq, pair_axis, rot_dim,
                     interleaved, slot_mapping, n, k_codes, v_codes, k_scales, v_scales, true, num_blocks, block_size,
                     num_heads, num_kv_heads, head_dim, dtype, stream);
}

size_t pa_decode_weights_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                        int32_t block_size, int32_t max_context, int dtype) {
    return decode_weights_workspace(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype, false);
}

pa_status pa_decode_weights(void* out, float* weights, int64_t weights_stride, const void* q, const void* k_cache,
                            const void* v_cache, const int32_t* block_tables, int32_t max_blocks,
                            const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                            int32_t head_dim, int32_t num_blocks, int32_t block_size, int32_t max_context,
                            float scale, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    return decode_weights_impl(out, weights, weights_stride, q, k_cache, v_cache, nullptr, nullptr, block_tables,
                               max_blocks, context_lens, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks,
                               block_size, max_context, scale, dtype, workspace, workspace_bytes, stream);
}

size_t pa_decode_weights_fp8_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                            int32_t head_dim, int32_t block_size, int32_t max_context, int dtype) {
    return decode_weights_workspace(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype, true);
}

pa_status pa_decode_weights_fp8(void* out, float* weights, int64_t weights_stride, const void* q, const void* k_codes,
                                const void* v_codes, const float* k_scales, const float* v_scales,
                                const int32_t* block_tables, int32_t max_blocks, const int32_t* context_lens,
                                int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                int32_t num_blocks, int32_t block_size, int32_t max_context, float scale, int dtype,
                                void* workspace, size_t workspace_bytes, void* stream) {
    if (num_seqs > 0 && (!k_scales || !v_scales)) return fail(PA_ERR_INVALID_ARG, "null pointer");
    return decode_weights_impl(out, weights, weights_stride, q, k_codes, v_codes, k_scales, v_scales, block_tables,
                               max_blocks, context_lens, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks,
                               block_size, max_context, scale, dtype, workspace, workspace_bytes, stream);
}

size_t pa_prompt_weights_workspace_size(int32_t num_seqs, int32_t total_q, int32_t max_q, int32_t num_heads,
                                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                        int32_t max_context, int32_t window, int dtype) {
    return prompt_weights_plan(num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim, block_size, max_context,
                               window, dtype, false)
        .bytes();
}

pa_status pa_prompt_weights(float* weights, int64_t weights_stride, const void* q, const void* k_cache,
                            const int32_t* block_tables, int32_t max_blocks, const int32_t* seq_lens,
                            const int32_t* cu_seqlens_q, int32_t num_seqs, int32_t total_q, int32_t max_q,
                            int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t num_blocks,
                            int32_t block_size, int32_t max_context, int32_t window, float scale, int causal,
                            int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    return prompt_weights_impl(weights, weights_stride, q, k_cache, nullptr, block_tables, max_blocks, seq_lens,
                               cu_seqlens_q, num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim, num_blocks,
                               block_size, max_context, window, scale, causal, dtype, workspace, workspace_bytes,
                               stream);
}

size_t pa_prompt_weights_fp8_workspace_size(int32_t num_seqs, int32_t total_q, int32_t max_q, int32_t num_heads,
                                            int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                            int32_t max_context, int32_t window, int dtype) {
    return prompt_weights_plan(num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim, block_size, max_context,
                               window, dtype, true)
        .bytes();
}

pa_status pa_prompt_weights_fp8(float* weights, int64_t weights_stride, const void* q, const void* k_codes,
                                const float* k_scales, const int32_t* block_tables, int32_t max_blocks,
                                const int32_t* seq_lens, const int32_t* cu_seqlens_q, int32_t num_seqs,
                                int32_t total_q, int32_t max_q, int32_t num_heads, int32_t num_kv_heads,
                                int32_t head_dim, int32_t num_blocks, int32_t block_size, int32_t max_context,
                                int32_t window, float scale, int causal, int dtype, void* workspace,
                                size_t workspace_bytes, void* stream) {
    if (num_seqs > 0 && total_q > 0 && !k_scales) return fail(PA_ERR_INVALID_ARG, "null pointer");
    return prompt_weights_impl(weights, weights_stride, q, k_codes, k_scales, block_tables, max_blocks, seq_lens,
                               cu_seqlens_q, num_seqs, total_q, max_q, num_heads, num_kv_heads, head_dim, num_blocks,
                               block_size, max_context, window, scale, causal, dtype, workspace, workspace_bytes,
                               stream);
}

// ------------------------------------------------------------------ eviction

size_t pa_evict_workspace_size(int32_t num_seqs, int32_t num_kv_heads, int32_t max_context, int32_t keep) {
    if (num_seqs <= 0 || num_kv_heads <= 0 || max_context < 0 || keep <= 0) return 0;
    return pa::evict_workspace(num_seqs, num_kv_heads, max_context, keep);
}

pa_status pa_evict(float* weights_out, int32_t* positions_out, int32_t* new_lens, const float* weights,
                   const int32_t* positions, const int32_t* recorded_lens, const int32_t* seen_lens,
                   int64_t weights_stride, void* k_cache, void* v_cache, float* k_scales, float* v_scales,
                   const int32_t* block_tables, int32_t max_blocks, const int32_t* new_block_tables,
                   int32_t new_max_blocks, const int32_t* context_lens, int32_t num_seqs, int32_t num_kv_heads,
                   int32_t head_dim, int32_t num_blocks, int32_t block_size, int32_t max_context, int32_t keep,
                   int32_t num_sink, int32_t num_recent, int dtype, void* workspace, size_t workspace_bytes,
                   void* stream) {
    pa_status g = check_geometry(num_kv_heads, num_kv_heads, head_dim, num_blocks, block_size, dtype, true);
    if (g != PA_OK) return g;
    if (num_seqs < 0 || max_blocks < 0 || new_max_blocks < 0 || max_context < 0)
        return fail(PA_ERR_INVALID_ARG, "sizes must be non-negative");
    if (keep < 1 || num_sink < 0 || num_recent < 0 || (int64_t)num_sink + num_recent > keep)
        return fail(PA_ERR_INVALID_ARG, "keep must be positive and hold num_sink + num_recent tokens");
    if (weights_stride < max_context)
        return fail(PA_ERR_INVALID_ARG, "weights_stride may not be smaller than max_context");
    if (num_seqs == 0) return PA_OK;
    if (!weights_out || !new_lens || !weights || !k_cache || !v_cache || !block_tables || !new_block_tables ||
        !context_lens)
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if ((recorded_lens != nullptr) != (positions != nullptr))
        return fail(PA_ERR_INVALID_ARG, "positions and recorded_lens go together");
    const bool fp8 = dtype == PA_FP8_E4M3;
    if (fp8 != (k_scales != nullptr) || fp8 != (v_scales != nullptr))
        return fail(PA_ERR_INVALID_ARG, "k_scales and v_scales go with PA_FP8_E4M3 pools, and only with them");
    if (new_lens == context_lens || new_lens == recorded_lens || new_lens == seen_lens)
        return fail(PA_ERR_INVALID_ARG, "new_lens must be memory apart from the other arrays");
    if (!aligned16(k_cache) || !aligned16(v_cache))
        return fail(PA_ERR_INVALID_ARG, "the pools must be 16-byte aligned");
    if ((int64_t)num_seqs * num_kv_heads > (1 << 24))
        return fail(PA_ERR_UNSUPPORTED, "num_seqs * num_kv_heads must be at most 2^24");
    if (max_context > pa::kEvictMaxContext) return fail(PA_ERR_UNSUPPORTED, "max_context must be at most 2^19");
    const size_t need = pa::evict_workspace(num_seqs, num_kv_heads, max_context, keep);
    if (workspace_bytes < need || (need && !workspace))
        return fail(PA_ERR_WORKSPACE, "workspace holds " + std::to_string(workspace_bytes) + " bytes, " +
                                          std::to_string(need) + " needed");
    if (!aligned16(workspace)) return fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    cudaStream_t st = as_stream(stream);
    if (check_mode()) {
        pa_status err = check_evict(recorded_lens, seen_lens, block_tables, max_blocks, new_block_tables, new_max_blocks,
                                    context_lens, num_seqs, num_blocks, block_size, max_context, keep, st);
        if (err != PA_OK) return err;
    }
    pa::EvictArgs a{};
    a.weights_out = weights_out;
    a.positions_out = positions_out;
    a.new_lens = new_lens;
    a.weights = weights;
    a.positions = positions;
    a.recorded_lens = recorded_lens;
    a.seen_lens = seen_lens;
    a.stride = weights_stride;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.block_tables = block_tables;
    a.max_blocks = max_blocks;
    a.new_block_tables = new_block_tables;
    a.new_max_blocks = new_max_blocks;
    a.context_lens = context_lens;
    a.num_seqs = num_seqs;
    a.num_kv_heads = num_kv_heads;
    a.block_size = block_size;
    a.max_context = max_context;
    a.keep = keep;
    a.num_sink = num_sink;
    a.num_recent = num_recent;
    a.row_bytes = (int64_t)head_dim * pa::elt_size(dtype);
    cudaError_t e = pa::launch_evict(a, workspace, st);
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "pa_evict launch");
}

}  // extern "C"

// ------------------------------------------------------------------ latent cache

extern "C" pa_status pa_latent_write(void* q_out, int64_t q_out_stride, int64_t q_out_head_stride, const void* q,
                                     int64_t q_stride, int64_t q_head_stride, const void* kv, int64_t kv_stride,
                                     const void* norm_weight, float eps, const int64_t* positions,
                                     const double* inv_freq, int32_t rope_dim, int interleaved,
                                     const int64_t* slot_mapping, int64_t n, void* cache, int32_t num_blocks,
                                     int32_t block_size, int32_t num_heads, int32_t latent_dim, int dtype,
                                     void* stream) {
    if (num_heads < 0 || latent_dim <= 0 || rope_dim < 2 || rope_dim % 2 || rope_dim > 256)
        return fail(PA_ERR_INVALID_ARG, "latent_dim must be positive, rope_dim even and in [2, 256], num_heads >= 0");
    if (latent_dim > 4096 || num_heads > (1 << 20))
        return fail(PA_ERR_UNSUPPORTED, "latent_dim must be at most 4096, num_heads at most 2^20");
    pa_status g = check_geometry(std::max(num_heads, 1), 1, latent_dim + rope_dim, num_blocks, block_size, dtype);
    if (g != PA_OK) return g;
    if (n < 0) return fail(PA_ERR_INVALID_ARG, "n must be non-negative");
    if (n == 0) return PA_OK;
    if (n > (int64_t)INT32_MAX) return fail(PA_ERR_UNSUPPORTED, "n must fit in int32");
    if (!kv || !positions || !inv_freq || !slot_mapping || !cache || (num_heads && (!q || !q_out)))
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    const int elt = pa::elt_size(dtype);
    const uintptr_t addr = reinterpret_cast<uintptr_t>(kv) | reinterpret_cast<uintptr_t>(norm_weight) |
                           (num_heads ? reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q_out) : 0);
    if (addr % (uintptr_t)elt) return fail(PA_ERR_INVALID_ARG, "pointers must be aligned to their type");
    if (!aligned16(cache)) return fail(PA_ERR_INVALID_ARG, "the cache must be 16-byte aligned");
    if (kv_stride < latent_dim + rope_dim)
        return fail(PA_ERR_INVALID_ARG, "kv_stride may not be smaller than a token's row");
    // no element of q_out twice: heads within tokens, or tokens within heads
    const int64_t qt = n > 1 ? q_out_stride : rope_dim, qh = num_heads > 1 ? q_out_head_stride : rope_dim;
    if (num_heads && !(qh >= rope_dim && (n == 1 || qt >= (num_heads - 1) * qh + rope_dim)) &&
        !(qt >= rope_dim && (num_heads == 1 || qh >= (n - 1) * qt + rope_dim)))
        return fail(PA_ERR_INVALID_ARG, "strides of q_out must keep heads and tokens apart");
    if (num_heads && (q_stride < 0 || q_head_stride < 0))
        return fail(PA_ERR_INVALID_ARG, "strides must be non-negative");
    cudaStream_t st = as_stream(stream);
    if (check_mode()) {
        pa_status err = check_slots(slot_mapping, n, num_blocks, block_size, st);
        if (err != PA_OK) return err;
    }
    pa::LatentWriteArgs a{};
    a.q_out = num_heads ? q_out : nullptr;
    a.q = num_heads ? q : nullptr;
    a.kv = kv;
    a.q_out_stride = num_heads && n > 1 ? q_out_stride : 0;
    a.q_out_head_stride = num_heads > 1 ? q_out_head_stride : 0;
    a.q_stride = num_heads && n > 1 ? q_stride : 0;
    a.q_head_stride = num_heads > 1 ? q_head_stride : 0;
    a.kv_stride = n > 1 ? kv_stride : 0;
    a.norm_weight = norm_weight;
    a.eps = eps;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.rope_dim = rope_dim;
    a.interleaved = interleaved ? 1 : 0;
    a.slots = slot_mapping;
    a.n = n;
    a.cache = cache;
    a.num_heads = num_heads;
    a.latent_dim = latent_dim;
    cudaError_t e = pa::launch_latent_write(a, dtype, st);
    return e == cudaSuccess ? PA_OK : cuda_fail(e, "pa_latent_write launch");
}

// The kernel of a latent attention call (`want`: the pinned one, 0 automatic).
static bool use_latent_umma(int64_t want, int dtype, int32_t latent_dim, int32_t rope_dim, int32_t block_size,
                            pa_status* st) {
    const bool ok = pa::latent_umma_supported(dtype, latent_dim, rope_dim, block_size);
    *st = PA_OK;
    if (want == 2 && !ok)
        *st = fail(PA_ERR_UNSUPPORTED, "the tensor-core latent kernel takes bf16/f16, latent_dim 512 and rope_dim 64");
    return ok && want != 1;
}

static size_t latent_workspace(int64_t want, bool varlen, int32_t num_seqs, int64_t total_q, int32_t num_heads,
                               int32_t latent_dim, int32_t rope_dim, int32_t block_size, int32_t max_context,
                               int dtype) {
    if (num_seqs <= 0 || total_q <= 0 || num_heads <= 0 || latent_dim <= 0) return 0;
    if (want != 1 && pa::latent_umma_supported(dtype, latent_dim, rope_dim, block_size))
        return pa::latent_umma_workspace(varlen ? total_q * num_heads : num_heads);  // rows of a request at most
    return pa::latent_simt_workspace(total_q, num_heads, latent_dim, max_context);
}

// cu == nullptr: one query per sequence.
static pa_status latent_impl(void* out, const void* q, const void* cache, const int32_t* block_tables,
                             int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu, int32_t num_seqs,
                             int32_t total_q, int32_t max_q, int32_t num_heads, int32_t latent_dim, int32_t rope_dim,
                             int32_t num_blocks, int32_t block_size, int32_t max_context, float scale, int causal,
                             int dtype, bool varlen, void* workspace, size_t workspace_bytes, void* stream) {
    const char* name = varlen ? "pa_latent_varlen" : "pa_latent_decode";
    if (latent_dim <= 0 || rope_dim < 0) return fail(PA_ERR_INVALID_ARG, "latent_dim must be positive, rope_dim >= 0");
    if ((int64_t)latent_dim + rope_dim > INT32_MAX) return fail(PA_ERR_UNSUPPORTED, "rows of at most 576 elements");
    pa_status g = check_geometry(num_heads, 1, latent_dim + rope_dim, num_blocks, block_size, dtype);
    if (g != PA_OK) return g;
    if (num_seqs < 0 || total_q < 0 || max_q < 0 || max_blocks < 0 || max_context < 0)
        return fail(PA_ERR_INVALID_ARG, "sizes must be non-negative");
    if (num_seqs == 0 || total_q == 0) return PA_OK;
    if (!out || !q || !cache || !block_tables || !seq_lens || (varlen && !cu))
        return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(out) || !aligned16(q) || !aligned16(cache))
        return fail(PA_ERR_INVALID_ARG, "out, q and the cache must be 16-byte aligned");
    if (!pa::latent_simt_supported(dtype, latent_dim + rope_dim))
        return fail(PA_ERR_UNSUPPORTED, "latent_dim + rope_dim must be at most 576");
    pa_status sel;
    const bool tc = use_latent_umma(g_options[varlen ? PA_OPT_VARLEN_KERNEL : PA_OPT_DECODE_KERNEL], dtype, latent_dim,
                                    rope_dim, block_size, &sel);
    if (sel != PA_OK) return sel;
    const int64_t rows = (int64_t)total_q * num_heads;
    if (!tc && num_heads > 65535) return fail(PA_ERR_UNSUPPORTED, "too many heads");
    if (tc && (rows > INT32_MAX - 128 ||
               (rows / 128 + num_seqs) * (((int64_t)max_context + 127) / 128 + 8) > INT32_MAX))
        return fail(PA_ERR_UNSUPPORTED, "too many query rows for one call");
    cudaStream_t st = as_stream(stream);
    if (check_mode()) {
        pa_status err = PA_OK;
        if (varlen) {
            err = check_varlen(block_tables, max_blocks, seq_lens, cu, num_seqs, total_q, max_q, num_blocks,
                               block_size, max_context, st);
        } else {
            std::vector<int32_t> lens;
            if (!to_host(lens, seq_lens, num_seqs, st, &err)) return err;
            err = check_tables(block_tables, num_seqs, max_blocks, lens, num_blocks, block_size, max_context, st);
        }
        if (err != PA_OK) return err;
    }
    pa::LatentArgs a{};
    a.out = out;
    a.q = q;
    a.cache = cache;
    a.block_tables = block_tables;
    a.max_blocks = max_blocks;
    a.seq_lens = seq_lens;
    a.cu = cu;
    a.num_seqs = num_seqs;
    a.total_q = total_q;
    a.num_heads = num_heads;
    a.latent_dim = latent_dim;
    a.rope_dim = rope_dim;
    a.block_size = block_size;
    a.max_context = max_context;
    a.scale = scale;
    a.causal = causal ? 1 : 0;
    a.dtype = dtype;
    std::string err;
    cudaError_t e;
    const size_t need = latent_workspace(g_options[varlen ? PA_OPT_VARLEN_KERNEL : PA_OPT_DECODE_KERNEL], varlen,
                                         num_seqs, total_q, num_heads, latent_dim, rope_dim, block_size, max_context,
                                         dtype);
    if (need && (workspace_bytes < need || !workspace))
        return fail(PA_ERR_WORKSPACE, "workspace holds " + std::to_string(workspace ? workspace_bytes : 0) +
                                          " bytes, " + std::to_string(need) + " needed");
    if (!aligned16(workspace)) return fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    e = tc ? pa::launch_latent_umma(a, num_blocks, workspace, &err, st) : pa::launch_latent_simt(a, workspace, st);
    if (e != cudaSuccess)
        return err.empty() ? cuda_fail(e, name) : fail(PA_ERR_CUDA, std::string(name) + ": " + err);
    return PA_OK;
}

extern "C" {

size_t pa_latent_decode_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t latent_dim, int32_t rope_dim,
                                       int32_t block_size, int32_t max_context, int dtype) {
    return latent_workspace(g_options[PA_OPT_DECODE_KERNEL], false, num_seqs, num_seqs, num_heads, latent_dim, rope_dim,
                            block_size, max_context, dtype);
}

pa_status pa_latent_decode(void* out, const void* q, const void* cache, const int32_t* block_tables,
                           int32_t max_blocks, const int32_t* context_lens, int32_t num_seqs, int32_t num_heads,
                           int32_t latent_dim, int32_t rope_dim, int32_t num_blocks, int32_t block_size,
                           int32_t max_context, float scale, int dtype, void* workspace, size_t workspace_bytes,
                           void* stream) {
    return latent_impl(out, q, cache, block_tables, max_blocks, context_lens, nullptr, num_seqs, num_seqs, 1,
                       num_heads, latent_dim, rope_dim, num_blocks, block_size, max_context, scale, 1, dtype, false,
                       workspace, workspace_bytes, stream);
}

size_t pa_latent_varlen_workspace_size(int32_t num_seqs, int32_t total_q, int32_t max_q, int32_t num_heads,
                                       int32_t latent_dim, int32_t rope_dim, int32_t block_size, int32_t max_context,
                                       int dtype) {
    (void)max_q;
    return latent_workspace(g_options[PA_OPT_VARLEN_KERNEL], true, num_seqs, total_q, num_heads, latent_dim, rope_dim,
                            block_size, max_context, dtype);
}

pa_status pa_latent_varlen(void* out, const void* q, const void* cache, const int32_t* block_tables,
                           int32_t max_blocks, const int32_t* seq_lens, const int32_t* cu_seqlens_q, int32_t num_seqs,
                           int32_t total_q, int32_t max_q, int32_t num_heads, int32_t latent_dim, int32_t rope_dim,
                           int32_t num_blocks, int32_t block_size, int32_t max_context, float scale, int causal,
                           int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    return latent_impl(out, q, cache, block_tables, max_blocks, seq_lens, cu_seqlens_q, num_seqs, total_q, max_q,
                       num_heads, latent_dim, rope_dim, num_blocks, block_size, max_context, scale, causal, dtype,
                       true, workspace, workspace_bytes, stream);
}

}  // extern "C"

// ------------------------------------------------------------------ shared prefixes

// Whether a call works its prefixes apart.  That takes three launches more, 12
// to 20 us, so there has to be something to save: the members beyond one a
// group would read their prefixes again, which the host can bound by
// max_context.  Measured on 55 batches (1-60 groups of 2-64 members, prefixes
// of 144-8,192 tokens, five head layouts): with 13-70 MB to save 25-47 us
// against 17-46 us by the plain decode, 200-290 MB 34-84 against 35-90, from
// 345 MB on 34-153 against 45-567 (one exception: 60 x 4 members behind 288
// tokens with tails of 256, 78 against 71).  PA_OPT_DECODE_KERNEL = 2 always
// works them apart.
static constexpr double kSharedMinBytes = 192e6;
static bool shares_prefixes(int32_t num_seqs, int32_t num_groups, int32_t num_heads, int32_t num_kv_heads,
                            int32_t head_dim, int32_t block_size, int32_t max_context, int dtype) {
    const int G = num_heads / num_kv_heads;
    const int64_t want = g_options[PA_OPT_DECODE_KERNEL];
    if (want == 1 || !pa::decode_shared_supported(dtype, head_dim, block_size, G, num_seqs, num_groups, max_context))
        return false;
    const double saved = ((double)num_seqs - num_groups) * max_context * num_kv_heads * head_dim * 4;
    if (want != 2 && saved < kSharedMinBytes) return false;
    // the units' costs are counted in int32
    const double units = ((double)num_seqs * G / 128 + num_groups) * 2 * num_kv_heads;
    return units * (max_context / 128 + 4.0) < 2e9;
}
static size_t shared_workspace(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                               int32_t block_size, int32_t max_context, int dtype) {
    const int grid = pa::decode_shared_grid(num_seqs, num_kv_heads, head_dim, max_context, dtype,
                                            num_heads / num_kv_heads, g_options[PA_OPT_DECODE_CTAS]);
    return pa::decode_shared_workspace(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, grid);
}

// Check-mode validation of the groups: their ranges, whole blocks, within the
// members' contexts, one run of blocks for all members.
static pa_status check_groups(const int32_t* group_starts, const int32_t* prefix_lens, int32_t num_groups,
                              const int32_t* block_tables, int32_t max_blocks, const int32_t* context_lens,
                              int32_t num_seqs, int32_t block_size, cudaStream_t st) {
    pa_status err = PA_OK;
    std::vector<int32_t> starts, prefix, lens, bt;
    if (!to_host(starts, group_starts, (int64_t)num_groups + 1, st, &err) ||
        !to_host(prefix, prefix_lens, num_groups, st, &err) || !to_host(lens, context_lens, num_seqs, st, &err) ||
        !to_host(bt, block_tables, (int64_t)num_seqs * max_blocks, st, &err))
        return err;
    if (starts[0] < 0 || starts[num_groups] > num_seqs)
        return fail(PA_ERR_INDEX, "group_starts must lie in [0, num_seqs]");
    for (int32_t g = 0; g < num_groups; ++g)  // (all of them first: what follows indexes by them)
        if (starts[g + 1] < starts[g]) return fail(PA_ERR_INDEX, "group_starts must be non-decreasing");
    for (int32_t g = 0; g < num_groups; ++g) {
        const std::string who = "group " + std::to_string(g);
        if (prefix[g] < 0 || prefix[g] % block_size)
            return fail(PA_ERR_INDEX, who + ": prefix_lens must be a non-negative multiple of block_size");
        for (int32_t s = starts[g]; s < starts[g + 1]; ++s) {
            if (prefix[g] > lens[s])
                return fail(PA_ERR_INDEX, who + ": the prefix is longer than sequence " + std::to_string(s));
            for (int32_t b = 0; b < prefix[g] / block_size; ++b)
                if (bt[(size_t)s * max_blocks + b] != bt[(size_t)starts[g] * max_blocks + b])
                    return fail(PA_ERR_INDEX, who + ": sequence " + std::to_string(s) + " does not share logical block " +
                                                  std::to_string(b));
        }
    }
    return PA_OK;
}

extern "C" {

size_t pa_decode_shared_workspace_size(int32_t num_seqs, int32_t num_groups, int32_t num_heads, int32_t num_kv_heads,
                                       int32_t head_dim, int32_t block_size, int32_t max_context, int dtype) {
    const size_t plain =
        decode_workspace(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype, false);
    if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads || block_size <= 0 ||
        !shares_prefixes(num_seqs, num_groups, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype))
        return plain;
    return std::max(plain, shared_workspace(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype));
}

pa_status pa_decode_shared(void* out, const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* block_tables, int32_t max_blocks, const int32_t* context_lens,
                           const int32_t* group_starts, const int32_t* prefix_lens, int32_t num_groups,
                           int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                           int32_t num_blocks, int32_t block_size, int32_t max_context, float scale, int dtype,
                           void* workspace, size_t workspace_bytes, void* stream) {
    if (num_groups < 0) return fail(PA_ERR_INVALID_ARG, "num_groups must be non-negative");
    if (num_groups > 0 && (!group_starts || !prefix_lens)) return fail(PA_ERR_INVALID_ARG, "null pointer");
    if (check_mode() && num_groups > 0 && num_seqs > 0 && block_size > 0 && block_tables && context_lens &&
        max_blocks >= 0) {
        pa_status err = (pa_status)pa::check_decode_indices(block_tables, max_blocks, context_lens, num_seqs,
                                                            num_blocks, block_size, max_context, as_stream(stream));
        if (err == PA_OK)
            err = check_groups(group_starts, prefix_lens, num_groups, block_tables, max_blocks, context_lens, num_seqs,
                               block_size, as_stream(stream));
        if (err != PA_OK) return err;
    }
    if (num_heads > 0 && num_kv_heads > 0 && block_size > 0 && num_seqs > 0 &&
        shares_prefixes(num_seqs, num_groups, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype)) {
        pa::AttnArgs a{};
        cudaStream_t st = as_stream(stream);
        pa_status g = decode_args(a, out, q, nullptr, nullptr, k_cache, v_cache, nullptr, nullptr, block_tables,
                                  max_blocks, context_lens, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks,
                                  block_size, max_context, scale, dtype, st);
        if (g != PA_OK) return g;
        const size_t need = shared_workspace(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context, dtype);
        if (workspace_bytes < need || !workspace)
            return fail(PA_ERR_WORKSPACE, "workspace holds " + std::to_string(workspace ? workspace_bytes : 0) +
                                              " bytes, " + std::to_string(need) + " needed");
        if (!aligned16(workspace)) return fail(PA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
        const int grid = pa::decode_shared_grid(num_seqs, num_kv_heads, head_dim, max_context, dtype,
                                                num_heads / num_kv_heads, g_options[PA_OPT_DECODE_CTAS]);
        std::string err;
        cudaError_t e =
            pa::launch_decode_shared(a, group_starts, prefix_lens, num_groups, num_blocks, grid, workspace, &err, st);
        if (e != cudaSuccess)
            return err.empty() ? cuda_fail(e, "pa_decode_shared launch") : fail(PA_ERR_CUDA, "pa_decode_shared: " + err);
        return PA_OK;
    }
    return decode_impl(out, q, nullptr, nullptr, k_cache, v_cache, nullptr, nullptr, block_tables, max_blocks,
                       context_lens, num_seqs, num_heads, num_kv_heads, head_dim, num_blocks, block_size, max_context,
                       scale, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
