// Internal interface between the key-value cache's host layer (kv_api.cu) and its kernels (kv_attention.cu,
// kv_cache.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace mbd {

// How a cache stores an element: bf16, E4M3 under one scale for all of k (of v), E4M3 under a scale for each token and
// head, or E2M1 under an E4M3 scale for each 16 elements and one scale for all of k (of v).
enum KvStore : int { kKvBf16 = 0, kKvFp8Static = 1, kKvFp8Dynamic = 2, kKvNvfp4 = 3 };

// Bytes of a row, the scales of its blocks apart.
constexpr int kv_row_bytes(int head_dim, int store) {
    return store == kKvBf16 ? head_dim * 2 : (store == kKvNvfp4 ? head_dim / 2 : head_dim);
}

// A paged cache as the kernels see it. Token `slot` of a sequence lies in page table[seq][slot >> page_shift]; the
// row of one head starts page * page_bytes + (head * page_size + slot % page_size) * row_bytes into k (and v); scales,
// weights and positions are dense, [n_pages, n_kv_heads, page_size]. kKvNvfp4: the scales of a row's blocks, head_dim / 16
// bytes, start page * page_bytes + block_offset + (head * page_size + slot % page_size) * head_dim / 16 into k (and v).
struct KvView {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    float* weight;
    int32_t* position;
    int64_t page_bytes;
    int64_t block_offset;
    int64_t n_pages;
    const int32_t* table;   // [n_seqs, pages_per_seq]
    int64_t pages_per_seq;
    int64_t capacity;       // pages_per_seq << page_shift: slots that a sequence's row of the table can name
    int page_shift;
    int n_kv_heads;
    int head_dim;
    int store;              // KvStore
};

struct AppendParams {
    KvView c;
    const void* k;              // [n_tokens] rows of n_kv_heads * head_dim bf16, row_bytes apart
    const void* v;
    int64_t row_bytes;
    const int32_t* seq_lens;
    const int32_t* cu_tokens;   // [n_seqs + 1], or null: row t is the one new token of sequence t
    const int32_t* positions;   // [n_tokens], or null: a token's position is its slot
    int64_t n_seqs;
    int64_t n_tokens;
};

struct AttendParams {
    KvView c;
    void* out;                  // [n_seqs, n_q_heads * head_dim] bf16
    const void* q;              // [n_seqs] rows of n_q_heads * head_dim bf16, q_bytes apart
    int64_t q_bytes;
    const int32_t* seq_lens;
    float* lse;                 // [n_seqs, n_q_heads] or null
    float* lse2;                // workspace: the same in units of log2, for the accumulation of weights
    float* logits;              // workspace: [n_seqs, n_kv_heads, capacity, logit_heads], units of log2
    int64_t n_seqs;
    int64_t window;             // 0: no window
    float scale_log2;           // scale * log2(e)
    int n_q_heads;
    int group;                  // query heads of a key-value head
    int chunk_heads;            // query heads that a CTA takes at once: 8 or 16
    int chunks;                 // of a group
    int grid;                   // CTAs: the shares that the work is cut into
    int sms;
    float* part_o;              // workspace: [grid, 2, chunk_heads, head_dim], sums of the items that are cut
    float4* part_ml;            // workspace: [grid, 2, chunk_heads], their maxima, sums and exponents
    unsigned long long* arrived;   // workspace: [2, grid], where the deliveries of parts meet
    unsigned long long call;    // the call's number
    int logit_heads;
    int accumulate;
};

struct EvictParams {
    KvView c;
    const int32_t* seq_lens;
    int32_t* new_lens;
    int64_t n_seqs;
    int64_t budget;
    int64_t recent;
    int ctas_per_row;           // cluster size: the CTAs that share one sequence's head
    int slots_per_cta;          // slots of the longest row that one of them holds, even
};

// How the attention covers a call: chunk_heads, chunks and grid of AttendParams; `rows`: n_seqs * n_kv_heads.
struct AttendPlan {
    int chunk_heads, chunks, grid;
};
void plan_kv_attend(int head_dim, int store, int group, int sms, int64_t capacity, int64_t rows, AttendPlan* plan);

cudaError_t launch_kv_append(const AppendParams& p, int sms, cudaStream_t s);
cudaError_t launch_kv_attend(const AttendParams& p, cudaStream_t s);   // any store; the others: their own
cudaError_t launch_kv_attend_fp8(const AttendParams& p, cudaStream_t s);
cudaError_t launch_kv_attend_fp8_dynamic(const AttendParams& p, cudaStream_t s);
cudaError_t launch_kv_attend_nvfp4(const AttendParams& p, cudaStream_t s);
cudaError_t launch_kv_weights(const AttendParams& p, cudaStream_t s);
cudaError_t launch_kv_evict(const EvictParams& p, cudaStream_t s);
cudaError_t device_error_flags_kv_cache(unsigned int* flags, bool clear);
cudaError_t device_error_flags_kv_attention(unsigned int* flags, bool clear);
cudaError_t device_error_flags_kv_attention_fp8(unsigned int* flags, bool clear);
cudaError_t device_error_flags_kv_attention_fp8_dynamic(unsigned int* flags, bool clear);
cudaError_t device_error_flags_kv_attention_nvfp4(unsigned int* flags, bool clear);

// What the C-ABI layer keeps for every entry point (api.cu): the SM count of the current device, and the status of
// a launch (counts it, or keeps its cudaError_t).
int kv_sm_count();
int kv_finish_launch(cudaError_t e);

// Launch `kernel` with programmatic stream serialization, in clusters of `cluster` CTAs where that is over 1.
template <class... Args>
inline cudaError_t kv_launch(void (*kernel)(Args...), unsigned grid, unsigned threads, size_t smem, unsigned cluster,
                             cudaStream_t s, const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace mbd
