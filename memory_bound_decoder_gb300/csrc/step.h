// Internal interface between the host layer of a serving step's other operators (step_api.cu) and their kernels
// (rotary.cu, kv_pages.cu, prompt_attention.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mbd {

struct RotaryParams {
    const void* x;              // [n_tokens] rows of n_heads * head_dim bf16, x_bytes apart
    void* out;                  // the same, out_bytes apart; may be x
    int64_t x_bytes;
    int64_t out_bytes;
    const uint64_t* turns;      // [rotary_dim / 2]: 2^64 of a turn a position
    const int32_t* positions;   // [n_tokens], or null: a token's position is its row
    float amplitude;
    int64_t n_tokens;
    int n_heads;
    int head_dim;
    int rotary_dim;
    int interleaved;
    int units;                  // of 16 elements in a head: those turned, and where out is not x the rest
};

struct ResizeParams {
    int32_t* table;             // [n_seqs, pages_per_seq]
    int64_t pages_per_seq;
    int64_t capacity;           // slots that a row of the table can name
    int page_shift;
    int64_t n_pages;
    int32_t* ring;              // [n_pages]
    int32_t* ends;              // [2]: place of the first free page in the ring, number of free pages
    int32_t* lens;              // [n_seqs]
    const int32_t* want;        // [n_seqs]
    int32_t* seen;              // [n_seqs] or null
    int64_t n_seqs;
    int32_t* cu;                // [n_seqs + 1]
    int32_t* positions;         // [n_tokens] or null
    int64_t* slots;             // [n_tokens] or null
    int64_t n_tokens;
    int ctas;                   // of the cluster
};

struct PromptParams {
    CUtensorMap q_map, k_map, v_map;   // boxes of 64 elements and 128 rows, swizzled by 128 bytes
    const void* v;              // rows v_bytes apart, as in v_map
    int64_t v_bytes;
    void* out;                  // [n_tokens, n_q_heads * head_dim] bf16
    float* lse;                 // [n_tokens, n_q_heads] or null
    const int32_t* cu;          // [n_seqs + 1]
    int64_t n_seqs;
    int64_t n_tokens;
    int64_t window;             // 0: no window
    int64_t units;              // query heads, or pairs of them, that share a row tile's number
    int64_t items;              // numbers of row tiles (some of them no tile's) * units, at most 2^31 - 1: the grid
    float scale_log2;           // |scale| * log2(e), not 0
    int negate;                 // the scale is negative
    int pair_rows;              // a CTA's two tiles are neighbours in the rows, not two heads
    int n_q_heads;
    int group;                  // query heads of a key-value head
    int head_dim;
};

int prompt_tiles(int head_dim);   // tiles of 128 query rows that a CTA works on at a time
cudaError_t launch_prompt(const PromptParams& p, cudaStream_t s);
cudaError_t device_error_flags_prompt(unsigned int* flags, bool clear);
cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t s);
cudaError_t launch_kv_resize(const ResizeParams& p, cudaStream_t s);
cudaError_t device_error_flags_kv_pages(unsigned int* flags, bool clear);

}  // namespace mbd
