// Decode attention over a paged cache (kv_attention_impl.cuh): the bf16 cache, the plan of a call, and the
// accumulation of attention weights.
#include "kv_attention_impl.cuh"

namespace mbd {

namespace {

// weight[slot] += sum over the group's query heads of exp2(logit - lse2): a thread per slot.
__global__ void __launch_bounds__(256) kv_weights_kernel(const __grid_constant__ AttendParams p, int blocks_per_row) {
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.x / blocks_per_row, seq = row / p.c.n_kv_heads;
    const int block = static_cast<int>(blockIdx.x - row * blocks_per_row);
    const int head = static_cast<int>(row - seq * p.c.n_kv_heads);
    const int64_t len = kv_len(p.c, p.seq_lens[seq]);
    const int64_t first = p.window > 0 && p.window < len ? len - p.window : 0;
    const float* lse2 = p.lse2 + seq * p.n_q_heads + head * p.group;
    for (int64_t j = first + static_cast<int64_t>(block) * 256 + threadIdx.x; j < len; j += int64_t{256} * blocks_per_row) {
        const int64_t page = kv_page(p.c, seq, j);
        if (page < 0) continue;
        const float* x = p.logits + (row * p.c.capacity + j) * p.logit_heads;
        float w = 0.0f;
        for (int h = 0; h < p.group; ++h) w += ex2(x[h] - lse2[h]);
        p.c.weight[kv_meta(p.c, page, head, j)] += w;
    }
}

}  // namespace

void plan_kv_attend(int head_dim, int store, int group, int sms, int64_t capacity, int64_t rows, AttendPlan* plan) {
    // Up to 8 query heads of a group fit one 8-column operand; more take two of them (not at head_dim 256, whose
    // accumulators would not fit the registers), in chunks of 16 (8).
    plan->chunk_heads = group > 8 && head_dim < 256 ? 16 : 8;
    plan->chunks = (group + plan->chunk_heads - 1) / plan->chunk_heads;
    const int64_t tile = int64_t{step_keys(head_dim, store)} * kWarps;
    // CTAs that are resident at once, no more than there can be tiles.
    const int64_t resident = int64_t{sms} * resident_ctas(head_dim, store, plan->chunk_heads / 8);
    const int64_t items = rows * plan->chunks;
    const int64_t tiles_per_item = (capacity + tile - 1) / tile + 1;
    plan->grid = static_cast<int>(items >= resident || items * tiles_per_item >= resident ? resident
                                                                                          : items * tiles_per_item);
}

cudaError_t launch_kv_attend(const AttendParams& p, cudaStream_t s) {
    switch (p.c.store) {
        case kKvBf16: return launch_store<kKvBf16>(p, s);
        case kKvFp8Static: return launch_kv_attend_fp8(p, s);
        case kKvFp8Dynamic: return launch_kv_attend_fp8_dynamic(p, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_weights(const AttendParams& p, cudaStream_t s) {
    const int64_t rows = p.n_seqs * p.c.n_kv_heads, blocks = (p.c.capacity + 255) / 256;
    const int per_row = static_cast<int>(blocks < 64 ? blocks : 64);
    return kv_launch(kv_weights_kernel, static_cast<unsigned>(rows * per_row), 256, 0, 1, s, p, per_row);
}

cudaError_t device_error_flags_kv_attention(unsigned int* flags, bool clear) { return kv_error_flags(flags, clear); }

}  // namespace mbd
