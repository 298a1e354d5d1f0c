// Decode attention over a paged cache (kv_attention_impl.cuh): the bf16 cache, the plan of a call, and the
// accumulation of attention weights.
#include "kv_attention_impl.cuh"

namespace mbd {

namespace {

constexpr int kWeighThreads = 256, kWeighSlots = 4;   // slots of a thread: their loads are in flight together

// weight[slot] += sum over the group's query heads of exp2(logit - lse2), with the logits that the attention left. Reads 4
// bytes a query head and slot (from L2, where short caches are concerned) besides the 8 of the weight.
__global__ void __launch_bounds__(kWeighThreads) kv_weights_kernel(const __grid_constant__ AttendParams p, int blocks_per_row) {
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.x / blocks_per_row, seq = row / p.c.n_kv_heads;
    const int block = static_cast<int>(blockIdx.x - row * blocks_per_row);
    const int head = static_cast<int>(row - seq * p.c.n_kv_heads);
    const int64_t len = kv_len(p.c, p.seq_lens[seq]);
    const int64_t first = p.window > 0 && p.window < len ? len - p.window : 0;
    const float* lse2 = p.lse2 + seq * p.n_q_heads + head * p.group;
    const int32_t* table = p.c.table + seq * p.c.pages_per_seq;
    for (int64_t base = first + static_cast<int64_t>(block) * kWeighThreads * kWeighSlots; base < len;
         base += int64_t{kWeighThreads} * kWeighSlots * blocks_per_row) {
        // Loads without a branch between them: a thread behind the end repeats the last slot, a page outside the pool
        // counts as page 0, and neither stores.
        int page[kWeighSlots];
        float w[kWeighSlots], old[kWeighSlots];
        auto slot = [&](int u) { return min(base + u * kWeighThreads + threadIdx.x, len - 1); };
#pragma unroll
        for (int u = 0; u < kWeighSlots; ++u) {
            page[u] = table[slot(u) >> p.c.page_shift];
            w[u] = 0.0f;
        }
#pragma unroll
        for (int u = 0; u < kWeighSlots; ++u) {
            const bool good = static_cast<uint32_t>(page[u]) < static_cast<uint32_t>(p.c.n_pages);
            old[u] = p.c.weight[kv_meta(p.c, good ? page[u] : 0, head, slot(u))];
        }
        for (int h = 0; h < p.group; h += 2) {
            const float a = lse2[h], b = h + 1 < p.group ? lse2[h + 1] : 0.0f;
#pragma unroll
            for (int u = 0; u < kWeighSlots; ++u) {
                const float2 x = *reinterpret_cast<const float2*>(p.logits + (row * p.c.capacity + slot(u)) * p.logit_heads + h);
                w[u] += ex2(x.x - a) + (h + 1 < p.group ? ex2(x.y - b) : 0.0f);
            }
        }
#pragma unroll
        for (int u = 0; u < kWeighSlots; ++u)
            if (base + u * kWeighThreads + threadIdx.x < len &&
                static_cast<uint32_t>(page[u]) < static_cast<uint32_t>(p.c.n_pages))
                p.c.weight[kv_meta(p.c, page[u], head, slot(u))] = old[u] + w[u];
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
    const int64_t rows = p.n_seqs * p.c.n_kv_heads, most = p.window > 0 && p.window < p.c.capacity ? p.window : p.c.capacity;
    const int64_t blocks = (most + kWeighThreads * kWeighSlots - 1) / (kWeighThreads * kWeighSlots);
    const int per_row = static_cast<int>(blocks < 64 ? blocks : 64);
    return kv_launch(kv_weights_kernel, static_cast<unsigned>(rows * per_row), kWeighThreads, 0, 1, s, p, per_row);
}

cudaError_t device_error_flags_kv_attention(unsigned int* flags, bool clear) { return kv_error_flags(flags, clear); }

}  // namespace mbd
