// Decode attention over a paged cache (kv_attention_impl.cuh): the bf16 cache, the plan of a call, and the
// accumulation of attention weights.
#include "kv_attention_impl.cuh"

namespace mbd {

namespace {

constexpr int kWeighThreads = 256, kWeighSlots = 4;   // slots of a lane group whose loads are in flight together

template <int V>
struct Logits {
    float v[V];
};
__device__ __forceinline__ void load_logits(Logits<4>& l, const float* p) {
    const float4 x = __ldcs(reinterpret_cast<const float4*>(p));
    l = Logits<4>{{x.x, x.y, x.z, x.w}};
}
__device__ __forceinline__ void load_logits(Logits<2>& l, const float* p) {
    const float2 x = __ldcs(reinterpret_cast<const float2*>(p));
    l = Logits<2>{{x.x, x.y}};
}

// weight[slot] += sum over the group's query heads of exp2(logit - lse2), with the logits that the attention left. Reads 4
// bytes a query head and slot (from L2, where they fit) besides the 8 of the weight. 2^shift lanes own a slot, V query
// heads each at a time, so that a warp reads whole lines of logits. The sum goes to its weight as a reduction in L2 (the
// only one for it in the call), which spares the round trip of reading the weight.
template <int V>
__global__ void __launch_bounds__(kWeighThreads) kv_weights_kernel(const __grid_constant__ AttendParams p, int blocks_per_row,
                                                                   int shift) {
    pdl_trigger();
    pdl_wait();
    const unsigned row = blockIdx.x / blocks_per_row, seq = row / p.c.n_kv_heads;
    const int block = static_cast<int>(blockIdx.x - row * blocks_per_row), head = static_cast<int>(row - seq * p.c.n_kv_heads);
    const int lanes = 1 << shift, part = threadIdx.x & (lanes - 1), place_mask = (1 << p.c.page_shift) - 1;
    const int len = static_cast<int>(kv_len(p.c, p.seq_lens[seq]));
    const int first = p.window > 0 && p.window < len ? len - static_cast<int>(p.window) : 0;
    const float* lse2 = p.lse2 + static_cast<int64_t>(seq) * p.n_q_heads + head * p.group;
    const float* logits = p.logits + static_cast<int64_t>(row) * p.c.capacity * p.logit_heads;
    const int32_t* table = p.c.table + static_cast<int64_t>(seq) * p.c.pages_per_seq;
    float* weight = p.c.weight + (static_cast<int64_t>(head) << p.c.page_shift);   // of page 0, this head
    const int64_t page_weights = static_cast<int64_t>(p.c.n_kv_heads) << p.c.page_shift;
    const int step = kWeighThreads >> shift;   // slots that the CTA reads at once
    float l[V];
    auto load_lse = [&](int h) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            l[i] = h + i < p.group ? lse2[h + i] : 0.0f;
            if (l[i] == -INFINITY) l[i] = INFINITY;   // every logit is -inf: nothing to add (-inf - -inf would be NaN)
        }
    };
    load_lse(part * V);
    for (int base = first + block * step * kWeighSlots; base < len; base += step * kWeighSlots * blocks_per_row) {
        // Loads without a branch between them: a thread behind the end repeats the last slot.
        int page[kWeighSlots], slot[kWeighSlots];
        float w[kWeighSlots];
#pragma unroll
        for (int u = 0; u < kWeighSlots; ++u) {
            slot[u] = min(base + u * step + static_cast<int>(threadIdx.x >> shift), len - 1);
            page[u] = table[slot[u] >> p.c.page_shift];
            w[u] = 0.0f;
        }
        for (int h = part * V; h < p.group; h += lanes * V) {   // once, up to 128 query heads
            if (h >= lanes * V) load_lse(h);
            Logits<V> x[kWeighSlots];
#pragma unroll
            for (int u = 0; u < kWeighSlots; ++u) load_logits(x[u], logits + static_cast<int64_t>(slot[u]) * p.logit_heads + h);
#pragma unroll
            for (int u = 0; u < kWeighSlots; ++u)
#pragma unroll
                for (int i = 0; i < V; ++i) w[u] += h + i < p.group ? ex2(x[u].v[i] - l[i]) : 0.0f;   // (padding holds anything)
            if (p.group > lanes * V) load_lse(part * V);
        }
#pragma unroll
        for (int u = 0; u < kWeighSlots; ++u) {
            for (int o = lanes >> 1; o > 0; o >>= 1) w[u] += __shfl_xor_sync(0xffffffffu, w[u], o);
            if (part == 0 && base + u * step + static_cast<int>(threadIdx.x >> shift) < len &&
                static_cast<uint32_t>(page[u]) < static_cast<uint32_t>(p.c.n_pages))
                atomicAdd(weight + page[u] * page_weights + (slot[u] & place_mask), w[u]);
        }
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
    int shift = 0;
    while (shift < 5 && (4 << shift) < p.group) ++shift;
    const int64_t slots = int64_t{kWeighThreads >> shift} * kWeighSlots, blocks = (most + slots - 1) / slots;
    // A few waves of CTAs at most: each first waits for its sequence's length.
    const int64_t want = (int64_t{16} * p.sms + rows - 1) / rows;
    const int per_row = static_cast<int>(blocks < want ? blocks : want);
    const unsigned grid = static_cast<unsigned>(rows * per_row);
    return p.logit_heads < 4 ? kv_launch(kv_weights_kernel<2>, grid, kWeighThreads, 0, 1, s, p, per_row, 0)
                             : kv_launch(kv_weights_kernel<4>, grid, kWeighThreads, 0, 1, s, p, per_row, shift);
}

cudaError_t device_error_flags_kv_attention(unsigned int* flags, bool clear) { return kv_error_flags(flags, clear); }

}  // namespace mbd
