// Attention of one new token per sequence over the paged key-value cache.
//
// For query head h of sequence b, with its key-value head's keys K and values V of the slots in view:
//     x_j = scale * q . K_j,  lse = log sum_j exp(x_j),  p_j = exp(x_j - lse),  out = sum_j p_j V_j
// and, where weights are accumulated, weight[j] += sum over the group's query heads of p_j.
//
// One CTA per query head: each warp takes every fourth key, its lanes head_dim / 32 elements each, and keeps the
// running maximum and sum of its keys in units of log2; the four warps join at the end.
#include "kv_common.cuh"

namespace mbd {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

template <int D, int STORE>
__device__ __forceinline__ void load_row(const char* row, int lane, float (&v)[D / 32]) {
#pragma unroll
    for (int e = 0; e < D / 32; ++e) {
        if constexpr (STORE == kKvBf16)
            v[e] = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(row)[e * 32 + lane]) << 16);
        else
            v[e] = e4m3_value(reinterpret_cast<const uint8_t*>(row)[e * 32 + lane]);
    }
}

template <int D, int STORE>
__global__ void __launch_bounds__(kThreads) kv_attend_kernel(const __grid_constant__ AttendParams p) {
    __shared__ float s_out[kWarps][D], s_max[kWarps], s_sum[kWarps];
    constexpr int N = D / 32, kRow = D * (STORE == kKvBf16 ? 2 : 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t seq = blockIdx.x / p.n_q_heads;
    const int head = static_cast<int>(blockIdx.x - seq * p.n_q_heads), kv_head = head / p.group;
    pdl_trigger();
    pdl_wait();
    const int64_t len = kv_len(p.c, p.seq_lens[seq]);
    const int64_t first = p.window > 0 && p.window < len ? len - p.window : 0;
    float q[N], o[N];
    const uint16_t* qrow = reinterpret_cast<const uint16_t*>(static_cast<const char*>(p.q) + seq * p.q_bytes) + head * D;
#pragma unroll
    for (int e = 0; e < N; ++e) {
        q[e] = __uint_as_float(static_cast<uint32_t>(qrow[e * 32 + lane]) << 16);
        o[e] = 0.0f;
    }
    float m = -INFINITY, sum = 0.0f;
    for (int64_t j = first + warp; j < len; j += kWarps) {
        const int64_t page = kv_page(p.c, seq, j);
        if (page < 0) continue;
        float kx[N], vx[N], dot = 0.0f, vs = 1.0f;
        const int64_t at = kv_row(p.c, page, kv_head, j, kRow);
        load_row<D, STORE>(static_cast<const char*>(p.c.k) + at, lane, kx);
        load_row<D, STORE>(static_cast<const char*>(p.c.v) + at, lane, vx);
#pragma unroll
        for (int e = 0; e < N; ++e) dot += q[e] * kx[e];
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        float x = dot * p.scale_log2;
        if constexpr (STORE != kKvBf16) {
            const int64_t i = STORE == kKvFp8Dynamic ? kv_meta(p.c, page, kv_head, j) : 0;
            x *= p.c.k_scale[i];
            vs = p.c.v_scale[i];
        }
        if (p.accumulate && lane == 0)
            p.logits[((seq * p.c.n_kv_heads + kv_head) * p.c.capacity + j) * p.logit_heads + head % p.group] = x;
        const float top = fmaxf(m, x), base = top == -INFINITY ? 0.0f : top;
        const float old = exp2f(m - base), w = exp2f(x - base);
        m = top;
        sum = sum * old + w;
#pragma unroll
        for (int e = 0; e < N; ++e) o[e] = o[e] * old + w * vs * vx[e];
    }
#pragma unroll
    for (int e = 0; e < N; ++e) s_out[warp][e * 32 + lane] = o[e];
    if (lane == 0) {
        s_max[warp] = m;
        s_sum[warp] = sum;
    }
    __syncthreads();
    float top = s_max[0], total = 0.0f;
    for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_max[w]);
    const float base = top == -INFINITY ? 0.0f : top;
    for (int w = 0; w < kWarps; ++w) total += s_sum[w] * exp2f(s_max[w] - base);
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float v = 0.0f;
        for (int w = 0; w < kWarps; ++w) v += s_out[w][d] * exp2f(s_max[w] - base);
        static_cast<__nv_bfloat16*>(p.out)[(seq * p.n_q_heads + head) * D + d] =
            __float2bfloat16_rn(first < len ? v / total : 0.0f);
    }
    if (threadIdx.x == 0) {
        const float lse2 = first < len ? base + log2f(total) : -INFINITY;
        if (p.lse) p.lse[seq * p.n_q_heads + head] = lse2 * 0.693147180559945309f;
        if (p.accumulate) p.lse2[seq * p.n_q_heads + head] = lse2;
    }
}

// weight[slot] += sum over the group's query heads of exp2(logit - lse2): a thread per slot.
__global__ void __launch_bounds__(256) kv_weights_kernel(const __grid_constant__ AttendParams p) {
    pdl_trigger();
    pdl_wait();
    const int64_t row = blockIdx.y, seq = row / p.c.n_kv_heads;
    const int head = static_cast<int>(row - seq * p.c.n_kv_heads);
    const int64_t len = kv_len(p.c, p.seq_lens[seq]);
    const int64_t first = p.window > 0 && p.window < len ? len - p.window : 0;
    const float* lse2 = p.lse2 + seq * p.n_q_heads + head * p.group;
    for (int64_t j = first + static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; j < len; j += int64_t{256} * gridDim.x) {
        const int64_t page = kv_page(p.c, seq, j);
        if (page < 0) continue;
        const float* x = p.logits + (row * p.c.capacity + j) * p.logit_heads;
        float w = 0.0f;
        for (int h = 0; h < p.group; ++h) w += exp2f(x[h] - lse2[h]);
        p.c.weight[kv_meta(p.c, page, head, j)] += w;
    }
}

template <int D>
cudaError_t launch_d(const AttendParams& p, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(p.n_seqs * p.n_q_heads);
    switch (p.c.store) {
        case kKvBf16: return kv_launch(kv_attend_kernel<D, kKvBf16>, grid, kThreads, 0, 1, s, p);
        case kKvFp8Static: return kv_launch(kv_attend_kernel<D, kKvFp8Static>, grid, kThreads, 0, 1, s, p);
        case kKvFp8Dynamic: return kv_launch(kv_attend_kernel<D, kKvFp8Dynamic>, grid, kThreads, 0, 1, s, p);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_kv_attend(const AttendParams& p, cudaStream_t s) {
    switch (p.c.head_dim) {
        case 64: return launch_d<64>(p, s);
        case 128: return launch_d<128>(p, s);
        case 256: return launch_d<256>(p, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_weights(const AttendParams& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    const int64_t rows = p.n_seqs * p.c.n_kv_heads, blocks = (p.c.capacity + 255) / 256;
    cfg.gridDim = dim3(static_cast<unsigned>(blocks < 64 ? blocks : 64), static_cast<unsigned>(rows));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_weights_kernel, p);
}

cudaError_t device_error_flags_kv_attention(unsigned int* flags, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(flags, g_device_error_flags, sizeof(unsigned int));
    if (e == cudaSuccess && clear) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_device_error_flags, &zero, sizeof(unsigned int));
    }
    return e;
}

}  // namespace mbd
