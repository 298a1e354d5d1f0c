// Rotary positions: each pair (a, b) of a head's elements is turned by its token's position times the pair's frequency,
//     a' = A (a cos t - b sin t),  b' = A (b cos t + a sin t),
// with the pairs half a rotary_dim apart or next to one another, and the elements behind rotary_dim as they are.
//
// Angles. A frequency is kept as a 64-bit fraction of a turn, so position * frequency mod 2^64 is the exact angle of the
// table's frequency, reduced to one turn by the overflow alone: at position 2^31 the angle is as good as at 1, where a
// product in fp32 is off by 2^-24 of the whole angle (0.008 rad at position 131071). Sine and cosine come from
// sincospif of the signed fraction, in fp32.
//
// Bound by bytes (each element is read and written once) and, for a decode step's few rows, by latency. A CTA owns a
// token: its threads' loads are under way while the token's rotary_dim / 2 angles are computed once, in shared memory,
// for all heads. A thread turns 16 elements (8 pairs, two 16-byte vectors) of one head at a time and keeps to the same 8
// pairs in all its heads, so their sines and cosines stay in registers. Measured on one GB300: 16380 rows of 72 heads of 128
// 91.0 us, 6630 GB/s; 9001 rows of 32 heads of 64, half of each turned, 13.4 us (5510 GB/s, part of them from L2); a decode
// step's 128 rows of 40 heads 5.7 us, the host's call.
#include "common.cuh"
#include "kv.h"
#include "step.h"

namespace mbd {

namespace {

constexpr int kRotaryThreads = 512;   // at most
constexpr int kRotaryBatch = 2;   // heads of a thread whose loads are in flight together

template <bool INTERLEAVED>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
    extern __shared__ __align__(16) float2 cs[];   // of the token: cosine and sine of each pair, times the amplitude
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, threads = blockDim.x, per_pass = threads / p.units;   // heads that the CTA's threads cover at once
    const int head0 = tid / p.units, unit = tid - head0 * p.units;
    const int64_t token = blockIdx.x;
    const bool turned = unit * 16 < p.rotary_dim;
    // The two vectors of a unit: adjacent, or half a rotary_dim apart.
    const int first = INTERLEAVED || !turned ? unit * 32 : unit * 16;
    const int second = INTERLEAVED || !turned ? first + 16 : first + p.rotary_dim;
    const char* x = static_cast<const char*>(p.x) + token * p.x_bytes;
    char* out = static_cast<char*>(p.out) + token * p.out_bytes;
    const int head_bytes = p.head_dim * 2;
    uint4 a[kRotaryBatch], b[kRotaryBatch];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kRotaryBatch; ++u) {
            const int head = base + u * per_pass + head0;
            if (head0 >= per_pass || head >= p.n_heads) continue;
            const char* from = x + static_cast<int64_t>(head) * head_bytes;
            a[u] = load_stream(reinterpret_cast<const uint4*>(from + first));
            b[u] = load_stream(reinterpret_cast<const uint4*>(from + second));
        }
    };
    load(0);   // before the angles, which need the position first
    const int64_t position = p.positions ? static_cast<int64_t>(p.positions[token]) : token;
    for (int i = tid; i < p.rotary_dim / 2; i += threads) {
        const uint64_t turns = static_cast<uint64_t>(position) * p.turns[i];
        float s, c;
        sincospif(__ll2float_rn(static_cast<int64_t>(turns)) * 0x1p-63f, &s, &c);
        cs[i] = make_float2(c * p.amplitude, s * p.amplitude);
    }
    __syncthreads();
    float2 r[8];
    if (turned) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = cs[unit * 8 + i];
    }
    for (int base = 0; base < p.n_heads; base += per_pass * kRotaryBatch) {
        if (base > 0) load(base);
#pragma unroll
        for (int u = 0; u < kRotaryBatch; ++u) {
            const int head = base + u * per_pass + head0;
            if (head0 >= per_pass || head >= p.n_heads) continue;
            if (turned) {
                uint32_t va[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, vb[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (INTERLEAVED) {
                        const float2 x0 = bf16x2_to_float2(va[i]), x1 = bf16x2_to_float2(vb[i]);
                        va[i] = pack_bf16x2(x0.x * r[i].x - x0.y * r[i].y, x0.y * r[i].x + x0.x * r[i].y);
                        vb[i] = pack_bf16x2(x1.x * r[4 + i].x - x1.y * r[4 + i].y, x1.y * r[4 + i].x + x1.x * r[4 + i].y);
                    } else {
                        const float2 x0 = bf16x2_to_float2(va[i]), x1 = bf16x2_to_float2(vb[i]);
                        const float2 e = r[2 * i], f = r[2 * i + 1];
                        va[i] = pack_bf16x2(x0.x * e.x - x1.x * e.y, x0.y * f.x - x1.y * f.y);
                        vb[i] = pack_bf16x2(x1.x * e.x + x0.x * e.y, x1.y * f.x + x0.y * f.y);
                    }
                }
                a[u] = make_uint4(va[0], va[1], va[2], va[3]);
                b[u] = make_uint4(vb[0], vb[1], vb[2], vb[3]);
            }
            char* to = out + static_cast<int64_t>(head) * head_bytes;
            *reinterpret_cast<uint4*>(to + first) = a[u];
            *reinterpret_cast<uint4*>(to + second) = b[u];
        }
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p, cudaStream_t s) {
    // Threads for kRotaryBatch units each, where that is not too many: 72 heads of 128 (16380 rows) take 91.0 us with 288 threads,
    // 99.9 with 256, whose last round is mostly idle; 32 heads of 64 (9001 rows) 13.4 with 64 and 19.1 with 256.
    const int64_t want = (static_cast<int64_t>(p.units) * ((p.n_heads + kRotaryBatch - 1) / kRotaryBatch) + 31) / 32 * 32;
    int threads = static_cast<int>(want < kRotaryThreads ? want : kRotaryThreads);
    if (threads < 64) threads = 64;
    const size_t smem = static_cast<size_t>(p.rotary_dim) / 2 * sizeof(float2);
    const unsigned grid = static_cast<unsigned>(p.n_tokens);
    return p.interleaved ? kv_launch(rotary_kernel<true>, grid, threads, smem, 1, s, p)
                         : kv_launch(rotary_kernel<false>, grid, threads, smem, 1, s, p);
}

}  // namespace mbd
