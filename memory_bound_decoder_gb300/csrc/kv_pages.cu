// Pages and slots of a step, handed out on the GPU: lengths go from what they are to what is wanted, pages that are no
// longer needed go back to a ring of free pages, pages that are needed come from it, and the new tokens' rows get their
// packed offsets, positions and slots.
//
// All of it is prefix sums over the sequences and then independent items (pages given up, pages taken, tokens), so it is
// bound by latency: one launch of one cluster, whose CTAs each read the lengths and sum for themselves, which spares
// them an exchange, and then share the items evenly, whatever sequences they belong to (an item finds its sequence by a
// search of the sums in shared memory). One cluster barrier stands in between: pages given up are in the ring before
// any is taken, and every CTA has read the lengths before they change. A queue rather than a stack, because pages that
// come and pages that go then never touch the same places at once. Measured on one GB300 (the kernel alone): 128 sequences that
// grow by a token 7.8 us with one CTA (8.1 with a cluster of 8), 256 with prompts of up to 700 tokens among them (18000 tokens) 12.0
// with 8 (15 with 4): a chain of round trips, each half a microsecond or more (ends and lengths, the sums, pages given up, the
// cluster's barrier, pages taken), where everything is granted with one scan, else with three.
#include "kv_common.cuh"
#include "mbd.h"
#include "step.h"

namespace mbd {

namespace {

constexpr int kResizeThreads = 1024;
constexpr int kResizeWarps = kResizeThreads / 32;

// Of each sequence: length before and after, tokens seen before, and how many tokens, pages taken and pages given up
// come before it.
struct ResizeSmem {
    int64_t sum[3][kResizeWarps];
    int64_t carry[3];
};
constexpr int kResizeArrays = 6;
constexpr size_t resize_shared(int64_t n) { return static_cast<size_t>(n + 1) * kResizeArrays * sizeof(int32_t); }

// Exclusive sums of N values over the CTA's threads, on top of sm.carry, which grows by the totals.
template <int N>
__device__ __forceinline__ void scan_block(ResizeSmem& sm, const int64_t (&own)[N], int64_t (&before)[N]) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t upto[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        upto[k] = own[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto[k], o);
            if (lane >= o) upto[k] += x;
        }
        if (lane == 31) sm.sum[k][warp] = upto[k];
    }
    __syncthreads();
    int64_t base[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int64_t mine = sm.sum[k][lane];
        int64_t all = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, all, o);
            if (lane >= o) all += x;
        }
        base[k] = sm.carry[k] + __shfl_sync(0xffffffffu, all - mine, warp);
        before[k] = base[k] + upto[k] - own[k];
    }
    __syncthreads();
    if (threadIdx.x == kResizeThreads - 1)
#pragma unroll
        for (int k = 0; k < N; ++k) sm.carry[k] = base[k] + upto[k];
    __syncthreads();
}

// The last b with before[b] <= i, of n ascending sums from 0.
__device__ __forceinline__ int sequence_of(const int32_t* before, int n, int64_t i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= i) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kResizeThreads) kv_resize_kernel(const __grid_constant__ ResizeParams p) {
    extern __shared__ __align__(16) int32_t arrays[];
    __shared__ ResizeSmem sm;
    const int n = static_cast<int>(p.n_seqs), tid = threadIdx.x;
    int32_t *const old_len = arrays, *const new_len = old_len + n + 1, *const seen = new_len + n + 1,
                  *const rows_before = seen + n + 1, *const taken_before = rows_before + n + 1,
                  *const given_before = taken_before + n + 1;
    const int rank = static_cast<int>(blockIdx.x), threads = static_cast<int>(gridDim.x) * kResizeThreads;
    pdl_trigger();
    pdl_wait();
    const int64_t head = p.ends[0], free_pages = p.ends[1];
    const bool good = head >= 0 && head < p.n_pages && free_pages >= 0 && free_pages <= p.n_pages;
    if (!good && tid == 0) kv_bad_index();
    auto pages_of = [&](int64_t len) { return (len + (int64_t{1} << p.page_shift) - 1) >> p.page_shift; };
    // Pages and rows that sequence b asks for.
    auto asked = [&](int b, int64_t (&x)[2]) {
        x[0] = x[1] = 0;
        if (b >= n || new_len[b] <= old_len[b]) return;
        x[0] = pages_of(new_len[b]) - pages_of(old_len[b]);
        x[1] = static_cast<int64_t>(new_len[b]) - old_len[b];
    };
    auto restart = [&] {
        __syncthreads();
        if (tid < 3) sm.carry[tid] = 0;
        __syncthreads();
    };
    restart();

    // Lengths, and what is asked for and given up. A sequence with a length out of range stays as it is.
    for (int b0 = 0; b0 < n; b0 += kResizeThreads) {
        const int b = b0 + tid;
        int64_t x[3] = {0, 0, 0}, before[3];
        if (b < n) {
            const int32_t from = p.lens[b], to = p.want[b];
            const bool fits = from >= 0 && from <= p.capacity && to >= 0 && to <= p.capacity;
            if (!fits) kv_bad_index();
            old_len[b] = from;
            new_len[b] = fits && good ? to : from;
            seen[b] = p.seen ? p.seen[b] : from;
            int64_t of[2];
            asked(b, of);
            x[0] = of[0];
            x[1] = of[1];
            if (new_len[b] < from) x[2] = pages_of(from) - pages_of(to);
        }
        scan_block<3>(sm, x, before);
        if (b < n) {   // (pages given up: the host bounds the table's entries; the others fit if all of them are granted)
            taken_before[b] = static_cast<int32_t>(before[0]);
            rows_before[b] = static_cast<int32_t>(before[1]);
            given_before[b] = static_cast<int32_t>(before[2]);
        }
    }
    // No more than n_pages have a place in the ring; more can only be pages that were named twice.
    const int64_t all_given = sm.carry[2], given = min(all_given, good ? p.n_pages - free_pages : 0);
    if (all_given > given && tid == 0) kv_bad_index();
    const int64_t there = good ? free_pages + given : 0;
    if (sm.carry[0] > there || sm.carry[1] > p.n_tokens) {
        // More is asked for than there is: granted in the order of the sequences, and summed anew.
        restart();
        for (int b0 = 0; b0 < n; b0 += kResizeThreads) {
            int64_t x[2], before[2];
            asked(b0 + tid, x);
            scan_block<2>(sm, x, before);
            if (x[1] > 0 && ((x[0] > 0 && before[0] + x[0] > there) || before[1] + x[1] > p.n_tokens))
                new_len[b0 + tid] = old_len[b0 + tid];
        }
        restart();
        for (int b0 = 0; b0 < n; b0 += kResizeThreads) {
            int64_t x[2], before[2];
            asked(b0 + tid, x);
            scan_block<2>(sm, x, before);
            if (b0 + tid >= n) continue;
            taken_before[b0 + tid] = static_cast<int32_t>(before[0]);
            rows_before[b0 + tid] = static_cast<int32_t>(before[1]);
        }
    }
    const int64_t taken = sm.carry[0], rows = sm.carry[1];
    __syncthreads();

    auto ring_place = [&](int64_t i) {
        const int64_t at = head + i;
        return at >= 2 * p.n_pages ? at - 2 * p.n_pages : (at >= p.n_pages ? at - p.n_pages : at);
    };
    for (int64_t i = static_cast<int64_t>(rank) * kResizeThreads + tid; i < all_given; i += threads) {
        const int b = sequence_of(given_before, n, i);
        int32_t* entry = p.table + b * p.pages_per_seq + pages_of(new_len[b]) + (i - given_before[b]);
        const int32_t page = *entry;
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.n_pages)) kv_bad_index();
        if (i < given) p.ring[ring_place(free_pages + i)] = page;
        *entry = -1;
    }
    if (p.ctas > 1) cg::this_cluster().sync();   // (of global memory too: release and acquire at cluster scope)
    else __syncthreads();

    for (int64_t i = static_cast<int64_t>(rank) * kResizeThreads + tid; i < taken; i += threads) {
        const int b = sequence_of(taken_before, n, i);
        const int32_t page = __ldcg(p.ring + ring_place(i));
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(p.n_pages)) kv_bad_index();
        p.table[b * p.pages_per_seq + pages_of(old_len[b]) + (i - taken_before[b])] = page;
    }
    for (int64_t i = static_cast<int64_t>(rank) * kResizeThreads + tid; i < p.n_tokens; i += threads) {
        int64_t slot = -1;
        int32_t position = 0;
        if (i < rows) {
            const int b = sequence_of(rows_before, n, i);
            const int64_t add = i - rows_before[b], at = old_len[b] + add, had = pages_of(old_len[b]);
            position = seen[b] + static_cast<int32_t>(add);
            if (p.slots) {
                const int64_t k = at >> p.page_shift;
                const int32_t page = k < had ? p.table[b * p.pages_per_seq + k]
                                             : __ldcg(p.ring + ring_place(taken_before[b] + (k - had)));
                if (static_cast<uint32_t>(page) < static_cast<uint32_t>(p.n_pages))
                    slot = (static_cast<int64_t>(page) << p.page_shift) + (at & ((int64_t{1} << p.page_shift) - 1));
                else
                    kv_bad_index();
            }
        }
        if (p.slots) p.slots[i] = slot;
        if (p.positions) p.positions[i] = position;
    }
    // Lengths, offsets and what the ring holds now.
    for (int b = rank * kResizeThreads + tid; b < n; b += threads) {
        const int32_t from = old_len[b], to = new_len[b];
        p.cu[b] = rows_before[b];
        if (to != from) p.lens[b] = to;
        if (p.seen) {
            if (to > from) p.seen[b] = seen[b] + (to - from);
            else if (to == 0 && good && p.want[b] == 0) p.seen[b] = 0;   // (not where an empty row was refused, or stays as it is)
        }
    }
    if (rank == 0 && tid == 0) {
        p.cu[n] = static_cast<int32_t>(rows);
        if (good) {
            p.ends[0] = static_cast<int32_t>(ring_place(taken));
            p.ends[1] = static_cast<int32_t>(there - taken);
        }
    }
}

}  // namespace

cudaError_t launch_kv_resize(const ResizeParams& p, cudaStream_t s) {
    const size_t smem = resize_shared(p.n_seqs);
    if (smem > 40 * 1024) {   // the limit is the kernel's: always the largest call's, whatever other threads launch
        const cudaError_t e = cudaFuncSetAttribute(kv_resize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(resize_shared(MBD_KV_MAX_RESIZE_SEQS)));
        if (e != cudaSuccess) return e;
    }
    return kv_launch(kv_resize_kernel, static_cast<unsigned>(p.ctas), kResizeThreads, smem, static_cast<unsigned>(p.ctas), s, p);
}

cudaError_t device_error_flags_kv_pages(unsigned int* flags, bool clear) { return kv_error_flags(flags, clear); }

}  // namespace mbd
