// Paged key-value cache: appending new tokens, and eviction by accumulated attention weight.
//
// Append. Row (token t, head h) of the stacked projection goes to slot lens[seq] - (new tokens of seq) + i of its
// sequence, as it is (bf16) or as E4M3 codes of value / scale; the dynamic scale is amax / 448 of the head's row.
// Both divisions are rounded to nearest, so codes and scales are those of the definition, ties included. Bound by bytes (2 D
// in, D or 2 D out for each of k and v) and, for a decode step's few rows, by latency: the rows need no slot to be read,
// so their loads are under way while the slots are looked up. head_dim / 8 lanes own a row, 16 bytes of k and of v
// each, so the maximum of a row is a few shuffles and nothing is staged. Measured on one GB300: 8190 prompt tokens of 8
// heads of 128 in bf16 7.4 us (5180 GB/s of the operation's bytes, part of them from L2), 8700 into E4M3 with a static
// scale 13.8 us (3870 GB/s) and with a scale a row 14.9, 128 single tokens 6 us (the host's call). The E4M3 forms are short of
// the bf16 one's rate for two reasons that a capture shows together: warps wait first of all at the block's barrier, for the
// slots and then for the static scales loaded behind it, and issue is busy half of the time, the ALU pipe 46%.
//
// Eviction. Of the `len` slots of one sequence and head the `budget` best stay: first those whose position is
// among the newest `recent`, then those of the largest weight, equal ones by the lowest slot. A kept row behind
// the budget moves into a slot before it that is given up, the i-th such row into the i-th such slot, so sources
// (>= budget) and destinations (< budget) never meet: nothing is staged, rows that may stay where they are do, and
// the order of the moves is free. One cluster owns a sequence's head: each CTA keeps its share of the slots as
// order-preserving 32-bit keys in shared memory (read from HBM once), the budget-th largest key is found by a
// radix selection of 8 bits a pass whose histograms are added up through distributed shared memory, and the
// ranks of the moving rows come from ballots and one scan in slot order. Measured on one GB300, the selection by calls whose
// best slots lie before the budget already: 16 sequences of 1500..4099 tokens to 2048, 8 heads of 128 in bf16, 27 us, 11 of
// them launch and selection, 16 moves (their bytes take 10 at the copy rate; only the longer rows' CTAs have any); one of 131072
// to 32768 in FP8 55 us, 25 of them launch and selection (up to eight cluster barriers and the passes between them), 31
// moves (16 at the copy rate; a cluster of 16 for each of 8 heads is all that the card's GPCs hold at once).
#include <cooperative_groups.h>

#include "kv_common.cuh"
#include "mbd.h"

namespace mbd {

namespace {

// ------------------------------------------------------------------------------------------ append

constexpr int kAppendThreads = 256;
constexpr int kAppendMaxTokens = 16;   // tokens of one CTA

// The sequence that owns row t of the new tokens, the last b with cu[b] <= t, found by a whole warp: 32 places at a time.
__device__ __forceinline__ int64_t owner_of(const int32_t* cu, int64_t n_seqs, int64_t t) {
    const int lane = threadIdx.x & 31;
    int64_t lo = 0, hi = n_seqs;   // cu[lo] <= t (or lo == 0), cu[hi] > t (or hi == n_seqs)
    while (hi - lo > 1) {
        const int64_t step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
        const unsigned above = __ballot_sync(0xffffffffu, at >= hi || cu[at] > t);   // the last lane's always is
        const int64_t from = lo + (__ffs(above) - 1) * step;
        hi = min(hi, from + step);
        lo = from;
    }
    return lo;
}

// A scale to divide by. A correctly rounded quotient from the correctly rounded reciprocal r and the remainder of v r
// (Markstein's theorem, "IA-64 and Elementary Functions", 2000; it excludes divisors whose significand is all ones):
// three instructions for two elements. It needs a remainder that does not underflow, so scales below 2^-60 (or above
// 2^60) are divided by.
struct Divisor {
    float scale, r;
    uint32_t most, least;   // +-1024 scales as pairs of bf16: codes saturate at 448, and the quotient has to stay finite
    bool fast;
};

__device__ __forceinline__ Divisor divisor(float scale) {
    Divisor d;
    d.scale = scale;
    d.r = __frcp_rn(scale);
    d.most = pack_bf16x2(1024.0f * scale, 1024.0f * scale);
    d.least = d.most ^ 0x80008000u;
    d.fast = scale >= 0x1p-60f && scale <= 0x1p60f && (__float_as_uint(scale) & 0x7fffffu) != 0x7fffffu;
    return d;
}

__device__ __forceinline__ float2 quotient(float2 v, const Divisor& d) {
    const float2 r = f2(d.r), q = __fmul2_rn(v, r);
    return __ffma2_rn(__ffma2_rn(q, f2(-d.scale), v), r, q);
}

__device__ __forceinline__ uint32_t clamp_bf16x2(uint32_t w, const Divisor& d) {
    uint32_t x;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w), "r"(d.most));
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(x), "r"(d.least));
    return x;
}

// Eight bf16 values over one scale as E4M3 codes; a zero scale gives zero codes. CLAMP: the values may exceed 1024
// scales (they do not where the scale is the row's own).
template <bool CLAMP>
__device__ __forceinline__ uint2 encode(const uint4& x, const Divisor& s) {
    if (s.scale == 0.0f) return make_uint2(0u, 0u);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float2 d[4];
    if (s.fast) {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = quotient(bf16x2_to_float2(CLAMP ? clamp_bf16x2(w[i], s) : w[i]), s);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = make_float2(__fdiv_rn(bf16_lo(w[i]), s.scale), __fdiv_rn(bf16_hi(w[i]), s.scale));
    }
    return make_uint2(pack_e4m3x4(d[0], d[1]), pack_e4m3x4(d[2], d[3]));
}

// Largest magnitude of eight bf16 values.
__device__ __forceinline__ float amax(const uint4& x) {
    uint32_t m = max_bf16x2_bits(max_bf16x2_bits(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                 max_bf16x2_bits(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
    return fmaxf(bf16_lo(m), bf16_hi(m));
}

template <int STORE, int LANES>   // LANES = head_dim / 8: the lanes that own one head's row
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendParams p,
                                                                   int tokens_per_cta, unsigned inverse) {
    // Of each token: the byte offset of head 0's row in the pools (-1: no slot), the index of its scale, the slot.
    __shared__ int64_t s_row[kAppendMaxTokens], s_meta[kAppendMaxTokens];
    __shared__ int s_slot[kAppendMaxTokens];
    constexpr int kRow = LANES * (STORE == kKvBf16 ? 16 : 8);
    pdl_trigger();
    pdl_wait();
    const int64_t first = static_cast<int64_t>(blockIdx.x) * tokens_per_cta;
    const int tid = threadIdx.x;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(tokens_per_cta), p.n_tokens - first));
    const int per_token = p.c.n_kv_heads * LANES;   // 16-byte vectors of one token's keys
    const int total = tokens * per_token, lane = tid % LANES;
    constexpr int kBatch = 2;                       // vectors of k and of v that a thread has in flight
    // i / per_token: `inverse` is 2^32 / per_token rounded up, exact while i * per_token < 2^32 (launch_kv_append).
    auto token_of = [&](int i) { return tokens_per_cta == 1 ? 0 : static_cast<int>(__umulhi(i, inverse)); };
    uint4 k[kBatch], v[kBatch];
    auto load = [&](int base) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = base + u * kAppendThreads + tid, local = token_of(i);
            k[u] = v[u] = make_uint4(0, 0, 0, 0);
            if (i >= total) continue;
            const int64_t at = (first + local) * p.row_bytes + static_cast<int64_t>(i - local * per_token) * 16;
            k[u] = load_stream(reinterpret_cast<const uint4*>(static_cast<const char*>(p.k) + at));
            v[u] = load_stream(reinterpret_cast<const uint4*>(static_cast<const char*>(p.v) + at));
        }
    };
    load(0);   // rows need no slot to be read: their loads are under way while the slots are looked up
    for (int j = tid >> 5; j < tokens; j += kAppendThreads / 32) {
        const int64_t t = first + j;
        const int64_t seq = p.cu_tokens ? owner_of(p.cu_tokens, p.n_seqs, t) : t;
        if ((tid & 31) == 0) {
            const int64_t begin = p.cu_tokens ? p.cu_tokens[seq] : t, end = p.cu_tokens ? p.cu_tokens[seq + 1] : t + 1;
            int64_t page = -1, slot = 0;
            if (t >= begin && t < end) {   // rows behind the last sequence's are padding
                slot = static_cast<int64_t>(p.seq_lens[seq]) - end + t;
                if (slot >= 0 && slot < p.c.capacity) page = kv_page(p.c, seq, slot);
                else kv_bad_index();
            }
            s_row[j] = page >= 0 ? kv_row(p.c, page, 0, slot, kRow) : -1;
            s_meta[j] = page >= 0 ? kv_meta(p.c, page, 0, slot) : 0;
            s_slot[j] = static_cast<int>(slot);
        }
    }
    __syncthreads();
    Divisor ks{}, vs{};
    if constexpr (STORE == kKvFp8Static) {
        ks = divisor(*p.c.k_scale);
        vs = divisor(*p.c.v_scale);
    }
    // Every thread stays in the loop until all are done: the dynamic scale shuffles.
    for (int base = 0; base < total; base += kAppendThreads * kBatch) {
        if (base > 0) load(base);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = base + u * kAppendThreads + tid, local = min(token_of(i), tokens - 1);
            const int head = (i - local * per_token) / LANES;
            const int64_t row = s_row[local];
            const bool live = i < total && row >= 0;
            const int64_t to = row + (static_cast<int64_t>(head) << p.c.page_shift) * kRow + lane * (kRow / LANES);
            const int64_t meta = s_meta[local] + (static_cast<int64_t>(head) << p.c.page_shift);
            if constexpr (STORE == kKvBf16) {
                if (live) {
                    *reinterpret_cast<uint4*>(static_cast<char*>(p.c.k) + to) = k[u];
                    *reinterpret_cast<uint4*>(static_cast<char*>(p.c.v) + to) = v[u];
                }
            } else {
                if constexpr (STORE == kKvFp8Dynamic) {
                    float ka = amax(k[u]), va = amax(v[u]);
#pragma unroll
                    for (int o = LANES / 2; o > 0; o >>= 1) {
                        ka = fmaxf(ka, __shfl_xor_sync(0xffffffffu, ka, o));
                        va = fmaxf(va, __shfl_xor_sync(0xffffffffu, va, o));
                    }
                    ks = divisor(__fdiv_rn(ka, 448.0f));
                    vs = divisor(__fdiv_rn(va, 448.0f));
                    if (live && lane == 0) {
                        p.c.k_scale[meta] = ks.scale;
                        p.c.v_scale[meta] = vs.scale;
                    }
                }
                if (live) {
                    constexpr bool kClamp = STORE == kKvFp8Static;
                    *reinterpret_cast<uint2*>(static_cast<char*>(p.c.k) + to) = encode<kClamp>(k[u], ks);
                    *reinterpret_cast<uint2*>(static_cast<char*>(p.c.v) + to) = encode<kClamp>(v[u], vs);
                }
            }
            if (live && lane == 0) {
                if (p.c.weight) p.c.weight[meta] = 0.0f;
                if (p.c.position) p.c.position[meta] = p.positions ? p.positions[first + local] : s_slot[local];
            }
        }
    }
}

template <int STORE>
cudaError_t launch_append(const AppendParams& p, unsigned grid, int tokens, unsigned inverse, cudaStream_t s) {
    switch (p.c.head_dim) {
        case 64: return kv_launch(kv_append_kernel<STORE, 8>, grid, kAppendThreads, 0, 1, s, p, tokens, inverse);
        case 128: return kv_launch(kv_append_kernel<STORE, 16>, grid, kAppendThreads, 0, 1, s, p, tokens, inverse);
        case 256: return kv_launch(kv_append_kernel<STORE, 32>, grid, kAppendThreads, 0, 1, s, p, tokens, inverse);
    }
    return cudaErrorInvalidValue;
}

// ------------------------------------------------------------------------------------------ eviction

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;

// Dynamic shared memory for a share of `slots` slots: a key and a position each, and the lists' last entry.
constexpr size_t evict_shared(int slots) { return (static_cast<size_t>(slots) * 2 + 4) * sizeof(uint32_t); }
constexpr int kEvictMaxShared = static_cast<int>(evict_shared(MBD_KV_MAX_EVICT_CAPACITY / 16));

struct EvictSmem {
    unsigned hist[2][256];   // alternate: peers may still read one while the next is cleared
    unsigned warp_sum[kEvictWarps][2];
    unsigned total[2][2];    // this CTA's counts, read by its peers
    int max_position;
    unsigned bin, need, count;
};

// A weight as an unsigned key of the same order; -0 counts as 0 and what is not a number comes last.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = w == 0.0f ? 0u : __float_as_uint(w);
    return u ^ ((u & 0x80000000u) ? 0xffffffffu : 0x80000000u);
}

// Exclusive sums over the warps of two counts per warp, and the CTA's totals in sm.total[which]. One barrier in,
// one out.
__device__ __forceinline__ uint2 scan_warps(EvictSmem& sm, unsigned a, unsigned b, int which) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) {
        sm.warp_sum[warp][0] = a;
        sm.warp_sum[warp][1] = b;
    }
    __syncthreads();
    uint2 before = make_uint2(0, 0), all = before;
    for (int w = 0; w < kEvictWarps; ++w) {
        const unsigned x = sm.warp_sum[w][0], y = sm.warp_sum[w][1];
        if (w < warp) before = make_uint2(before.x + x, before.y + y);
        all = make_uint2(all.x + x, all.y + y);
    }
    if (threadIdx.x == 0) {
        sm.total[which][0] = all.x;
        sm.total[which][1] = all.y;
    }
    return before;
}

__device__ __forceinline__ bool on_pool(int page, const KvView& c) {
    return static_cast<uint32_t>(page) < static_cast<uint32_t>(c.n_pages);
}

__global__ void __launch_bounds__(kEvictThreads, 2) kv_evict_kernel(const __grid_constant__ EvictParams p) {
    constexpr int kLoads = 8;   // slots of a thread whose weight and position are in flight
    constexpr int kMoves = 4;   // rows of a lane group in flight
    extern __shared__ __align__(16) uint32_t slots[];   // keys [slots_per_cta], then positions, later the lists of moves
    __shared__ EvictSmem sm;
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = p.ctas_per_row, rank = static_cast<int>(blockIdx.x) % ctas;
    const int64_t row = blockIdx.x / ctas;
    const int64_t seq = row / p.c.n_kv_heads;
    const int head = static_cast<int>(row - seq * p.c.n_kv_heads);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_trigger();
    pdl_wait();
    const int64_t len = kv_len(p.c, p.seq_lens[seq]);
    if (head == 0 && rank == 0 && tid == 0) p.new_lens[seq] = static_cast<int32_t>(len < p.budget ? len : p.budget);
    if (len <= p.budget || p.budget == 0) return;   // the whole cluster

    const int share = static_cast<int>((len + ctas - 1) / ctas);
    const int64_t first = static_cast<int64_t>(rank) * share;
    const int n = static_cast<int>(max(int64_t{0}, min(static_cast<int64_t>(share), len - first)));
    uint32_t* key = slots;
    const int32_t* const table = p.c.table + seq * p.c.pages_per_seq;
    int* aux = reinterpret_cast<int*>(slots + p.slots_per_cta);

    // Loads are issued kLoads at a time without a branch between them: a thread behind the end repeats the last slot, a
    // bad page counts as page 0 until its slot's key is set.
    int newest = INT32_MIN;
    bool bad = false;
    for (int i0 = tid; i0 < n; i0 += kEvictThreads * kLoads) {
        int page[kLoads], at[kLoads];
        float w[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
            page[u] = table[(first + min(i0 + u * kEvictThreads, n - 1)) >> p.c.page_shift];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int64_t m = kv_meta(p.c, on_pool(page[u], p.c) ? page[u] : 0, head, first + min(i0 + u * kEvictThreads, n - 1));
            w[u] = p.c.weight[m];
            at[u] = p.c.position[m];
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
            const int i = i0 + u * kEvictThreads;
            const bool good = on_pool(page[u], p.c);
            bad |= !good;
            if (i < n) {
                // A bad page's slot has no row to keep and no room for one: before the budget it stays, and takes up its place;
                // behind it it comes last, and `budget` slots are found without it.
                key[i] = good ? order_key(w[u]) : (first + i < p.budget ? 0xffffffffu : 0u);
                aux[i] = good ? at[u] : INT32_MIN;
            }
            newest = max(newest, good ? at[u] : INT32_MIN);
        }
    }
    if (bad) kv_bad_index();
    if (tid == 0) sm.max_position = INT32_MIN;
    if (tid < 256) sm.hist[0][tid] = 0;
    __syncthreads();
    newest = __reduce_max_sync(0xffffffffu, newest);
    if (lane == 0) atomicMax(&sm.max_position, newest);
    if (p.recent > 0) {   // protected slots come before every weight
        cluster.sync();
        // (Here and below a lane reads a peer's word: one round trip, where a loop over the peers would wait for each.)
        const int all = __reduce_max_sync(0xffffffffu, lane < ctas ? *cluster.map_shared_rank(&sm.max_position, lane) : INT32_MIN);
        const int64_t from = static_cast<int64_t>(all) - p.recent;
        for (int i = tid; i < n; i += kEvictThreads)
            if (aux[i] > from) key[i] = 0xffffffffu;
        __syncthreads();
    }

    // The budget-th largest key: kept are the slots whose masked key is above `value`, and `need` of the `count`
    // slots where it is equal to it.
    uint32_t mask = 0, value = 0;
    unsigned need = static_cast<unsigned>(p.budget), count = 0;
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        unsigned* hist = sm.hist[pass & 1];
#pragma unroll 4
        for (int i = tid; i < n; i += kEvictThreads)
            if ((key[i] & mask) == value) atomicAdd(&hist[(key[i] >> shift) & 255u], 1u);
        cluster.sync();
        unsigned mine = 0, at_least = 0;
        if (tid < 256) {
            if (ctas == 16) {
                unsigned part[16];   // all at once: each is a round trip to another SM
#pragma unroll
                for (int r = 0; r < 16; ++r) part[r] = cluster.map_shared_rank(hist, r)[tid];
#pragma unroll
                for (int r = 0; r < 16; ++r) mine += part[r];
            } else {
#pragma unroll 4
                for (int r = 0; r < ctas; ++r) mine += cluster.map_shared_rank(hist, r)[tid];
            }
            sm.hist[(pass + 1) & 1][tid] = 0;
            at_least = mine;   // of this bin and the higher ones: within the warp, then over the warps
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned x = __shfl_down_sync(0xffffffffu, at_least, o);
                if (lane + o < 32) at_least += x;
            }
            if (lane == 0) sm.warp_sum[warp][0] = at_least;
        }
        __syncthreads();
        if (tid < 256) {
            for (int w = warp + 1; w < 8; ++w) at_least += sm.warp_sum[w][0];
            if (at_least >= need && at_least - mine < need) {
                sm.bin = tid;
                sm.need = need - (at_least - mine);
                sm.count = mine;
            }
        }
        __syncthreads();
        mask |= 255u << shift;
        value |= sm.bin << shift;
        need = sm.need;
        count = sm.count;
        if (need == count) break;   // all of them stay: the lower bits decide nothing
        __syncthreads();            // bin, need and count are read before the next pass writes them
    }

    // Ranks in slot order: each warp owns a contiguous share of this CTA's slots, 32 at a time.
    const int per_warp = (n + kEvictThreads - 1) / kEvictThreads * 32;
    const int lo = min(n, warp * per_warp), hi = min(n, lo + per_warp);
    unsigned equal_before = 0;
    if (need != count) {
        unsigned equal = 0;
#pragma unroll 4
        for (int i = lo; i < hi; i += 32)
            equal += __popc(__ballot_sync(0xffffffffu, i + lane < hi && (key[i + lane] & mask) == value));
        equal_before = scan_warps(sm, equal, 0, 0).x;
        cluster.sync();
        equal_before += __reduce_add_sync(0xffffffffu, lane < rank ? cluster.map_shared_rank(&sm.total[0][0], lane)[0] : 0u);
    }
    // kept(): whether lane's slot i + lane stays; `equal` counts the equal slots before i.
    auto kept = [&](int i, unsigned& equal) {
        const bool in = i + lane < hi;
        const uint32_t k = in ? key[i + lane] & mask : 0u;
        const bool same = in && k == value;
        bool keep = in && k > value;
        if (need == count) return keep || same;
        const unsigned who = __ballot_sync(0xffffffffu, same);
        keep |= same && equal + __popc(who & ((1u << lane) - 1u)) < need;
        equal += __popc(who);
        return keep;
    };
    unsigned holes = 0, movers = 0, equal = equal_before;
#pragma unroll 4
    for (int i = lo; i < hi; i += 32) {
        const bool in = i + lane < hi, low = first + i + lane < p.budget, keep = kept(i, equal);
        holes += __popc(__ballot_sync(0xffffffffu, in && low && !keep));
        movers += __popc(__ballot_sync(0xffffffffu, in && !low && keep));
    }
    uint2 at = scan_warps(sm, holes, movers, 1);
    cluster.sync();
    uint2 peer = make_uint2(0, 0);
    if (lane < ctas) {
        const unsigned* t = cluster.map_shared_rank(&sm.total[1][0], lane);
        peer = make_uint2(t[0], t[1]);
    }
    const unsigned moves = __reduce_add_sync(0xffffffffu, peer.y);
    at.x += __reduce_add_sync(0xffffffffu, lane < rank ? peer.x : 0u);
    at.y += __reduce_add_sync(0xffffffffu, lane < rank ? peer.y : 0u);
    // The lists, entry i with CTA i / chunk of the cluster: slots given up, then the rows that take their places.
    // (At most half of the slots move, and slots_per_cta is even: a CTA's entries fit it, and begin on eight bytes.)
    const unsigned chunk = (moves + ctas - 1) / ctas;
    // An entry is a slot's place in the pool, page * page_size + place (it fits: the host checks), or -1.
    auto token_at = [&](int64_t slot) {
        const int page = table[slot >> p.c.page_shift];
        return on_pool(page, p.c) ? (page << p.c.page_shift) + static_cast<int>(slot & ((1 << p.c.page_shift) - 1)) : -1;
    };
    if (moves > 0) {
        // e / chunk by a product: exact while e * chunk < 2^32, and 425984 slots give at most 212992 * 13312.
        const unsigned inverse = chunk > 1 ? 0xffffffffu / chunk + 1 : 0;
        const unsigned below = (1u << lane) - 1u;
        equal = equal_before;
#pragma unroll 2
        for (int i = lo; i < hi; i += 32) {
            const bool in = i + lane < hi, low = first + i + lane < p.budget, keep = kept(i, equal);
            const unsigned h = __ballot_sync(0xffffffffu, in && low && !keep);
            const unsigned m = __ballot_sync(0xffffffffu, in && !low && keep);
            const bool hole = (h >> lane) & 1u, mover = (m >> lane) & 1u;
            if (hole || mover) {
                const unsigned e = hole ? at.x + __popc(h & below) : at.y + __popc(m & below);
                const unsigned owner = chunk > 1 ? __umulhi(e, inverse) : e;
                int* list = cluster.map_shared_rank(aux, owner);
                list[(e - owner * chunk) * 2 + (mover ? 1 : 0)] = token_at(first + i + lane);
            }
            at = make_uint2(at.x + __popc(h), at.y + __popc(m));
        }
    }
    cluster.sync();   // the lists are complete; no CTA touches another's shared memory from here on
    const int mine = min(static_cast<int>(chunk), static_cast<int>(moves) - rank * static_cast<int>(chunk));
    if (mine <= 0) return;
    const int row_bytes = p.c.head_dim * (p.c.store == kKvBf16 ? 2 : 1);
    const int lanes = row_bytes / 16, part = tid % lanes, groups = kEvictThreads / lanes;   // 4 to 32 lanes own a row
    // Weights, positions and scales, a thread for a row: neighbours in the lists are neighbours in the cache, and share
    // sectors. (With the row's own lanes, one word each, they took longer than k and v: 26 of 58 thousand cycles at
    // 1546 rows of 128 bytes a CTA.)
    for (int i = tid; i < mine; i += kEvictThreads) {
        const int2 move = reinterpret_cast<const int2*>(aux)[i];
        if (move.x < 0 || move.y < 0) continue;
        const int64_t a = kv_meta(p.c, move.y >> p.c.page_shift, head, move.y), b = kv_meta(p.c, move.x >> p.c.page_shift, head, move.x);
        const float w = p.c.weight[a];
        const int32_t at_position = p.c.position[a];
        float ks = 0.0f, vs = 0.0f;
        if (p.c.store == kKvFp8Dynamic) {
            ks = p.c.k_scale[a];
            vs = p.c.v_scale[a];
        }
        p.c.weight[b] = w;
        p.c.position[b] = at_position;
        if (p.c.store == kKvFp8Dynamic) {
            p.c.k_scale[b] = ks;
            p.c.v_scale[b] = vs;
        }
    }
    for (int i0 = tid / lanes; i0 < mine; i0 += groups * kMoves) {   // loads without a branch between them, as above
        int2 move[kMoves];
        uint4 k[kMoves], v[kMoves];
#pragma unroll
        for (int u = 0; u < kMoves; ++u) {
            move[u] = reinterpret_cast<const int2*>(aux)[min(i0 + u * groups, mine - 1)];
            const int from = max(move[u].y, 0);
            const int64_t a = kv_row(p.c, from >> p.c.page_shift, head, from, row_bytes) + part * 16;
            k[u] = load_stream(reinterpret_cast<const uint4*>(static_cast<const char*>(p.c.k) + a));
            v[u] = load_stream(reinterpret_cast<const uint4*>(static_cast<const char*>(p.c.v) + a));
        }
#pragma unroll
        for (int u = 0; u < kMoves; ++u) {
            if (i0 + u * groups >= mine || move[u].x < 0 || move[u].y < 0) continue;
            const int64_t b = kv_row(p.c, move[u].x >> p.c.page_shift, head, move[u].x, row_bytes) + part * 16;
            *reinterpret_cast<uint4*>(static_cast<char*>(p.c.k) + b) = k[u];
            *reinterpret_cast<uint4*>(static_cast<char*>(p.c.v) + b) = v[u];
        }
    }
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p, int sms, cudaStream_t s) {
    // Few tokens: one to a CTA, as many SMs as there are. Many: as many as give each thread two vectors of k and of v.
    const int64_t per_token = static_cast<int64_t>(p.c.n_kv_heads) * (p.c.head_dim / 8);
    int64_t tokens = p.n_tokens < 4 * int64_t{sms} ? 1 : 2 * kAppendThreads / per_token;
    tokens = tokens < 1 ? 1 : (tokens > kAppendMaxTokens ? kAppendMaxTokens : tokens);   // (per_token is at most 512 here)
    const unsigned inverse = static_cast<unsigned>(((uint64_t{1} << 32) + per_token - 1) / per_token);
    const unsigned grid = static_cast<unsigned>((p.n_tokens + tokens - 1) / tokens);
    const int t = static_cast<int>(tokens);
    switch (p.c.store) {
        case kKvBf16: return launch_append<kKvBf16>(p, grid, t, inverse, s);
        case kKvFp8Static: return launch_append<kKvFp8Static>(p, grid, t, inverse, s);
        case kKvFp8Dynamic: return launch_append<kKvFp8Dynamic>(p, grid, t, inverse, s);
    }
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_evict(const EvictParams& p, cudaStream_t s) {
    const size_t smem = evict_shared(p.slots_per_cta);
    cudaError_t e = cudaSuccess;
    // The limit is the kernel's, not the launch's: always the largest share's, or a smaller call of another thread could
    // lower it between this call's two steps. (What a launch takes is its own size.)
    if (smem > 40 * 1024)
        e = cudaFuncSetAttribute(kv_evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictMaxShared);
    if (e == cudaSuccess && p.ctas_per_row > 8)
        e = cudaFuncSetAttribute(kv_evict_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(p.n_seqs * p.c.n_kv_heads * p.ctas_per_row);
    return kv_launch(kv_evict_kernel, grid, kEvictThreads, smem, p.ctas_per_row, s, p);
}

cudaError_t device_error_flags_kv_cache(unsigned int* flags, bool clear) { return kv_error_flags(flags, clear); }

}  // namespace mbd
